// Block cache: many-query causal attention on the 5th-generation tensor cores.
//
// A segment is (sequence, KV head, pair of query tiles); a tile is 128 rows (query token,
// head of the KV head's r), token-major, M = 128 of tcgen05.mma kind::f16. Keys come in steps
// of 128 tokens:
//   QK  S = Q code^T (f16 operands, exact codes, fp32 sums); logit x = S scale s_K.
//   PV  O += W code, W = 2^(x + log2 s_V - m + 7) in f16 with m the running maximum of
//       x + log2 s_V (raised only when it grows by more than 8, with O and the sum rescaled
//       then): weights fit f16 whatever V's range, at most 2^15, and keep all of f16's bits
//       down to 2^-21 of the largest. The denominator adds W / s_V in fp32 (units of 2^12,
//       kDenomUnit). f16 weights (off by 2^-11 of each at most, less in sum than the output's own
//       rounding) are kept for bf16 caches too: bf16 would cost eight times that.
// Scales belong to 32-token parts of a step (a part is sealed or exact as a whole), so each
// is one constant for 32 columns. Exact values and bf16 queries enter after an exact power of two
// per part or row (what f16 then drops is 2^-33 of the largest, 2^-39 for K and queries).
//
// Roles (512 threads): two softmax warpgroups, one a tile, a thread a row, its 128 logits in
// registers; an expansion warpgroup that turns codes into f16 K and V tiles (K-major, 128-byte
// swizzle, two stages; warp w takes part w of a step); a warp that issues every MMA: PV and the
// next QK of one tile run while the other tile's softmax does; one that hands out segments.
// Both tiles share each expanded K and V tile, which halves the expansion a product costs.
// Tensor memory (512 columns): S0, S1 (128 each; weights over the first half), O0, O1.
//
// Work is laid out in one of two ways, on one CTA a SM. With many segments the CTAs take whole
// ones, the longest first, from a counter. With few, all steps form one line cut evenly over the
// CTAs; a segment that crosses a cut leaves partial O, m, l in the workspace and a second kernel
// adds them in order. Either way a CTA's expansion runs on into its next segment.
// Every wait is bounded (2 s) and sets the error word when it gives up.
//
// Bound by the issue of the MMAs: one takes 64 clocks alone and about 100 while its scheduler's
// expansion warp runs. Measured, 32 / 8 heads of 128, fp16: a 4096-token prompt 121 us (1,140 TFLOP/s
// of the causal products), 512 queries against 32,768 tokens 208 us (1,310 TFLOP/s). The prompt takes 110
// us where its 75 MB stay in L2 from one call to the next, and 107 with normal values, on which no warp
// ever rescales O (28 % of a warp's steps do with outlier channels and token norms of a wide spread).
#include "kvarn_block_dev.cuh"
#include "kvarn_tc.cuh"

namespace kvarn {
namespace {

constexpr int kThreads = 512;
constexpr int kRegsLaunch = 128, kRegsSoftmax = 184, kRegsExpand = 112, kRegsIssue = 32;
static_assert(2 * kRegsSoftmax + kRegsExpand + kRegsIssue <= 4 * kRegsLaunch, "register split");
constexpr uint32_t kColS = 0, kColO = 256;
constexpr int kStep = 128;  // keys of a step
constexpr float kRaise = 8.f, kShift = 7.f;  // m is raised when it would grow by more; weights are at most 2^(both)
#define kNegInf (-__int_as_float(0x7f800000))

// feed: segments handed to the roles
constexpr int kFeed = 8;
constexpr int kBarKFull = 0, kBarVFull = 4, kBarKEmpty = 8, kBarVEmpty = 10, kBarSFull = 12, kBarPFull = 14, kBarOFull = 16,
              kBarQFull = 18, kBarDrain = 20, kBarTake = 21, kBarFeedFull = 22, kBarFeedEmpty = kBarFeedFull + kFeed,
              kNumBars = kBarFeedEmpty + kFeed;

template <int D>
struct Shape {
    static constexpr int kAtom = 128 * 128;            // 128 rows of 64 f16
    static constexpr int kQ = 0;                        // 2 tiles of D / 64 atoms
    static constexpr int kTileQ = D / 64 * kAtom;
    static constexpr int kK = kQ + 2 * kTileQ;          // 2 stages of D / 64 atoms
    static constexpr int kV = kK + 2 * kTileQ;          // 2 stages of 2 atoms (64 tokens) of D rows
    static constexpr int kTileV = 2 * D * 128;
    static constexpr int kHdr = kV + 2 * kTileV;        // float4[4][4]: by step % 4 and part
    static constexpr int kBars = kHdr + 4 * 4 * 16;
    static constexpr int kFeedAt = kBars + 8 * kNumBars;  // Seg[kFeed], where Walk looks for it
    static constexpr int kTmem = kFeedAt + 32 * kFeed;
    static_assert(kFeedAt % 16 == 0, "entries are read 16 bytes at a time");
    static constexpr int kSmem = kTmem + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

// K-major operand with 128-byte swizzle: rows of 128 bytes, 8-row groups 1024 bytes apart. Given
// by its address / 16, to which offsets of a k-step are added.
__device__ __forceinline__ uint64_t desc128(uint32_t addr16) {
    constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride, version, swizzle
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(addr16 | (1u << 16)), "n"(hi));
    return d;
}
// byte of 16-byte chunk `chunk` of row `row` in such an atom
__device__ __forceinline__ int swz(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// instruction descriptor of kind::f16: f32 accumulator, f16 operands, both K-major, M = 128
template <int N>
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
    return ok != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float max32(const uint32_t (&r)[32]) {
    float a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
#pragma unroll
    for (int k = 2; k < 30; k += 4) {
        a = max3(a, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
        b = max3(b, __uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]));
    }
    return fmaxf(max3(a, __uint_as_float(r[30]), __uint_as_float(r[31])), b);
}

// ---- the line of steps ----
// Steps of a query tile pair: up to the last position that its queries see.
__device__ __forceinline__ int pair_steps(const BlockPrefillSeq& e, int pair, int pair_tokens) {
    return (e.n - e.q_len + min((pair + 1) * pair_tokens, e.q_len) - 1) / kStep + 1;
}

// A segment: sequence entry, KV head, tile pair, its steps and the part [j0, j1) of them to take
// (j1 = 0: no more); whether its second tile has rows.
struct Seg {
    int i, kvh, pair, steps, j0, j1, two, pad;
};

// The segments of CTA b's range of the line, in order.
struct LineWalk {
    const BlockPrefillParams& p;
    int pt, left;  // query tokens of a pair; steps of the range from this segment's j0 on
    Seg s;
    __device__ __forceinline__ void set() {
        const BlockPrefillSeq& e = p.seqs[s.i];
        s.steps = pair_steps(e, s.pair, pt);
        s.j1 = left > 0 ? min(s.steps, s.j0 + left) : 0;
        s.two = (2 * s.pair + 1) * (pt / 2) < e.q_len;
    }
    __device__ __forceinline__ LineWalk(const BlockPrefillParams& p_, int b) : p(p_), pt(2 * (128 / p_.r)) {
        const int u0 = (int)((int64_t)p.steps * b / p.grid), u1 = (int)((int64_t)p.steps * (b + 1) / p.grid);
        int i = 0;
#pragma unroll 1
        while (i + 1 < p.n_seqs && p.seqs[i + 1].step_begin <= u0) ++i;
        const BlockPrefillSeq& e = p.seqs[i];
        int rel = u0 - e.step_begin, n;
        s.i = i;
        s.kvh = rel / e.head_steps;
        rel -= s.kvh * e.head_steps;
        s.pair = e.pairs - 1;
#pragma unroll 1
        while (rel >= (n = pair_steps(e, s.pair, pt))) rel -= n, --s.pair;
        s.j0 = rel;
        left = u1 - u0;
        set();
    }
    __device__ __forceinline__ void next() {
        left -= s.j1 - s.j0;
        s.j0 = 0;
        if (left > 0 && --s.pair < 0) {
            if (++s.kvh == p.c.hkv) s.kvh = 0, ++s.i;
            s.pair = p.seqs[s.i].pairs - 1;
        }
        if (left > 0) set();
        else s.j1 = 0;
    }
};

// Hands out a CTA's segments to its roles: the line's, or whole ones, the longest first, as the CTAs
// get to them (the first by the CTA's index, the next from a counter; the last CTA to run out sets
// the counters back for the next call). One entry is made ahead of what the expansion has taken.
__device__ __forceinline__ void feed_role(const BlockPrefillParams& p, uint64_t* bars, int32_t* err) {
    int32_t* counters = reinterpret_cast<int32_t*>(p.c.base + p.c.lay.counters);
    LineWalk line(p, p.line ? blockIdx.x : 0);
    Seg* ring = reinterpret_cast<Seg*>(bars + kNumBars);
    bool ok = true;
#pragma unroll 1
    for (int k = 0;; ++k) {
        if (k >= kFeed) ok = bar_wait(bars + kBarFeedEmpty + (k & (kFeed - 1)), (uint32_t)((k / kFeed - 1) & 1), err) && ok;
        if (k > 0) ok = bar_wait(bars + kBarTake, (uint32_t)((k - 1) & 1), err) && ok;
        if (p.line) {
            if (k > 0) line.next();
        } else {
            const int u = k == 0 ? (int)blockIdx.x : p.grid + atomicAdd(counters, 1);
            line.left = 0;
            if (u < p.segs) {
                int i = 0;
#pragma unroll 1
                while (i + 1 < p.n_seqs && p.seqs[i + 1].seg_begin <= u) ++i;
                const int rel = u - p.seqs[i].seg_begin;
                line.s.i = i;
                line.s.kvh = rel % p.c.hkv;
                line.s.pair = p.seqs[i].pairs - 1 - rel / p.c.hkv;
                line.s.j0 = 0;
                line.left = 1 << 30;  // all of it
            }
            line.set();
        }
        if (!ok) line.s.j1 = 0;
        ring[k & (kFeed - 1)] = line.s;
        mbar_arrive(bars + kBarFeedFull + (k & (kFeed - 1)));
        if (line.s.j1 == 0) break;
    }
    if (p.line) return;
    __threadfence();
    if (atomicAdd(counters + 1, 1) == p.grid - 1) {
        counters[0] = 0;
        counters[1] = 0;
    }
}

// A warp's way through the segments; every warp that walks takes each entry once.
struct Walk {
    uint64_t* bars;
    int k;
    Seg s;
    __device__ __forceinline__ explicit Walk(uint64_t* bars_) : bars(bars_), k(0) {}
    __device__ __forceinline__ bool next(int32_t* err) {
        // one answer for the warp: a lane that gave up alone would leave for the kernel's end while the others
        // wait for it at the next warp-wide instruction
        if (!__all_sync(0xffffffffu, bar_wait(bars + kBarFeedFull + (k & (kFeed - 1)), (uint32_t)((k / kFeed) & 1), err)))
            return false;
        const int4* at = reinterpret_cast<const int4*>(reinterpret_cast<const Seg*>(bars + kNumBars) + (k & (kFeed - 1)));
        const int4 a = at[0], b = at[1];
        s = Seg{a.x, a.y, a.z, a.w, b.x, b.y, b.z, 0};
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars + kBarFeedEmpty + (k & (kFeed - 1)));
        ++k;
        return s.j1 > 0;
    }
    __device__ __forceinline__ bool whole() const { return s.j0 == 0 && s.j1 == s.steps; }
};

// ---- the MMA issuer ----
// An MMA of this size runs 64 clocks, but takes its warp about 30 turns at a scheduler that it shares
// with two softmax warps and one of the expansion's, so that the issue, near 100 clocks an MMA, is
// what bounds a step. The whole warp walks and each MMA is predicated by itself (with a single
// thread walking, operands go through vector registers: 160 clocks), tiles are unrolled, and
// waits suspend (polling takes issue slots and shared-memory cycles from everyone). One warp
// issues both tiles' MMAs in turn, which keeps the tiles half a step apart; with a warp a tile they
// fall into step, both softmaxes run at once and then both tiles' MMAs.
template <int D>
__device__ __forceinline__ void issue_role(uint32_t sbase, uint64_t* bars, int32_t* err) {
    using Sh = Shape<D>;
    const bool leader = elect_one();
    const uint32_t base = sbase >> 4;  // (addresses stay under 2^18: descriptor fields)
    int jj = 0;
    uint32_t segs = 0, steps = 0;  // bit b: phase of tile b's segments, steps
    Walk w(bars);
#pragma unroll 1
    while (w.next(err)) {
        // broadcast from a lane, so that the loop is seen to be uniform
        const int tiles = __shfl_sync(0xffffffffu, w.s.two, 0) ? 2 : 1, j0 = __shfl_sync(0xffffffffu, w.s.j0, 0),
                  j1 = __shfl_sync(0xffffffffu, w.s.j1, 0);
        // step j0 - 1 has no PV, step j1 - 1 no QK behind it
#pragma unroll 1
        for (int j = j0 - 1; j < j1; ++j) {
            const bool more = j + 1 < j1, any = j >= j0;
            // jj: step j + 1. The expansion makes K(0) V(0) K(1) V(1) ..: the next K being there, so is this V
            const int at = more ? kBarKFull + (jj & 3) : kBarVFull + ((jj - 1) & 3);
            bar_wait(bars + at, (uint32_t)(((more ? jj : jj - 1) >> 2) & 1), err);
            const uint32_t k = base + ((Sh::kK + (jj & 1) * Sh::kTileQ) >> 4), v = base + ((Sh::kV + (~jj & 1) * Sh::kTileV) >> 4);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (b >= tiles) break;
                if (any) {
                    bar_wait(bars + kBarPFull + b, steps >> b & 1, err);
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        if (leader)
                            mma_ts(kColO + 128 * b, kColS + 128 * b + 8 * ks,
                                   desc128(v + (((ks >> 2) * (D * 128) + (ks & 3) * 32) >> 4)), kIdesc<D>,
                                   ks > 0 || j > j0 ? 1u : 0u);
                    steps ^= 1u << b;
                    if (leader && b == tiles - 1) mma_commit(bars + kBarVEmpty + (~jj & 1));
                } else {
                    bar_wait(bars + kBarQFull + b, segs >> b & 1, err);
                    segs ^= 1u << b;
                    tc_fence_after();
                }
                if (more) {
                    const uint32_t q = base + ((Sh::kQ + b * Sh::kTileQ) >> 4);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = ((ks >> 2) * Sh::kAtom + (ks & 3) * 32) >> 4;
                        if (leader) mma_ss(kColS + 128 * b, desc128(q + off), desc128(k + off), kIdesc<128>, ks > 0);
                    }
                    if (leader) mma_commit(bars + kBarSFull + b);
                    if (leader && b == tiles - 1) mma_commit(bars + kBarKEmpty + (jj & 1));
                } else if (leader) {
                    mma_commit(bars + kBarOFull + b);
                }
            }
            if (more) ++jj;
        }
    }
    if (leader) mma_commit(bars + kBarDrain);
    // every MMA has completed before tensor memory is released
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!mbar_try_wait(bars + kBarDrain, 0u) && global_ns() - t0 < kWaitLimitNs) {
    }
}

// Exact tokens of a part (none: zeros) as its K or V tile rows. A later token's infinity or NaN
// must not reach a query that does not see it through 0 x NaN: non-finite V enters as 0, and `bad`
// says that there is some, for add_non_finite at the segment's end. K needs no such care (logits
// of unseen tokens are replaced), but neither may set the part's power of two.
// h: K scale, or log2 of the V scale and kDenomUnit over it. x: registers to use.
template <int D, bool BF16, bool IS_V>
__device__ __forceinline__ void expand_exact(const BlockView& c, const BlockPrefillSeq& e, int kvh, int tile, int wp, int lane,
                                             uint8_t* dst, float2& h, uint32_t& bad, uint4 (&x)[D / 16]) {
    const int g = lane >> 2, t = lane & 3;
    const int first = (tile - (e.n >> c.log2_block << (c.log2_block - 5))) * kTileTokens;  // row of the tail
    const int nv = min(kTileTokens, e.n - tile * kTileTokens);  // valid tokens, none if <= 0
    h = IS_V ? make_float2(0.f, 1.f) : make_float2(1.f, 0.f);
    bad = 0;
    // D / 8 pieces of 16 bytes a lane, four at a time so that their loads overlap; twice, first for the largest
    constexpr int kTurn = 4;
    if (IS_V) {  // piece i: tokens 8 t .. of channel 8 i + g
        const uint16_t* v = tail_ptr(c, c.lay.tail_v, e.seq, kvh) + (ptrdiff_t)first * D;
        uint32_t keep[4];
#pragma unroll
        for (int z = 0; z < 4; ++z)
            keep[z] = (8 * t + 2 * z < nv ? 0xffffu : 0u) | (8 * t + 2 * z + 1 < nv ? 0xffff0000u : 0u);
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                x[i] = make_uint4(0, 0, 0, 0);
                if (nv > 0) x[i] = *reinterpret_cast<const uint4*>(v + (8 * (i0 + i) + g) * kTileTokens + 8 * t);
            }
#pragma unroll
            for (int i = 0; i < kTurn; ++i)
                x[i] = make_uint4(x[i].x & keep[0], x[i].y & keep[1], x[i].z & keep[2], x[i].w & keep[3]);
        };
        uint32_t top = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < D / 8; i0 += kTurn) {
            load(i0);
#pragma unroll
            for (int i = 0; i < kTurn; ++i) top = max_of(top, finite_only<BF16>(x[i]));
        }
        const int ex = warp_exponent_v<BF16>(top);
        const float f = power2(-ex);
        h = make_float2((float)ex, f * kDenomUnit);
        uint8_t* atom = dst + (wp >> 1) * (D * 128);
#pragma unroll 1
        for (int i0 = 0; i0 < D / 8; i0 += kTurn) {
            load(i0);
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                const uint4 r = x[i];
                bad |= bad_pair<BF16>(r.x) | bad_pair<BF16>(r.y) | bad_pair<BF16>(r.z) | bad_pair<BF16>(r.w);
                *reinterpret_cast<uint4*>(atom + swz(8 * (i0 + i) + g, 4 * (wp & 1) + t)) =
                    scaled_f16<BF16>(finite_only<BF16>(r), f);
            }
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
    } else {  // piece i: bytes i * 512 + lane * 16 of the part's 32 D values
        const uint16_t* k = tail_ptr(c, c.lay.tail_k, e.seq, kvh) + (ptrdiff_t)first * D;
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                const int y = (i0 + i) * 32 + lane;
                x[i] = make_uint4(0, 0, 0, 0);
                if (y / (D / 8) < nv) x[i] = *reinterpret_cast<const uint4*>(k + y * 8);
            }
        };
        float f = 1.f;
        if (BF16) {
            uint32_t top = 0;
#pragma unroll 1
            for (int i0 = 0; i0 < D / 8; i0 += kTurn) {
                load(i0);
#pragma unroll
                for (int i = 0; i < kTurn; ++i) top = max_of(top, finite_only<BF16>(x[i]));
            }
            const int ex = warp_exponent<BF16>(top) - kExactK;
            f = power2(-ex);
            h.x = power2(ex);
        }
#pragma unroll 1
        for (int i0 = 0; i0 < D / 8; i0 += kTurn) {
            load(i0);
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                const int y = (i0 + i) * 32 + lane, ch8 = y % (D / 8);
                *reinterpret_cast<uint4*>(dst + (ch8 >> 3) * Shape<D>::kAtom + swz(32 * wp + y / (D / 8), ch8 & 7)) =
                    BF16 ? scaled_f16<BF16>(x[i], f) : x[i];
            }
        }
    }
}

// Warp wp turns part wp of every step into rows of the step's K tile, then of its V tile. A lane's 16
// bytes of each chunk sit in registers and are reloaded in place: V codes while K's are converted,
// the next step's K codes while V's are. (Staging the codes in shared memory with bulk copies took
// 9 to 14 % more time.) Lanes take V's chunks in an order in which the stores of eight lanes meet
// eight different banks.
template <int D, bool INT8, bool BF16>
__device__ __forceinline__ void expand_role(const BlockPrefillParams& p, uint8_t* smem, uint64_t* bars, int32_t* err, int wp,
                                            int lane) {
    using Sh = Shape<D>;
    const BlockView& c = p.c;
    const int sh = c.log2_block - 5;
    const int t = lane & 3, kg = lane >> 2, vg = (lane >> 3) + (lane & 4);
    constexpr int kChunks = D / 16;  // 512-byte chunks of a part's K or V
    auto load_k = [&](const uint8_t* rec, int i) { return __ldg(reinterpret_cast<const uint4*>(rec + 16 + i * 512) + lane); };
    auto load_v = [&](const uint8_t* rec, int i) {
        return __ldg(reinterpret_cast<const uint4*>(rec + 16 + kTileTokens * D + i * 512) + 4 * vg + t);
    };
    auto halves = [&](uint32_t u, uint32_t v) {  // 8 codes
        return make_uint4(codes_lo<INT8>(u), codes_hi<INT8>(u), codes_lo<INT8>(v), codes_hi<INT8>(v));
    };
    // The part of a step: its sequence entry and KV head (head * 256 + entry, -1 for none), its
    // 32-token tile, with bit 31 set where the tile is exact or not there. A turn of the loop looks two
    // steps ahead (so that the pool slot is there when its address is needed), loads one ahead and
    // expands one.
    Walk w(bars);
    bool more = true;
    int j = 0, end = 0, slot = 0;  // the next step to look at, and its segment's end
    int who = -1, who1 = -1;
    uint32_t tile = 0x80000000u, tile1 = 0x80000000u;
    const uint8_t* rec = nullptr;
    uint4 x[kChunks];
    float4 hd = make_float4(1.f, 0.f, 0.f, 1.f);
#pragma unroll 1
    for (int jj = -2; jj < 0 || who >= 0; ++jj) {
        const uint8_t* rec1 = tile1 >> 31 ? nullptr : tile_ptr(c, slot, who1 >> 8, (int)tile1 & ((1 << sh) - 1));
        int who2 = -1;
        uint32_t tile2 = 0x80000000u;
        if (j == end && more) {
            more = w.next(err);
            j = w.s.j0;
            end = w.s.j1;
            if (lane == 0) mbar_arrive(bars + kBarTake);  // lets the feed make the next entry
        }
        if (more) {
            const BlockPrefillSeq& e = p.seqs[w.s.i];
            who2 = w.s.kvh * 256 + w.s.i;
            const int y = 4 * j++ + wp;
            tile2 = (uint32_t)y;
            if (y < e.n >> c.log2_block << sh) slot = __ldg(block_table(c, e.seq) + (y >> sh));
            else tile2 |= 0x80000000u;
        }
        if (jj >= 0) {
            float* head = reinterpret_cast<float*>(smem + Sh::kHdr) + ((jj & 3) * 4 + wp) * 4;
            float2 h;
            uint32_t bad = 0;
            // K
            if (jj >= 2) bar_wait(bars + kBarKEmpty + (jj & 1), (uint32_t)(((jj >> 1) - 1) & 1), err);
            uint8_t* dst = smem + Sh::kK + (jj & 1) * Sh::kTileQ;
            if (rec) {
                h = make_float2(hd.x, 0.f);
                const int row0 = 32 * wp + 8 * (kg >> 1) + (kg & 1);
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    const uint4 a = halves(x[i].x, x[i].y), b = halves(x[i].z, x[i].w);
                    x[i] = load_v(rec, i);
                    // 16 channels of one token
                    const int s = i / (D / 32), cc = i / 2 % (D / 64), row = row0 + 4 * s + 2 * (i & 1);
                    *reinterpret_cast<uint4*>(dst + cc * Sh::kAtom + swz(row, 2 * t)) = a;
                    *reinterpret_cast<uint4*>(dst + cc * Sh::kAtom + swz(row, 2 * t + 1)) = b;
                }
            } else {
                expand_exact<D, BF16, false>(c, p.seqs[who & 255], who >> 8, (int)(tile & 0x7fffffffu), wp, lane, dst, h, bad, x);
            }
            if (lane == 0) head[0] = h.x;
            fence_proxy_async_smem();
            mbar_arrive(bars + kBarKFull + (jj & 3));
            // V
            if (jj >= 2) bar_wait(bars + kBarVEmpty + (jj & 1), (uint32_t)(((jj >> 1) - 1) & 1), err);
            dst = smem + Sh::kV + (jj & 1) * Sh::kTileV;
            if (rec) {
                h = make_float2(hd.z, hd.w);
                uint8_t* to = dst + (wp >> 1) * (D * 128) + swz(vg, 4 * (wp & 1) + t);
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    // 8 tokens of channels 16 i + vg and + 8
                    *reinterpret_cast<uint4*>(to + i * 2048) = halves(x[i].x, x[i].y);
                    *reinterpret_cast<uint4*>(to + i * 2048 + 1024) = halves(x[i].z, x[i].w);
                    if (rec1) x[i] = load_k(rec1, i);
                }
            } else {
                expand_exact<D, BF16, true>(c, p.seqs[who & 255], who >> 8, (int)(tile & 0x7fffffffu), wp, lane, dst, h, bad, x);
            }
            if (lane == 0) head[1] = __uint_as_float(bad), head[2] = h.x, head[3] = h.y;
            fence_proxy_async_smem();
            mbar_arrive(bars + kBarVFull + (jj & 3));
        }
        if (rec1) {
            if (!rec) {  // nothing was reloaded in place
#pragma unroll
                for (int i = 0; i < kChunks; ++i) x[i] = load_k(rec1, i);
            }
            hd = __ldg(reinterpret_cast<const float4*>(rec1));
        }
        who = who1;
        tile = tile1;
        rec = rec1;
        who1 = who2;
        tile1 = tile2;
    }
}

// Non-finite V of exact tokens went into the products as 0. Here a row takes those of the positions
// [from, to) that it sees, each into its own channel: on top of the finished row `out`, or of the
// partial one `part` (the other null).
template <int D, bool BF16>
__device__ __forceinline__ void add_non_finite(const BlockView& c, const BlockPrefillSeq& e, int kvh, int from, int to,
                                               uint16_t* out, float* part) {
    const int sealed = e.n & ~(c.block - 1);
    const uint16_t* v = tail_ptr(c, c.lay.tail_v, e.seq, kvh);
#pragma unroll 1
    for (int ch = 0; ch < D; ++ch) {
        float sum = 0.f;
#pragma unroll 1
        for (int pos = max(from, sealed); pos < to; ++pos) {
            const uint32_t x = v[tail_v_off(D, pos - sealed, ch)];
            if (bad_pair<BF16>(x)) sum += unpack2<BF16>(x).x;
        }
        if (sum == 0.f) continue;
        if (out) out[ch] = (uint16_t)pack2<BF16>(unpack2<BF16>(out[ch]).x + sum, 0.f);
        else part[ch] += sum;
    }
}

// ---- softmax: thread et owns row et of tile b ----
template <int D, bool BF16>
__device__ __forceinline__ void softmax_role(const BlockPrefillParams& p, uint8_t* smem, uint64_t* bars, uint32_t tmem,
                                             int32_t* err, int et, int b, uint32_t lane_off) {
    using Sh = Shape<D>;
    const uint32_t ts = tmem + kColS + 128 * b + lane_off, to = tmem + kColO + 128 * b + lane_off;
    const int tpt = 128 / p.r, tok_in = et / p.r, head_in = et % p.r, lane = et & 31;
    const float4* hdr = reinterpret_cast<const float4*>(smem + Sh::kHdr);
    // the warp's 32 rows of the tile's Q: query rows on the way in, output rows on the way out
    uint8_t* rows = smem + Sh::kQ + b * Sh::kTileQ + (et & 96) * 128;
    // a negative scale turns the query's sign, so that larger S is always a larger logit
    // (and a scale of 0 the query to zeros: every logit is 0)
    const bool zero = p.scale_log2 == 0.f;
    const float scale = zero ? 1.f : fabsf(p.scale_log2);
    const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    int jj = 0, step = 0, seg = 0;
    Walk w(bars);
#pragma unroll 1
    while (w.next(err)) {
        if (b == 1 && !w.s.two) {
            jj += w.s.j1 - w.s.j0;
            continue;
        }
        const BlockPrefillSeq& e = p.seqs[w.s.i];
        const int tok = (2 * w.s.pair + b) * tpt + tok_in;
        const bool valid = tok_in < tpt && tok < e.q_len;
        const int row = valid ? (e.q_row + tok) * p.hq + w.s.kvh * p.r + head_in : -1;  // of q and out
        const int pos = valid ? e.n - e.q_len + tok : e.n - 1;
        float qs = scale;
        {
            // D / 8 lanes a row; loops stay short: this code runs once a segment, from a cold cache
            constexpr int kLanes = D / 8, kRows = 32 / kLanes, kTurn = 8;
#pragma unroll 1
            for (int i0 = 0; i0 < kLanes; i0 += kTurn) {
                uint4 x[kTurn];
#pragma unroll
                for (int z = 0; z < kTurn; ++z) {
                    const int at = __shfl_sync(0xffffffffu, row, (i0 + z) * kRows + lane / kLanes);
                    x[z] = make_uint4(0, 0, 0, 0);
                    if (at >= 0 && !zero) x[z] = reinterpret_cast<const uint4*>(p.q + (size_t)at * D)[lane % kLanes];
                }
#pragma unroll
                for (int z = 0; z < kTurn; ++z) {
                    const int i = i0 + z;
                    uint4 r = x[z];
                    if (BF16) {
                        uint32_t top = max_of(0, r);
                        top = max(top & 0xffffu, top >> 16);
#pragma unroll
                        for (int d = kLanes / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const int ex = exponent_of<BF16>(top) - kExactK;
                        r = scaled_f16<BF16>(r, power2(-ex));
                        const int mine = __shfl_sync(0xffffffffu, ex, lane % kRows * kLanes);  // of row i kRows + lane % kRows
                        if (lane / kRows == i) qs *= power2(mine);
                    }
                    r = make_uint4(r.x ^ sign, r.y ^ sign, r.z ^ sign, r.w ^ sign);
                    *reinterpret_cast<uint4*>(rows + (lane % kLanes >> 3) * Sh::kAtom + swz(i * kRows + lane / kLanes, lane & 7)) = r;
                }
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(bars + kBarQFull + b);
        float m = kNegInf, l = 0.f;
        uint32_t bad = 0;  // non-finite V among the segment's exact tokens
#pragma unroll 1
        for (int j = w.s.j0; j < w.s.j1; ++j, ++jj, ++step) {
            // A tile that sat out a segment may be whole phases ahead of the expansion; once its first
            // step's QK is done both barriers are at that step's phase or the one before. Within a
            // segment they are waited for first, and the headers read, while QK runs.
            if (j == w.s.j0) bar_wait(bars + kBarSFull + b, (uint32_t)(step & 1), err);
            bar_wait(bars + kBarKFull + (jj & 3), (uint32_t)((jj >> 2) & 1), err);
            bar_wait(bars + kBarVFull + (jj & 3), (uint32_t)((jj >> 2) & 1), err);
            // logit = S c[ch] (+ log2 of V's scale in the weight); c > 0 or NaN
            float c[4], lv[4], iv[4];
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
                const float4 h = hdr[(jj & 3) * 4 + ch];
                c[ch] = qs * h.x;
                if (c[ch] < 1e-37f) c[ch] = 1e-37f;  // 0 would make -inf of a masked column NaN
                lv[ch] = h.z;
                iv[ch] = h.w;
                bad |= __float_as_uint(h.y);
            }
            bar_wait(bars + kBarSFull + b, (uint32_t)(step & 1), err);
            tc_fence_after();
            const int lim = pos + 1 - j * kStep;  // visible columns
            uint32_t r[4][32];
            float mx = kNegInf;
            const bool plain = __all_sync(0xffffffffu, lim >= kStep);
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) tm_ld32(ts + 32 * ch, r[ch]);
            tm_wait_ld();
            if (__builtin_expect(plain, 1)) {
                mx = fmaxf(mx, fmaf(max32(r[0]), c[0], lv[0]));
                mx = fmaxf(mx, fmaf(max32(r[1]), c[1], lv[1]));
                mx = fmaxf(mx, fmaf(max32(r[2]), c[2], lv[2]));
                mx = fmaxf(mx, fmaf(max32(r[3]), c[3], lv[3]));
            } else {
                // columns behind the row's position leave, with all of a part that is not seen at all
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    const int left = lim - 32 * ch;  // visible columns from the part's first on
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (k >= left) r[ch][k] = 0xff800000u;
                    if (left <= 0) c[ch] = 1.f, lv[ch] = 0.f, iv[ch] = 1.f;
                    mx = fmaxf(mx, fmaf(max32(r[ch]), c[ch], lv[ch]));
                }
            }
            const bool up = mx > m + kRaise;  // also from -inf
            const bool rescale = __any_sync(0xffffffffu, up);
            const float f = up ? ex2f(m - mx) : 1.f;  // 0 from -inf
            if (up) m = mx;
            l *= f;
            const float mm = m == kNegInf ? 0.f : m - kShift;
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
                const float ad = lv[ch] - mm;
                const float2 c2 = make_float2(c[ch], c[ch]), a2 = make_float2(ad, ad);
                float2 s0 = make_float2(0.f, 0.f), s1 = s0;
                uint32_t o[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 x =
                        __ffma2_rn(make_float2(__uint_as_float(r[ch][2 * k]), __uint_as_float(r[ch][2 * k + 1])), c2, a2);
                    const float2 y = make_float2(ex2f(x.x), ex2f(x.y));
                    if (k & 1) s1 = __fadd2_rn(s1, y);
                    else s0 = __fadd2_rn(s0, y);
                    o[k] = h2u(__float22half2_rn(y));
                }
                s0 = __fadd2_rn(s0, s1);
                l = fmaf(s0.x + s0.y, iv[ch], l);
                tm_st16(ts + 16 * ch, o);
            }
            if (rescale && j > w.s.j0) {  // O, now that the logits' registers are free
#pragma unroll 1
                for (int ch = 0; ch < D / 64; ++ch) {
                    uint32_t o[2][32];
                    tm_ld32(to + 64 * ch, o[0]);
                    tm_ld32(to + 64 * ch + 32, o[1]);
                    tm_wait_ld();
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[z][k] = __float_as_uint(__uint_as_float(o[z][k]) * f);
                        tm_st32(to + 64 * ch + 32 * z, o[z]);
                    }
                }
            }
            tm_wait_st();
            tc_fence_before();
            mbar_arrive(bars + kBarPFull + b);
        }
        bar_wait(bars + kBarOFull + b, (uint32_t)(seg++ & 1), err);
        tc_fence_after();
        // out through the warp's Q rows (their MMAs are done), 128 bytes a row at a time, so that a row
        // leaves in whole sectors
        auto give = [&](int piece, const uint32_t (&o)[32]) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4*>(rows + piece * Sh::kAtom + swz(lane, k)) =
                    make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        };
        auto take = [&](int piece, int k) {  // 16 bytes of row 4 k + lane / 8
            return *reinterpret_cast<const uint4*>(rows + piece * Sh::kAtom + swz(4 * k + (lane >> 3), lane & 7));
        };
        if (w.whole()) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
            for (int piece = 0; piece < D / 64; ++piece) {
                uint32_t x[2][32], o[32];
                tm_ld32(to + 64 * piece, x[0]);
                tm_ld32(to + 64 * piece + 32, x[1]);
                tm_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    o[k] = pack2<BF16>(__uint_as_float(x[k >> 4][2 * k & 31]) * kDenomUnit * inv,
                                       __uint_as_float(x[k >> 4][(2 * k & 31) + 1]) * kDenomUnit * inv);
                give(piece, o);
            }
            __syncwarp();
#pragma unroll 4
            for (int k = 0; k < 8; ++k) {
                const int at = __shfl_sync(0xffffffffu, row, 4 * k + (lane >> 3));
#pragma unroll
                for (int piece = 0; piece < D / 64; ++piece) {
                    const uint4 x = take(piece, k);
                    if (at >= 0) *reinterpret_cast<uint4*>(p.out + (size_t)at * D + 64 * piece + 8 * (lane & 7)) = x;
                }
            }
            if (__builtin_expect(bad, 0)) {
                __syncwarp();  // the row is there
                if (valid) add_non_finite<D, BF16>(p.c, e, w.s.kvh, 0, pos + 1, p.out + (size_t)row * D, nullptr);
            }
        } else {
            float* part = reinterpret_cast<float*>(p.c.base + p.c.lay.partials) +
                          (size_t)(2 * blockIdx.x + (w.s.j0 == 0 ? 1 : 0)) * (256 * (D + 2));
            const int first = 128 * b + (et & 96);
            if (__any_sync(0xffffffffu, row >= 0)) {  // (rows without a query are not read back)
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t x[32];
                    tm_ld32(to + 32 * ch, x);
                    tm_wait_ld();
                    give(0, x);
                    __syncwarp();
#pragma unroll 4
                    for (int k = 0; k < 8; ++k) {
                        const int rr = first + 4 * k + (lane >> 3);
                        *reinterpret_cast<uint4*>(part + (size_t)rr * D + 32 * ch + 4 * (lane & 7)) = take(0, k);
                    }
                    __syncwarp();
                }
                if (__builtin_expect(bad, 0) && valid)
                    add_non_finite<D, BF16>(p.c, e, w.s.kvh, w.s.j0 * kStep, min(pos + 1, w.s.j1 * kStep), nullptr,
                                            part + (size_t)(128 * b + et) * D);
                part[256 * D + 128 * b + et] = m;
                part[256 * D + 256 + 128 * b + et] = l;
            }
        }
        __syncwarp();
        tc_fence_before();  // O has been read before this thread lets the next segment's PV start
    }
}

template <int D, bool INT8, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ BlockPrefillParams p) {
    using Sh = Shape<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int t = threadIdx.x, w = t >> 5, lane = t & 31, wg = w >> 2;
    int32_t* err = reinterpret_cast<int32_t*>(p.c.base + p.c.lay.err);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kBars);
    if (t == 0) {
        for (int k = 0; k < 4; ++k) {
            mbar_init(bars + kBarKFull + k, 128);
            mbar_init(bars + kBarVFull + k, 128);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(bars + kBarKEmpty + k, 1);
            mbar_init(bars + kBarVEmpty + k, 1);
            mbar_init(bars + kBarSFull + k, 1);
            mbar_init(bars + kBarPFull + k, 128);
            mbar_init(bars + kBarOFull + k, 1);
            mbar_init(bars + kBarQFull + k, 128);
        }
        mbar_init(bars + kBarDrain, 1);
        mbar_init(bars + kBarTake, 4);  // the expansion's warps
        for (int k = 0; k < kFeed; ++k) {
            mbar_init(bars + kBarFeedFull + k, 1);
            mbar_init(bars + kBarFeedEmpty + k, 13);  // the warps that walk: 8 softmax, 4 expansion, 1 issuer
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (w == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(smem + Sh::kTmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // All of tensor memory is this CTA's, so it starts at address 0, and shared memory on 1024 bytes;
    // both are counted on below. Were it ever not so, the launch would do nothing but say so.
    const bool placed = *reinterpret_cast<volatile uint32_t*>(smem + Sh::kTmem) == 0 && (smem_addr(smem) & 1023) == 0;
    constexpr uint32_t tmem = 0;
    if (!placed && t == 0) atomicOr(err, kErrBadSlot);
    const uint32_t lane_off = (uint32_t)(32 * (w & 3)) << 16;
    if (!placed) {
    } else if (wg < 2) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_role<D, BF16>(p, smem, bars, tmem, err, t & 127, wg, lane_off);
    } else if (wg == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
        expand_role<D, INT8, BF16>(p, smem, bars, err, w & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (w == 12) issue_role<D>(smem_addr(smem), bars, err);
        else if (w == 13 && lane == 0) feed_role(p, bars, err);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 12) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*reinterpret_cast<volatile uint32_t*>(smem + Sh::kTmem))
                     : "memory");
    }
}

// Adds the partials of the segment that begins in CTA b's range and ends behind it, in the order
// of the cuts. A warp (half of one at head_dim 64) a row, 4 channels a lane; the parts' maxima and
// sums 32 at a time, a lane each, then their rows eight at a time. blockIdx.y: kCombineRows rows.
constexpr int kCombineThreads = 256;
template <int D, bool BF16>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ BlockPrefillParams p) {
    constexpr int kCombineRows = kCombineThreads / 32;
    const int b = blockIdx.x, lane = threadIdx.x & 31;
    const int u0 = (int)((int64_t)p.steps * b / p.grid), u1 = (int)((int64_t)p.steps * (b + 1) / p.grid);
    LineWalk w(p, b);
    int u = u0;
#pragma unroll 1
    while (u + (w.s.j1 - w.s.j0) < u1) u += w.s.j1 - w.s.j0, w.next();
    if (w.s.j0 > 0 || w.s.j1 == w.s.steps) return;  // no segment both begins here and goes on
    const BlockPrefillSeq& e = p.seqs[w.s.i];
    const int tpt = 128 / p.r, rr = blockIdx.y * kCombineRows + threadIdx.x / 32, et = rr & 127;
    const int tok = (2 * w.s.pair + (rr >> 7)) * tpt + et / p.r;
    if (et / p.r >= tpt || tok >= e.q_len) return;
    const int parts = (int)(((int64_t)(u + w.s.steps) * p.grid - 1) / p.steps) - b + 1;
    const bool live = 4 * lane < D;
    constexpr size_t kPart = 256 * (D + 2);
    const float* base = reinterpret_cast<const float*>(p.c.base + p.c.lay.partials);
    // part z: slot 1 of the CTA where the segment begins, slot 0 of the others
    auto part = [&](int z) { return base + (size_t)(2 * (b + z) + (z == 0 ? 1 : 0)) * kPart; };
    float big = kNegInf, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int z0 = 0; z0 < parts; z0 += 32) {
        const int n = min(32, parts - z0);
        float m = kNegInf, s = 0.f;
        if (lane < n) {
            m = part(z0 + lane)[256 * D + rr];
            s = part(z0 + lane)[256 * D + 256 + rr];
        }
        float top = m;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(top, big);
        const float f = m == kNegInf ? 1.f : ex2f(m - top), g = big == kNegInf ? 1.f : ex2f(big - top);  // -inf: zeros or NaN
        s *= f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        l = fmaf(l, g, s);
        o.x *= g, o.y *= g, o.z *= g, o.w *= g;
        big = top;
#pragma unroll 8
        for (int z = 0; z < n; ++z) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (live) x = *reinterpret_cast<const float4*>(part(z0 + z) + (size_t)rr * D + 4 * lane);
            const float y = __shfl_sync(0xffffffffu, f, z);
            o.x = fmaf(x.x, y, o.x);
            o.y = fmaf(x.y, y, o.y);
            o.z = fmaf(x.z, y, o.z);
            o.w = fmaf(x.w, y, o.w);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l, y = kDenomUnit;
    const size_t row = ((size_t)(e.q_row + tok) * p.hq + w.s.kvh * p.r + et % p.r) * D;
    if (live)
        *reinterpret_cast<uint2*>(p.out + row + 4 * lane) =
            make_uint2(pack2<BF16>(o.x * y * inv, o.y * y * inv), pack2<BF16>(o.z * y * inv, o.w * y * inv));
}

template <int D, bool INT8, bool BF16>
int launch(const BlockPrefillParams& p, cudaStream_t s) {
    static SmemOnce once;
    const int e = once.allow(reinterpret_cast<const void*>(prefill_kernel<D, INT8, BF16>), Shape<D>::kSmem);
    if (e) return e;
    prefill_kernel<D, INT8, BF16><<<p.grid, kThreads, Shape<D>::kSmem, s>>>(p);
    if (p.line) combine_kernel<D, BF16><<<dim3(p.grid, 256 / (kCombineThreads / 32)), kCombineThreads, 0, s>>>(p);
    return (int)cudaGetLastError();
}

}  // namespace

int launch_block_prefill(const BlockPrefillParams& p, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    switch ((p.c.d == 128 ? 4 : 0) + (p.c.int8 ? 2 : 0) + (p.c.bf16 ? 1 : 0)) {
        case 0: return launch<64, false, false>(p, s);
        case 1: return launch<64, false, true>(p, s);
        case 2: return launch<64, true, false>(p, s);
        case 3: return launch<64, true, true>(p, s);
        case 4: return launch<128, false, false>(p, s);
        case 5: return launch<128, false, true>(p, s);
        case 6: return launch<128, true, false>(p, s);
        default: return launch<128, true, true>(p, s);
    }
}

}  // namespace kvarn
