// Block cache: many-query causal attention on the 5th-generation tensor cores.
//
// A segment is (sequence, KV head, pair of query tiles); a tile is 128 rows (query token,
// head of the KV head's r), token-major, M = 128 of tcgen05.mma kind::f16. Keys come in steps
// of 128 tokens:
//   QK  S = Q code^T (f16 operands, exact codes, fp32 sums); logit x = S scale s_K.
//   PV  O += W code, W = 2^(x + log2 s_V - m) in f16 with m the running maximum of x + log2 s_V
//       (raised only when it grows by more than 8, with O and the sum rescaled then), so
//       weights fit f16 whatever V's range; the denominator adds W / s_V in fp32. f16 weights
//       (rounded by 2^-12) are kept for bf16 caches too: bf16 would cost eight times that.
// Scales belong to 32-token parts of a step (a part is sealed or exact as a whole), so each
// is one constant for 32 columns. Exact fp16 values enter as they are; exact bf16 values and
// bf16 queries after an exact power of two per part or row (what that drops is 2^-39 of the
// largest).
//
// Roles (512 threads): two softmax warpgroups, one a tile, a thread a row, its 128 logits in
// registers; an expansion warpgroup that turns codes into f16 K and V tiles (K-major, 128-byte
// swizzle, two stages; warp w takes part w of a step); a warp that issues every MMA: PV and the
// next QK of one tile run while the other tile's softmax does. Both tiles share each
// expanded K and V tile, which halves the expansion a product costs.
// Tensor memory (512 columns): S0, S1 (128 each; weights over the first half), O0, O1.
//
// Work is laid out in one of two ways. With many segments a CTA takes one each, the longest
// first. With few, all steps form one line cut evenly over the CTAs; a segment that crosses
// a cut leaves partial O, m, l in the workspace and a second kernel adds them in order.
// Every wait is bounded (2 s) and sets the error word when it gives up.
#include "kvarn_block_dev.cuh"
#include "kvarn_tc.cuh"

namespace kvarn {
namespace {

constexpr int kThreads = 512;
constexpr int kRegsLaunch = 128, kRegsSoftmax = 184, kRegsExpand = 104, kRegsIssue = 40;
static_assert(2 * kRegsSoftmax + kRegsExpand + kRegsIssue <= 4 * kRegsLaunch, "register split");
constexpr uint32_t kColS = 0, kColO = 256;
constexpr int kStep = 128;  // keys of a step
#define kNegInf (-__int_as_float(0x7f800000))

// p_full: by tile, two halves of 64 keys each (2 b + half)
constexpr int kBarKFull = 0, kBarVFull = 4, kBarKEmpty = 8, kBarVEmpty = 10, kBarSFull = 12, kBarPFull = 14, kBarOFull = 18,
              kBarQFull = 20, kBarDrain = 22, kNumBars = 23;

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
    static constexpr int kTmem = kBars + 8 * kNumBars;
    static constexpr int kSmem = kTmem + 16 + 1024;     // slack to start on 1024 bytes
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
__device__ __forceinline__ void tm_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
    return ok != 0;
}
// mbar_wait for the waits that every step's latency goes through: polls without suspending first.
__device__ __forceinline__ void mbar_spin(uint64_t* bar, uint32_t parity, int32_t* err) {
    for (int i = 0; i < 1024; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (ok) return;
    }
    mbar_wait(bar, parity, err);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// ---- the line of steps ----
// Steps of a query tile pair: up to the last position that its queries see.
__device__ __forceinline__ int pair_steps(const BlockPrefillSeq& e, int pair, int pair_tokens) {
    return (e.n - e.q_len + min((pair + 1) * pair_tokens, e.q_len) - 1) / kStep + 1;
}

// The segments (steps [j0, j1) of each) of CTA b in order.
struct Walk {
    const BlockPrefillParams& p;
    int pt, left;  // query tokens of a pair; steps of this CTA behind this segment's j0
    int i, kvh, pair, steps, j0, j1;
    __device__ __forceinline__ Walk(const BlockPrefillParams& p_, int b) : p(p_) {
        pt = 2 * (128 / p.r);
        int lo = 0, rel;
        if (!p.line) {
            for (int hi = p.n_seqs - 1; lo < hi;) {
                const int mid = (lo + hi + 1) / 2;
                if (p.seqs[mid].cta_begin <= b) lo = mid; else hi = mid - 1;
            }
            i = lo;
            rel = b - p.seqs[i].cta_begin;
            kvh = rel % p.c.hkv;
            pair = p.seqs[i].pairs - 1 - rel / p.c.hkv;
            steps = pair_steps(p.seqs[i], pair, pt);
            j0 = 0;
            j1 = left = steps;
            return;
        }
        const int u0 = (int)((int64_t)p.steps * b / p.grid), u1 = (int)((int64_t)p.steps * (b + 1) / p.grid);
        for (int hi = p.n_seqs - 1; lo < hi;) {
            const int mid = (lo + hi + 1) / 2;
            if (p.seqs[mid].step_begin <= u0) lo = mid; else hi = mid - 1;
        }
        i = lo;
        rel = u0 - p.seqs[i].step_begin;
        kvh = rel / p.seqs[i].head_steps;
        rel -= kvh * p.seqs[i].head_steps;
        pair = p.seqs[i].pairs - 1;
        while (rel >= (steps = pair_steps(p.seqs[i], pair, pt))) rel -= steps, --pair;
        j0 = rel;
        left = u1 - u0;
        j1 = min(steps, j0 + left);
    }
    __device__ __forceinline__ bool valid() const { return left > 0; }
    __device__ __forceinline__ void next() {
        left -= j1 - j0;
        if (left <= 0) return;
        if (--pair < 0) {
            if (++kvh == p.c.hkv) kvh = 0, ++i;
            pair = p.seqs[i].pairs - 1;
        }
        steps = pair_steps(p.seqs[i], pair, pt);
        j0 = 0;
        j1 = min(steps, left);
    }
    __device__ __forceinline__ bool two() const { return (2 * pair + 1) * (pt / 2) < p.seqs[i].q_len; }  // the second tile has rows
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == steps; }
};

__device__ __forceinline__ int bf16_exponent(uint32_t top) { return max((int)(top >> 7) - 127, -100); }
__device__ __forceinline__ float power2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ uint32_t scaled_f16(uint32_t w, float f) {
    const float2 a = unpack2<true>(w);
    return pack2<false>(a.x * f, a.y * f);
}
__device__ __forceinline__ uint4 scaled_f16(uint4 w, float f) {
    return make_uint4(scaled_f16(w.x, f), scaled_f16(w.y, f), scaled_f16(w.z, f), scaled_f16(w.w, f));
}
__device__ __forceinline__ uint32_t max_of(uint32_t top, uint4 x) {
    top = __vmaxu2(top, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu));
    return __vmaxu2(top, __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
}
__device__ __forceinline__ int warp_exponent(uint32_t top) {
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    return bf16_exponent(top) - 14;
}

// ---- the MMA issuer ----
// The whole warp walks and waits, so that addresses stay in uniform registers; one lane issues.
// (With a single thread walking, each MMA took its operands through vector registers and
// eight of them about 1,300 clocks to issue; they run in 512.)
template <int D>
__device__ __forceinline__ void issue_role(const BlockPrefillParams& p, uint32_t sbase, uint64_t* bars, uint32_t tmem,
                                           int32_t* err) {
    using Sh = Shape<D>;
    const bool leader = elect_one();
    sbase >>= 4;  // (addresses stay under 2^18: descriptor fields)
    auto qk = [&](int b, int jj) {
        const uint32_t q = sbase + ((Sh::kQ + b * Sh::kTileQ) >> 4), k = sbase + ((Sh::kK + (jj & 1) * Sh::kTileQ) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * Sh::kAtom + (ks & 3) * 32) >> 4;
            if (leader) mma_ss(tmem + kColS + 128 * b, desc128(q + off), desc128(k + off), kIdesc<128>, ks > 0);
        }
        if (leader) mma_commit(bars + kBarSFull + b);
    };
    auto pv = [&](int b, int jj, int half, uint32_t acc) {  // 64 keys
        const uint32_t v = sbase + ((Sh::kV + (jj & 1) * Sh::kTileV + half * (D * 128)) >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            if (leader)
                mma_ts(tmem + kColO + 128 * b, tmem + kColS + 128 * b + 32 * half + 8 * ks, desc128(v + 2 * ks), kIdesc<D>,
                       ks > 0 ? 1u : acc);
    };
    int jj = 0;
    uint32_t segs = 0, steps = 0;  // bit b: phase of tile b's segments, steps
    for (Walk w(p, blockIdx.x); w.valid(); w.next()) {
        const int tiles = w.two() ? 2 : 1;
#pragma unroll 1
        for (int b = 0; b < tiles; ++b) {
            mbar_wait(bars + kBarQFull + b, segs >> b & 1, err);
            segs ^= 1u << b;
        }
        mbar_wait(bars + kBarKFull + (jj & 3), (uint32_t)((jj >> 2) & 1), err);
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < tiles; ++b) qk(b, jj);
        if (leader) mma_commit(bars + kBarKEmpty + (jj & 1));
#pragma unroll 1
        for (int j = w.j0; j < w.j1; ++j, ++jj) {
            mbar_wait(bars + kBarVFull + (jj & 3), (uint32_t)((jj >> 2) & 1), err);
            const bool more = j + 1 < w.j1;
#pragma unroll 1
            for (int b = 0; b < tiles; ++b) {
                mbar_spin(bars + kBarPFull + 2 * b, steps >> b & 1, err);
                tc_fence_after();
                pv(b, jj, 0, j > w.j0 ? 1u : 0u);
                mbar_spin(bars + kBarPFull + 2 * b + 1, steps >> b & 1, err);
                steps ^= 1u << b;
                tc_fence_after();
                pv(b, jj, 1, 1u);
                if (b == tiles - 1 && leader) mma_commit(bars + kBarVEmpty + (jj & 1));
                if (more) {
                    if (b == 0) {
                        mbar_wait(bars + kBarKFull + ((jj + 1) & 3), (uint32_t)(((jj + 1) >> 2) & 1), err);
                        tc_fence_after();
                    }
                    qk(b, jj + 1);
                    if (b == tiles - 1 && leader) mma_commit(bars + kBarKEmpty + ((jj + 1) & 1));
                } else if (leader) {
                    mma_commit(bars + kBarOFull + b);
                }
            }
        }
    }
    if (leader) mma_commit(bars + kBarDrain);
}

// ---- expansion: one part (32 tokens) a warp ----
// The steps of a CTA in order, for the expansion warps.
struct StepWalk {
    Walk w;
    int j;
    __device__ __forceinline__ StepWalk(const BlockPrefillParams& p, int b) : w(p, b), j(w.j0) {}
    __device__ __forceinline__ bool valid() const { return w.valid(); }
    __device__ __forceinline__ void next() {
        if (++j < w.j1) return;
        w.next();
        j = w.j0;
    }
};

// Non-finite 16-bit values of a word, as the bits of a pair (bit 0, bit 1).
template <bool BF16>
__device__ __forceinline__ uint32_t bad_pair(uint32_t w) {
    constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
    return ((w & e) == e ? 1u : 0u) | ((w >> 16 & e) == e ? 2u : 0u);
}
// The word with its non-finite values made zero.
template <bool BF16>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
    const uint32_t b = bad_pair<BF16>(w);
    return w & ((b & 1 ? 0u : 0xffffu) | (b & 2 ? 0u : 0xffff0000u));
}
template <bool BF16>
__device__ __forceinline__ uint4 finite_only(uint4 w) {
    return make_uint4(finite_only<BF16>(w.x), finite_only<BF16>(w.y), finite_only<BF16>(w.z), finite_only<BF16>(w.w));
}

// Exact tokens of a part (none: zeros) as its K or V tile rows. A later token's infinity or NaN
// must not reach a query that does not see it through 0 x NaN: non-finite V enters as 0, and its
// token is named in `bad` for the softmax to make visible weights NaN. K needs no such care (logits
// of unseen tokens are replaced), but neither may set the part's power of two.
// h: K scale, or log2 and reciprocal of the V scale.
template <int D, bool BF16, bool IS_V>
__device__ __forceinline__ void expand_exact(const BlockView& c, const BlockPrefillSeq& e, int kvh, int tile, int wp, int lane,
                                             uint8_t* dst, float2& h, uint32_t& bad) {
    const int g = lane >> 2, t = lane & 3;
    const int first = (tile - (e.n >> c.log2_block << (c.log2_block - 5))) * kTileTokens;  // row of the tail
    const int nv = min(kTileTokens, e.n - tile * kTileTokens);  // valid tokens, none if <= 0
    h = IS_V ? make_float2(0.f, 1.f) : make_float2(1.f, 0.f);
    bad = 0;
    float f = 1.f;
    if (IS_V) {
        const uint16_t* v = tail_ptr(c, c.lay.tail_v, e.seq, kvh) + first;
        uint32_t keep[4];
#pragma unroll
        for (int z = 0; z < 4; ++z)
            keep[z] = (8 * t + 2 * z < nv ? 0xffffu : 0u) | (8 * t + 2 * z + 1 < nv ? 0xffff0000u : 0u);
        auto row = [&](int ch) {
            if (nv <= 0) return make_uint4(0, 0, 0, 0);
            const uint4 r = *reinterpret_cast<const uint4*>(v + (size_t)ch * c.block + 8 * t);
            return make_uint4(r.x & keep[0], r.y & keep[1], r.z & keep[2], r.w & keep[3]);
        };
        if (BF16) {
            uint32_t top = 0;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) top = max_of(top, finite_only<BF16>(row(8 * i + g)));
            const int ex = warp_exponent(top);
            f = power2(-ex);
            h = make_float2((float)ex, f);
        }
        uint8_t* atom = dst + (wp >> 1) * (D * 128);
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
            uint4 r = row(8 * i + g);
            bad |= (bad_pair<BF16>(r.x) | bad_pair<BF16>(r.y) << 2 | bad_pair<BF16>(r.z) << 4 | bad_pair<BF16>(r.w) << 6) << (8 * t);
            r = finite_only<BF16>(r);
            if (BF16) r = scaled_f16(r, f);
            *reinterpret_cast<uint4*>(atom + swz(8 * i + g, 4 * (wp & 1) + t)) = r;
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
    } else {
        const uint16_t* k = tail_ptr(c, c.lay.tail_k, e.seq, kvh) + (ptrdiff_t)first * D;
        auto piece = [&](int z) {  // 16 bytes z * 32 + lane of the part's 32 D values
            const int y = z * 32 + lane, tok = y / (D / 8);
            if (tok >= nv) return make_uint4(0, 0, 0, 0);
            return *reinterpret_cast<const uint4*>(k + tok * D + y % (D / 8) * 8);
        };
        if (BF16) {
            uint32_t top = 0;
#pragma unroll 4
            for (int z = 0; z < D / 8; ++z) top = max_of(top, finite_only<BF16>(piece(z)));
            const int ex = warp_exponent(top);
            f = power2(-ex);
            h.x = power2(ex);
        }
#pragma unroll 4
        for (int z = 0; z < D / 8; ++z) {
            uint4 r = piece(z);
            if (BF16) r = scaled_f16(r, f);
            const int y = z * 32 + lane, ch8 = y % (D / 8);
            *reinterpret_cast<uint4*>(dst + (ch8 >> 3) * Shape<D>::kAtom + swz(32 * wp + y / (D / 8), ch8 & 7)) = r;
        }
    }
}

// Warp wp turns part wp of every step into rows of the step's K tile, then of its V tile. Its 16
// bytes a lane and chunk are reloaded in place: V codes while K's are converted, the next step's K
// codes while V's are.
template <int D, bool INT8, bool BF16>
__device__ __forceinline__ void expand_role(const BlockPrefillParams& p, uint8_t* smem, uint64_t* bars, int32_t* err, int wp,
                                            int lane) {
    using Sh = Shape<D>;
    const BlockView& c = p.c;
    const int g = lane >> 2, t = lane & 3, sh = c.log2_block - 5;
    constexpr int kChunks = D / 16;  // 512-byte chunks of a part's K or V
    StepWalk ahead(p, blockIdx.x);
    // The part of a step: its sequence entry and KV head (head * 256 + entry, -1 behind the last
    // step), its 32-token tile, with bit 31 set where the tile is exact or not there. The pool slot
    // is loaded a step before its address is needed.
    int slot = 0;
    auto look = [&](int& who, uint32_t& tile) {
        who = -1;
        tile = 0x80000000u;
        if (!ahead.valid()) return;
        const BlockPrefillSeq& e = p.seqs[ahead.w.i];
        who = ahead.w.kvh * 256 + ahead.w.i;
        const int x = 4 * ahead.j + wp;
        tile = (uint32_t)x;
        if (x < e.n >> c.log2_block << sh) slot = __ldg(block_table(c, e.seq) + (x >> sh));
        else tile |= 0x80000000u;
        ahead.next();
    };
    auto address = [&](int who, uint32_t tile) -> const uint8_t* {
        return tile >> 31 ? nullptr : tile_ptr(c, slot, who >> 8, (int)tile & ((1 << sh) - 1));
    };
    auto load = [&](const uint8_t* rec, int i) { return __ldg(reinterpret_cast<const uint4*>(rec + 16 + i * 512) + lane); };
    uint4 x[kChunks];
    float4 hd = make_float4(1.f, 0.f, 0.f, 1.f);
    int who, who1;
    uint32_t tile, tile1;
    look(who, tile);
    const uint8_t* rec = address(who, tile);
    if (rec) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) x[i] = load(rec, i);
        hd = __ldg(reinterpret_cast<const float4*>(rec));
    }
    look(who1, tile1);
#pragma unroll 1
    for (int jj = 0; who >= 0; ++jj) {
        float* head = reinterpret_cast<float*>(smem + Sh::kHdr) + ((jj & 3) * 4 + wp) * 4;
        float2 h;
        uint32_t bad = 0;
        // K
        if (jj >= 2) mbar_wait(bars + kBarKEmpty + (jj & 1), (uint32_t)(((jj >> 1) - 1) & 1), err);
        uint8_t* dst = smem + Sh::kK + (jj & 1) * Sh::kTileQ;
        if (rec) {
            h = make_float2(hd.x, 0.f);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const uint4 a = make_uint4(codes_lo<INT8>(x[i].x), codes_hi<INT8>(x[i].x), codes_lo<INT8>(x[i].y),
                                           codes_hi<INT8>(x[i].y));
                const uint4 b = make_uint4(codes_lo<INT8>(x[i].z), codes_hi<INT8>(x[i].z), codes_lo<INT8>(x[i].w),
                                           codes_hi<INT8>(x[i].w));
                x[i] = load(rec, kChunks + i);
                // 16 channels of one token
                const int s = i / (D / 32), cc = i / 2 % (D / 64), hh = i & 1;
                const int row = 32 * wp + 8 * (g >> 1) + 4 * s + 2 * hh + (g & 1);
                *reinterpret_cast<uint4*>(dst + cc * Sh::kAtom + swz(row, 2 * t)) = a;
                *reinterpret_cast<uint4*>(dst + cc * Sh::kAtom + swz(row, 2 * t + 1)) = b;
            }
        } else {
            expand_exact<D, BF16, false>(c, p.seqs[who & 255], who >> 8, (int)(tile & 0x7fffffffu), wp, lane, dst, h, bad);
        }
        if (lane == 0) head[0] = h.x;
        fence_proxy_async_smem();
        mbar_arrive(bars + kBarKFull + (jj & 3));
        // V
        const uint8_t* rec1 = address(who1, tile1);
        int who2;
        uint32_t tile2;
        look(who2, tile2);
        if (jj >= 2) mbar_wait(bars + kBarVEmpty + (jj & 1), (uint32_t)(((jj >> 1) - 1) & 1), err);
        dst = smem + Sh::kV + (jj & 1) * Sh::kTileV;
        if (rec) {
            h = make_float2(hd.z, hd.w);
            uint8_t* atom = dst + (wp >> 1) * (D * 128);
            const int chunk = 4 * (wp & 1) + t;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const uint4 a = make_uint4(codes_lo<INT8>(x[i].x), codes_hi<INT8>(x[i].x), codes_lo<INT8>(x[i].y),
                                           codes_hi<INT8>(x[i].y));
                const uint4 b = make_uint4(codes_lo<INT8>(x[i].z), codes_hi<INT8>(x[i].z), codes_lo<INT8>(x[i].w),
                                           codes_hi<INT8>(x[i].w));
                if (rec1) x[i] = load(rec1, i);
                // 8 tokens of channels 16 i + g and + 8
                *reinterpret_cast<uint4*>(atom + swz(16 * i + g, chunk)) = a;
                *reinterpret_cast<uint4*>(atom + swz(16 * i + g + 8, chunk)) = b;
            }
        } else {
            expand_exact<D, BF16, true>(c, p.seqs[who & 255], who >> 8, (int)(tile & 0x7fffffffu), wp, lane, dst, h, bad);
            if (rec1) {
#pragma unroll
                for (int i = 0; i < kChunks; ++i) x[i] = load(rec1, i);
            }
        }
        if (rec1) hd = __ldg(reinterpret_cast<const float4*>(rec1));
        if (lane == 0) head[1] = __uint_as_float(bad), head[2] = h.x, head[3] = h.y;
        fence_proxy_async_smem();
        mbar_arrive(bars + kBarVFull + (jj & 3));
        who = who1;
        tile = tile1;
        rec = rec1;
        who1 = who2;
        tile1 = tile2;
    }
}

// ---- softmax: thread et owns row et of tile b ----
template <int D, bool BF16>
__device__ __forceinline__ void softmax_role(const BlockPrefillParams& p, uint8_t* smem, uint64_t* bars, uint32_t tmem,
                                             int32_t* err, int et, int b, uint32_t lane_off) {
    using Sh = Shape<D>;
    const uint32_t ts = tmem + kColS + 128 * b + lane_off, to = tmem + kColO + 128 * b + lane_off;
    const int tpt = 128 / p.r, tok_in = et / p.r, head_in = et % p.r;
    const float4* hdr = reinterpret_cast<const float4*>(smem + Sh::kHdr);
    // a negative scale turns the query's sign, so that larger S is always a larger logit
    // (and a scale of 0 the query to zeros: every logit is 0)
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    const bool zero = p.scale_log2 == 0.f;
    const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    int jj = 0, step = 0, seg = 0;
    for (Walk w(p, blockIdx.x); w.valid(); w.next()) {
        if (b == 1 && !w.two()) {
            jj += w.j1 - w.j0;
            continue;
        }
        const BlockPrefillSeq& e = p.seqs[w.i];
        const int tok = (2 * w.pair + b) * tpt + tok_in;
        const bool valid = tok_in < tpt && tok < e.q_len;
        const size_t row = ((size_t)(e.q_row + tok) * p.hq + w.kvh * p.r + head_in) * D;
        const int pos = valid ? e.n - e.q_len + tok : e.n - 1;
        float qs = scale;
        {
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (valid ? row : 0));
            float f = 1.f;
            if (BF16) {
                uint32_t top = 0;
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i)
                    if (valid) top = max_of(top, src[i]);
                const int ex = bf16_exponent(max(top & 0xffffu, top >> 16)) - 14;
                f = power2(-ex);
                qs *= power2(ex);
            }
            uint8_t* dst = smem + Sh::kQ + b * Sh::kTileQ;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                uint4 r = make_uint4(0, 0, 0, 0);
                if (valid && !zero) r = src[i];
                if (BF16) r = scaled_f16(r, f);
                r = make_uint4(r.x ^ sign, r.y ^ sign, r.z ^ sign, r.w ^ sign);
                *reinterpret_cast<uint4*>(dst + (i >> 3) * Sh::kAtom + swz(et, i & 7)) = r;
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(bars + kBarQFull + b);
        float m = kNegInf, l = 0.f;
        for (int j = w.j0; j < w.j1; ++j, ++jj, ++step) {
            // A tile that sat out a segment may be whole phases ahead of the expansion; once its first
            // step's QK is done both barriers are at that step's phase or the one before. Within a
            // segment they are waited for first, and the headers read, while QK runs.
            if (j == w.j0) mbar_wait(bars + kBarSFull + b, (uint32_t)(step & 1), err);
            mbar_wait(bars + kBarKFull + (jj & 3), (uint32_t)((jj >> 2) & 1), err);
            mbar_wait(bars + kBarVFull + (jj & 3), (uint32_t)((jj >> 2) & 1), err);
            // logit = S c[ch] (+ log2 of V's scale in the weight); c > 0 or NaN
            float c[4], lv[4], iv[4];
            uint32_t bad = 0;
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
                const float4 h = hdr[(jj & 3) * 4 + ch];
                c[ch] = qs * h.x;
                if (c[ch] < 1e-37f) c[ch] = 1e-37f;  // 0 would make -inf of a masked column NaN
                lv[ch] = h.z;
                iv[ch] = h.w;
                bad |= __float_as_uint(h.y);
            }
            mbar_spin(bars + kBarSFull + b, (uint32_t)(step & 1), err);
            tc_fence_after();
            const int lim = pos + 1 - j * kStep;  // visible columns
            uint32_t r[4][32];
            float mx = kNegInf;
            auto raise = [&](int ch) {
                float a = __uint_as_float(r[ch][0]), a2 = __uint_as_float(r[ch][1]);
#pragma unroll
                for (int k = 2; k < 30; k += 4) {
                    a = max3(a, __uint_as_float(r[ch][k]), __uint_as_float(r[ch][k + 1]));
                    a2 = max3(a2, __uint_as_float(r[ch][k + 2]), __uint_as_float(r[ch][k + 3]));
                }
                a = max3(a, __uint_as_float(r[ch][30]), __uint_as_float(r[ch][31]));
                mx = fmaxf(mx, fmaf(fmaxf(a, a2), c[ch], lv[ch]));
            };
            const bool plain = !bad && __all_sync(0xffffffffu, lim >= kStep);
            tm_ld32(ts, r[0]);
            tm_ld32(ts + 32, r[1]);
            tm_wait_ld();
            tm_ld32(ts + 64, r[2]);
            tm_ld32(ts + 96, r[3]);
            if (plain) {  // over the loads' latency
                raise(0);
                raise(1);
            }
            tm_wait_ld();
            if (plain) {
                raise(2);
                raise(3);
            } else {
                // non-finite V tokens' weights become NaN where they are seen; then columns behind the
                // row's position leave, with all of a part that is not seen at all
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    const uint32_t y = __float_as_uint(hdr[(jj & 3) * 4 + ch].y);
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (y >> k & 1) r[ch][k] = 0x7fc00000u;
                        if (32 * ch + k >= lim) r[ch][k] = 0xff800000u;
                    }
                    if (32 * ch >= lim) c[ch] = 1.f, lv[ch] = 0.f, iv[ch] = 1.f;
                    raise(ch);
                }
            }
            const bool up = mx > m + 8.f;  // also from -inf
            if (__any_sync(0xffffffffu, up)) {
                const float f = up ? ex2f(m - mx) : 1.f;  // 0 from -inf
                if (up) m = mx;
                l *= f;
                if (j > w.j0) {
                    // O is rescaled 16 columns at a time: the 128 logits stay in registers
#pragma unroll 1
                    for (int ch = 0; ch < D / 16; ++ch) {
                        uint32_t o[16];
                        tm_ld16(to + 16 * ch, o);
                        tm_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tm_st16(to + 16 * ch, o);
                    }
                }
            }
            const float mm = m == kNegInf ? 0.f : m;
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
                if (ch & 1) {  // 64 keys: their PV may start
                    tm_wait_st();
                    tc_fence_before();
                    mbar_arrive(bars + kBarPFull + 2 * b + (ch >> 1));
                }
            }
        }
        mbar_wait(bars + kBarOFull + b, (uint32_t)(seg++ & 1), err);
        tc_fence_after();
        if (w.whole()) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t r[32];
                tm_ld32(to + 32 * ch, r);
                tm_wait_ld();
                if (valid) {
                    uint4* dst = reinterpret_cast<uint4*>(p.out + row + 32 * ch);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            o[z] = pack2<BF16>(__uint_as_float(r[8 * k + 2 * z]) * inv, __uint_as_float(r[8 * k + 2 * z + 1]) * inv);
                        dst[k] = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
        } else {
            float* part = reinterpret_cast<float*>(p.c.base + p.c.lay.partials) +
                          (size_t)(2 * blockIdx.x + (w.j0 == 0 ? 1 : 0)) * (256 * (D + 2));
            const int rr = 128 * b + et;
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t r[32];
                tm_ld32(to + 32 * ch, r);
                tm_wait_ld();
                float4* dst = reinterpret_cast<float4*>(part + (size_t)rr * D + 32 * ch);
                if (valid) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dst[k] = make_float4(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]),
                                             __uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3]));
                }
            }
            part[256 * D + rr] = m;
            part[256 * D + 256 + rr] = l;
        }
        tc_fence_before();  // O has been read before this thread lets the next segment's PV start
    }
}

template <int D, bool INT8, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ BlockPrefillParams p) {
    using Sh = Shape<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
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
            mbar_init(bars + kBarPFull + 2 + k, 128);
            mbar_init(bars + kBarOFull + k, 1);
            mbar_init(bars + kBarQFull + k, 128);
        }
        mbar_init(bars + kBarDrain, 1);
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
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Sh::kTmem);
    const uint32_t lane_off = (uint32_t)(32 * (w & 3)) << 16;
    if (wg < 2) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        softmax_role<D, BF16>(p, smem, bars, tmem, err, t & 127, wg, lane_off);
    } else if (wg == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
        expand_role<D, INT8, BF16>(p, smem, bars, err, w & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (w == 12) {
            issue_role<D>(p, smem_addr(smem), bars, tmem, err);
            // every MMA has completed before tensor memory is released
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(bars + kBarDrain, 0u) && global_ns() - t0 < kWaitLimitNs) {
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 12) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// Adds the partials of the segment that begins in CTA b's range and ends behind it, in the order
// of the cuts. blockIdx.y: 32 of the pair's 256 rows; 4 channels a thread.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ BlockPrefillParams p) {
    const int b = blockIdx.x;
    const int u0 = (int)((int64_t)p.steps * b / p.grid), u1 = (int)((int64_t)p.steps * (b + 1) / p.grid);
    Walk w(p, b);
    int u = u0;
    while (u + (w.j1 - w.j0) < u1) u += w.j1 - w.j0, w.next();
    if (w.j0 > 0 || w.j1 == w.steps) return;  // no segment both begins here and goes on
    const int last = (int)(((int64_t)(u + w.steps) * p.grid - 1) / p.steps);
    const BlockPrefillSeq& e = p.seqs[w.i];
    const int tpt = 128 / p.r;
    const float* base = reinterpret_cast<const float*>(p.c.base + p.c.lay.partials);
    constexpr size_t kPart = 256 * (D + 2);
    for (int x = threadIdx.x; x < 32 * (D / 4); x += 256) {
        const int rr = blockIdx.y * 32 + x / (D / 4), ch = x % (D / 4) * 4, et = rr & 127;
        const int tok = (2 * w.pair + (rr >> 7)) * tpt + et / p.r;
        if (et / p.r >= tpt || tok >= e.q_len) continue;
        float big = kNegInf, l = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        auto part = [&](int z) { return base + (size_t)(2 * z + (z == b ? 1 : 0)) * kPart; };
        for (int z = b; z <= last; ++z) big = fmaxf(big, part(z)[256 * D + rr]);
        for (int z = b; z <= last; ++z) {
            const float* q = part(z);
            const float mz = q[256 * D + rr], f = mz == kNegInf ? 1.f : ex2f(mz - big);  // -inf: zeros or NaN
            const float4 o = *reinterpret_cast<const float4*>(q + (size_t)rr * D + ch);
            sum.x = fmaf(o.x, f, sum.x);
            sum.y = fmaf(o.y, f, sum.y);
            sum.z = fmaf(o.z, f, sum.z);
            sum.w = fmaf(o.w, f, sum.w);
            l = fmaf(q[256 * D + 256 + rr], f, l);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t row = ((size_t)(e.q_row + tok) * p.hq + w.kvh * p.r + et % p.r) * D;
        *reinterpret_cast<uint2*>(p.out + row + ch) =
            make_uint2(pack2<BF16>(sum.x * inv, sum.y * inv), pack2<BF16>(sum.z * inv, sum.w * inv));
    }
}

template <int D, bool INT8, bool BF16>
int launch(const BlockPrefillParams& p, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(prefill_kernel<D, INT8, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Shape<D>::kSmem);
    if (e != cudaSuccess) return (int)e;
    prefill_kernel<D, INT8, BF16><<<p.grid, kThreads, Shape<D>::kSmem, s>>>(p);
    if (p.line) combine_kernel<D, BF16><<<dim3(p.grid, 8), 256, 0, s>>>(p);
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
