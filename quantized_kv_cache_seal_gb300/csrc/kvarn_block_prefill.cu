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
// Roles (640 threads): two softmax warpgroups, one a tile, a thread a row; a K and a V
// warpgroup that turn codes into f16 tiles (K-major, 128-byte swizzle; warp w takes part w,
// loads a step ahead, two stages); one thread that issues every MMA: PV and the next QK of
// one tile run while the other tile's softmax does. Both tiles share each expanded K and V
// tile, which halves the expansion a product costs. Bound by the tensor cores and, close
// behind, by the softmax's issue slots.
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

constexpr int kThreads = 640;
constexpr int kRegsLaunch = 96, kRegsSoftmax = 136, kRegsExpand = 88, kRegsIssue = 32;
static_assert(2 * kRegsSoftmax + 2 * kRegsExpand + kRegsIssue <= 5 * kRegsLaunch, "register split");
constexpr uint32_t kColS = 0, kColO = 256;
constexpr int kStep = 128;  // keys of a step
#define kNegInf (-__int_as_float(0x7f800000))

constexpr int kBarKFull = 0, kBarVFull = 4, kBarKEmpty = 8, kBarVEmpty = 10, kBarSFull = 12, kBarPFull = 14, kBarOFull = 16,
              kBarQFull = 18, kBarDrain = 20, kNumBars = 21;

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

// ---- the MMA issuer (one thread) ----
template <int D>
__device__ __forceinline__ void issue_role(const BlockPrefillParams& p, uint32_t sbase, uint64_t* bars, uint32_t tmem,
                                           int32_t* err) {
    using Sh = Shape<D>;
    sbase >>= 4;  // (addresses stay under 2^18: descriptor fields)
    auto qk = [&](int b, int jj) {
        const uint32_t q = sbase + ((Sh::kQ + b * Sh::kTileQ) >> 4), k = sbase + ((Sh::kK + (jj & 1) * Sh::kTileQ) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * Sh::kAtom + (ks & 3) * 32) >> 4;
            mma_ss(tmem + kColS + 128 * b, desc128(q + off), desc128(k + off), kIdesc<128>, ks > 0);
        }
        mma_commit(bars + kBarSFull + b);
    };
    auto pv = [&](int b, int jj, bool first) {
        const uint32_t v = sbase + ((Sh::kV + (jj & 1) * Sh::kTileV) >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
            mma_ts(tmem + kColO + 128 * b, tmem + kColS + 128 * b + 8 * ks,
                   desc128(v + (((ks >> 2) * (D * 128) + (ks & 3) * 32) >> 4)), kIdesc<D>, (ks > 0 || !first) ? 1u : 0u);
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
        mma_commit(bars + kBarKEmpty + (jj & 1));
#pragma unroll 1
        for (int j = w.j0; j < w.j1; ++j, ++jj) {
            mbar_wait(bars + kBarVFull + (jj & 3), (uint32_t)((jj >> 2) & 1), err);
            const bool more = j + 1 < w.j1;
#pragma unroll 1
            for (int b = 0; b < tiles; ++b) {
                mbar_wait(bars + kBarPFull + b, steps >> b & 1, err);
                steps ^= 1u << b;
                tc_fence_after();
                pv(b, jj, j == w.j0);
                if (b == tiles - 1) mma_commit(bars + kBarVEmpty + (jj & 1));
                if (more) {
                    if (b == 0) {
                        mbar_wait(bars + kBarKFull + ((jj + 1) & 3), (uint32_t)(((jj + 1) >> 2) & 1), err);
                        tc_fence_after();
                    }
                    qk(b, jj + 1);
                    if (b == tiles - 1) mma_commit(bars + kBarKEmpty + ((jj + 1) & 1));
                } else {
                    mma_commit(bars + kBarOFull + b);
                }
            }
        }
    }
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

struct Part {
    const uint8_t* rec;  // its record, or null: exact tokens or none
    int i, kvh, tile;    // sequence entry, KV head, 32-token tile
};

template <int D, bool INT8, bool BF16, bool IS_V>
__device__ __forceinline__ void expand_role(const BlockPrefillParams& p, uint8_t* smem, uint64_t* bars, int32_t* err, int wp,
                                            int lane) {
    using Sh = Shape<D>;
    const BlockView& c = p.c;
    const int g = lane >> 2, t = lane & 3, sh = c.log2_block - 5;
    constexpr int kChunks = D / 16;  // 512-byte chunks of a part
    constexpr int kFull = IS_V ? kBarVFull : kBarKFull, kEmpty = IS_V ? kBarVEmpty : kBarKEmpty;
    constexpr int kRecOff = 16 + (IS_V ? kTileTokens * D : 0);
    StepWalk ahead(p, blockIdx.x);
    int slot = 0;
    // the part of the step at `ahead`, its slot on the way
    auto look = [&](Part& x) {
        x.i = -1;
        x.rec = nullptr;
        if (!ahead.valid()) return;
        const BlockPrefillSeq& e = p.seqs[ahead.w.i];
        x.i = ahead.w.i;
        x.kvh = ahead.w.kvh;
        x.tile = 4 * ahead.j + wp;
        if (x.tile < e.n >> c.log2_block << sh) {
            slot = __ldg(block_table(c, e.seq) + (x.tile >> sh));
            x.rec = c.base;  // the address follows when the slot is here
        }
        ahead.next();
    };
    auto address = [&](Part& x) {
        if (x.rec) x.rec = tile_ptr(c, slot, x.kvh, x.tile & ((1 << sh) - 1));
    };
    uint4 x[kChunks];
    float2 hd = make_float2(1.f, 1.f);  // K scale, or log2 and reciprocal of the V scale
    auto scales = [&](const Part& s) {
        return IS_V ? __ldg(reinterpret_cast<const float2*>(s.rec + 8)) : make_float2(__ldg(reinterpret_cast<const float*>(s.rec)), 0.f);
    };
    auto load = [&](const Part& s, int i) { return __ldg(reinterpret_cast<const uint4*>(s.rec + kRecOff + i * 512) + lane); };
    Part cur, nxt;
    look(cur);
    address(cur);
    if (cur.rec) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) x[i] = load(cur, i);
        hd = scales(cur);
    }
    look(nxt);
    for (int jj = 0; cur.i >= 0; ++jj) {
        address(nxt);
        Part nn;
        look(nn);
        if (jj >= 2) mbar_wait(bars + kEmpty + (jj & 1), (uint32_t)(((jj >> 1) - 1) & 1), err);
        uint8_t* dst = smem + (IS_V ? Sh::kV + (jj & 1) * Sh::kTileV : Sh::kK + (jj & 1) * Sh::kTileQ);
        float2 h = hd;
        if (cur.rec) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const uint4 a = make_uint4(codes_lo<INT8>(x[i].x), codes_hi<INT8>(x[i].x), codes_lo<INT8>(x[i].y),
                                           codes_hi<INT8>(x[i].y));
                const uint4 b = make_uint4(codes_lo<INT8>(x[i].z), codes_hi<INT8>(x[i].z), codes_lo<INT8>(x[i].w),
                                           codes_hi<INT8>(x[i].w));
                if (nxt.rec) x[i] = load(nxt, i);
                if (IS_V) {  // 8 tokens of channels 16 i + g and + 8
                    uint8_t* atom = dst + (wp >> 1) * (D * 128);
                    const int chunk = 4 * (wp & 1) + t;
                    *reinterpret_cast<uint4*>(atom + swz(16 * i + g, chunk)) = a;
                    *reinterpret_cast<uint4*>(atom + swz(16 * i + g + 8, chunk)) = b;
                } else {  // 16 channels of one token
                    const int s = i / (D / 32), cc = i / 2 % (D / 64), hh = i & 1;
                    const int row = 32 * wp + 8 * (g >> 1) + 4 * s + 2 * hh + (g & 1);
                    *reinterpret_cast<uint4*>(dst + cc * Sh::kAtom + swz(row, 2 * t)) = a;
                    *reinterpret_cast<uint4*>(dst + cc * Sh::kAtom + swz(row, 2 * t + 1)) = b;
                }
            }
            if (nxt.rec) hd = scales(nxt);
        } else {
            const BlockPrefillSeq& e = p.seqs[cur.i];
            const int first = (cur.tile - (e.n >> c.log2_block << sh)) * kTileTokens;  // row of the tail
            const int nv = min(kTileTokens, e.n - cur.tile * kTileTokens);             // valid tokens, none if <= 0
            h = IS_V ? make_float2(0.f, 1.f) : make_float2(1.f, 0.f);
            if (IS_V) {
                const uint16_t* v = tail_ptr(c, c.lay.tail_v, e.seq, cur.kvh) + first;
                uint32_t keep[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    keep[z] = (8 * t + 2 * z < nv ? 0xffffu : 0u) | (8 * t + 2 * z + 1 < nv ? 0xffff0000u : 0u);
                auto row = [&](int ch) {
                    if (nv <= 0) return make_uint4(0, 0, 0, 0);
                    const uint4 r = *reinterpret_cast<const uint4*>(v + (size_t)ch * c.block + 8 * t);
                    return make_uint4(r.x & keep[0], r.y & keep[1], r.z & keep[2], r.w & keep[3]);
                };
                float f = 1.f;
                if (BF16) {
                    uint32_t top = 0;
                    for (int i = 0; i < 2 * kChunks; ++i) top = max_of(top, row(8 * i + g));
                    const int ex = warp_exponent(top);
                    f = power2(-ex);
                    h = make_float2((float)ex, f);
                }
                uint8_t* atom = dst + (wp >> 1) * (D * 128);
                for (int i = 0; i < 2 * kChunks; ++i) {
                    uint4 r = row(8 * i + g);
                    if (BF16) r = scaled_f16(r, f);
                    *reinterpret_cast<uint4*>(atom + swz(8 * i + g, 4 * (wp & 1) + t)) = r;
                }
            } else {
                const uint16_t* k = tail_ptr(c, c.lay.tail_k, e.seq, cur.kvh) + (size_t)first * D;
                auto piece = [&](int z) {  // 16 bytes z * 32 + lane of the part's 32 D values
                    const int at = z * 32 + lane, tok = at / (D / 8);
                    if (tok >= nv) return make_uint4(0, 0, 0, 0);
                    return *reinterpret_cast<const uint4*>(k + (size_t)tok * D + at % (D / 8) * 8);
                };
                float f = 1.f;
                if (BF16) {
                    uint32_t top = 0;
                    for (int z = 0; z < D / 8; ++z) top = max_of(top, piece(z));
                    const int ex = warp_exponent(top);
                    f = power2(-ex);
                    h.x = power2(ex);
                }
                for (int z = 0; z < D / 8; ++z) {
                    uint4 r = piece(z);
                    if (BF16) r = scaled_f16(r, f);
                    const int at = z * 32 + lane, ch8 = at % (D / 8);
                    *reinterpret_cast<uint4*>(dst + (ch8 >> 3) * Sh::kAtom + swz(32 * wp + at / (D / 8), ch8 & 7)) = r;
                }
            }
            if (nxt.rec) {
#pragma unroll
                for (int i = 0; i < kChunks; ++i) x[i] = load(nxt, i);
                hd = scales(nxt);
            }
        }
        if (lane == 0) {
            float* at = reinterpret_cast<float*>(smem + Sh::kHdr) + ((jj & 3) * 4 + wp) * 4;
            if (IS_V) at[2] = h.x, at[3] = h.y;
            else at[0] = h.x;
        }
        fence_proxy_async_smem();
        mbar_arrive(bars + kFull + (jj & 3));
        cur = nxt;
        nxt = nn;
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
    const float scale = fabsf(p.scale_log2);
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
                if (valid) r = src[i];
                if (BF16) r = scaled_f16(r, f);
                r = make_uint4(r.x ^ sign, r.y ^ sign, r.z ^ sign, r.w ^ sign);
                *reinterpret_cast<uint4*>(dst + (i >> 3) * Sh::kAtom + swz(et, i & 7)) = r;
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(bars + kBarQFull + b);
        float m = kNegInf, l = 0.f;
        for (int j = w.j0; j < w.j1; ++j, ++jj, ++step) {
            // S first: a tile that sat out a segment may be whole phases ahead of the expansion,
            // and once this step's QK is done both barriers are at this step's phase or the one before
            mbar_wait(bars + kBarSFull + b, (uint32_t)(step & 1), err);
            mbar_wait(bars + kBarKFull + (jj & 3), (uint32_t)((jj >> 2) & 1), err);
            mbar_wait(bars + kBarVFull + (jj & 3), (uint32_t)((jj >> 2) & 1), err);
            tc_fence_after();
            const int lim = pos + 1 - j * kStep;  // visible columns
            const bool all = __all_sync(0xffffffffu, lim >= kStep);
            float mx = kNegInf;
#pragma unroll
            for (int ch = 0; ch < 4; ch += 2) {
                uint32_t r[2][32];
                tm_ld32(ts + 32 * ch, r[0]);
                tm_ld32(ts + 32 * ch + 32, r[1]);
                tm_wait_ld();
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float4 h = hdr[(jj & 3) * 4 + ch + z];
                    float a = kNegInf, a2 = kNegInf;
                    if (all) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            a = max3(a, __uint_as_float(r[z][k]), __uint_as_float(r[z][k + 1]));
                            a2 = max3(a2, __uint_as_float(r[z][k + 2]), __uint_as_float(r[z][k + 3]));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * (ch + z) + k < lim) a = fmaxf(a, __uint_as_float(r[z][k]));
                    }
                    a = fmaxf(a, a2);
                    if (a > kNegInf) mx = fmaxf(mx, fmaf(a, qs * h.x, h.z));
                }
            }
            const bool up = mx > m + 8.f;  // also from -inf
            if (__any_sync(0xffffffffu, up)) {
                const float f = up ? ex2f(m - mx) : 1.f;  // 0 from -inf
                if (up) m = mx;
                l *= f;
                if (j > w.j0) {
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t r[32];
                        tm_ld32(to + 32 * ch, r);
                        tm_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * f);
                        tm_st32(to + 32 * ch, r);
                    }
                }
            }
            const float mm = m == kNegInf ? 0.f : m;
#pragma unroll
            for (int ch = 0; ch < 4; ch += 2) {
                uint32_t r[2][32];
                tm_ld32(ts + 32 * ch, r[0]);
                tm_ld32(ts + 32 * ch + 32, r[1]);
                tm_wait_ld();
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float4 h = hdr[(jj & 3) * 4 + ch + z];
                    const float cc = qs * h.x, ad = h.z - mm;
                    const float2 c2 = make_float2(cc, cc), a2 = make_float2(ad, ad);
                    float2 sum = make_float2(0.f, 0.f);
                    uint32_t o[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 x =
                            __ffma2_rn(make_float2(__uint_as_float(r[z][2 * k]), __uint_as_float(r[z][2 * k + 1])), c2, a2);
                        float2 y = make_float2(ex2f(x.x), ex2f(x.y));
                        if (!all) {
                            if (32 * (ch + z) + 2 * k >= lim) y.x = 0.f;
                            if (32 * (ch + z) + 2 * k + 1 >= lim) y.y = 0.f;
                        }
                        sum = __fadd2_rn(sum, y);
                        o[k] = h2u(__float22half2_rn(y));
                    }
                    l = fmaf(sum.x + sum.y, h.w, l);
                    tm_st16(ts + 16 * (ch + z), o);
                }
            }
            tm_wait_st();
            tc_fence_before();
            mbar_arrive(bars + kBarPFull + b);
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
            mbar_init(bars + kBarOFull + k, 1);
            mbar_init(bars + kBarQFull + k, 128);
        }
        mbar_init(bars + kBarDrain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (w == 16) {
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
        expand_role<D, INT8, BF16, false>(p, smem, bars, err, w & 3, lane);
    } else if (wg == 3) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
        expand_role<D, INT8, BF16, true>(p, smem, bars, err, w & 3, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (w == 16 && lane == 0) {
            issue_role<D>(p, smem_addr(smem), bars, tmem, err);
            // every MMA has completed before tensor memory is released
            mma_commit(bars + kBarDrain);
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(bars + kBarDrain, 0u) && global_ns() - t0 < kWaitLimitNs) {
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == 16) {
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
