// Block cache: a prefix that many sequences share, walked once for the queries of all of them.
//
// Rows (query, head of the KV head's r) of all sequences behind a prefix are stacked to tiles of 128, M of tcgen05.mma; every row
// sees all of the prefix. What prefill does for a pair of tiles this does for one, since few queries rarely fill two:
// steps of 128 tokens go in turn to two (S, O) pairs in tensor memory with a softmax warpgroup each, which keep their own running maximum,
// so that one's logits and products run while the other's weights are made (weights, scales and denominators as in prefill).
// With a single tile nothing but depth hides the memory: codes come by bulk copies into rings of eight expansion warps (four
// take K, four V, a warp 32 tokens), 66 KB in flight a SM. The line of all steps is cut evenly over the CTAs; each leaves its
// sums, unnormalised, and join_kernel adds them in order into fp32 rows with the log2 of their denominators, which the kernels that
// take the sequences' own tokens join with theirs (where blocks' weights are noted, also the denominators as maximum and sum). Every wait is bounded and sets the error word when it gives up.
//
// Measured, 32 sequences behind each of two prefixes of 32k, 40 / 10 heads, int8, bf16 (128 rows of a KV head, 43 GFLOP, 168 MB): 57 us and
// 8 for the join; two row tiles at a time, as prefill takes them, 83 and 11. Bound by the chain of a step: weights of one tile, its
// products, a free V tile, the expansion into it; 34 steps a CTA, and about 10 us at its two ends. 64 rows or fewer take as long.
#include "kvarn_block_ring.cuh"

namespace kvarn {
namespace {

// Warps: two softmax warpgroups, then the first of each four the issuer and the two that fill the rings, the others
// expansion warps.
// The issuer's scheduler has no expansion warp: an MMA takes its warp about 30 turns there.
constexpr int kSoftWarps = 8, kExpWarps = 8, kIssuer = kSoftWarps, kThreads = 32 * (kSoftWarps + kExpWarps + 3);
__device__ __forceinline__ int expansion_warp(int w) { return (w - kSoftWarps) / 4 * 3 + (w & 3) - 1; }  // 0 .. 7, of w & 3 > 0
static_assert(kSoftWarps % 4 == 0 && kExpWarps == 8, "warps by scheduler");
constexpr int kStep = 128, kRing = 8;
constexpr float kRaise = 8.f, kShift = 7.f;  // m is raised when it would grow by more; weights are at most 2^(both)
constexpr uint32_t kColS = 0, kColO = 256;
// barriers
constexpr int kKFull = 0, kVFull = kKFull + kRing, kVHead = kVFull + kRing, kQFull = kVHead + kRing, kKEmpty = kQFull + kRing, kVEmpty = kKEmpty + 2,
              kSFull = kVEmpty + 2, kPFull = kSFull + 2, kOFull = kPFull + 2, kOEmpty = kOFull + 2, kQEmpty = kOEmpty + 2,
              kDrain = kQEmpty + 1, kRaw = kDrain + 1, kNumBars = kRaw + 2 * kExpWarps + 4;

template <int D>
struct Shape {
    static constexpr int kTileK = D / 64 * kAtom, kTileV = 2 * D * 128;
    static constexpr int kQ = 0;
    static constexpr int kK = kTileK;                            // 2 stages
    static constexpr int kV = kK + 2 * kTileK;                   // 2 stages
    static constexpr int kRings = kV + 2 * kTileV;
    static constexpr int kHeadV = kRings + Rings<D>::kBytes;     // float4[kRing][4]: log2 of V's scale, kDenomUnit over it, non-finite
    static constexpr int kHeadK = kHeadV + kRing * 64;           // float[kRing][4]: K's scale
    static constexpr int kPower = kHeadK + kRing * 16;           // int8[kRing][128]
    static constexpr int kBars = kPower + kRing * 128;
    static constexpr int kWhat = kBars + 8 * kNumBars;           // int[8][2]
    static constexpr int kTmem = kWhat + 64;
    static constexpr int kSmem = kTmem + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

typedef RowWalk<BlockFlatParams> Walk;

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

// Step k of the CTA goes to tile k & 1. A step's QK is issued before the PV of the step before it, and writes S behind the PV
// that read the weights there, two steps before (MMAs complete in the order of their issue).
template <int D>
__device__ __forceinline__ void issue_role(const BlockFlatParams& p, uint32_t sbase, uint64_t* bars, int32_t* err) {
    using Sh = Shape<D>;
    const bool leader = elect_one();
    const uint32_t base = sbase >> 4;
    int k = 0, seg = 0;
    Walk w(p);
#pragma unroll 1
    for (; w.next(); ++seg) {
        const int n = __shfl_sync(0xffffffffu, w.j1 - w.j0, 0);
        bar_wait(bars + kQFull + seg % kRing, (uint32_t)(seg / kRing & 1), err);
        // turn i: QK of the segment's step i (but the last turn), PV of step i - 1 (but the first)
#pragma unroll 1
        for (int i = 0; i <= n; ++i) {
            if (i < n) {
                bar_wait(bars + kKFull + k % kRing, (uint32_t)(k / kRing & 1), err);
                __syncwarp();
                tc_fence_after();
                const int b = __shfl_sync(0xffffffffu, k & 1, 0);  // seen to be uniform
                const uint32_t q = base + (Sh::kQ >> 4), kt = base + ((Sh::kK + b * Sh::kTileK) >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = ((ks >> 2) * kAtom + (ks & 3) * 32) >> 4;
                    if (leader) mma_ss(kColS + 128 * b, desc128(q + off), desc128(kt + off), kIdesc<128>, ks > 0);
                }
                if (leader) mma_commit(bars + kSFull + (k & 1));
                if (leader) mma_commit(bars + kKEmpty + (k & 1));
                if (leader && i == n - 1) mma_commit(bars + kQEmpty);
                ++k;
            }
            if (i > 0) {
                const int at = i < n ? k - 2 : k - 1, b = __shfl_sync(0xffffffffu, at & 1, 0);
                if (seg > 0 && i <= 2) bar_wait(bars + kOEmpty + b, (uint32_t)((seg - 1) & 1), err);  // the last segment's sums are out
                bar_wait(bars + kVFull + at % kRing, (uint32_t)(at / kRing & 1), err);
                bar_wait(bars + kPFull + b, (uint32_t)(at >> 1 & 1), err);
                __syncwarp();
                tc_fence_after();
                const uint32_t more = __shfl_sync(0xffffffffu, i > 2 ? 1u : 0u, 0);
                const uint32_t v = base + ((Sh::kV + b * Sh::kTileV) >> 4);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    if (leader)
                        mma_ts(kColO + 128 * b, kColS + 128 * b + 8 * ks, desc128(v + (((ks >> 2) * (D * 128) + (ks & 3) * 32) >> 4)),
                               kIdesc<D>, ks > 0 ? 1u : more);
                if (leader) mma_commit(bars + kVEmpty + b);
            }
        }
        if (leader) mma_commit(bars + kOFull);
        if (leader) mma_commit(bars + kOFull + 1);
    }
    if (leader) mma_commit(bars + kDrain);
    // every MMA has completed before tensor memory is released
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!mbar_try_wait(bars + kDrain, 0u) && global_ns() - t0 < kWaitLimitNs) {
    }
}

// Floats of a part: O^T in pieces of four channels, [D / 4][128 rows][4], then m, l and the non-finite flag of each row.
template <int D>
constexpr int kPart = 128 * (D + 3);

// Warpgroup b has tile b; thread et owns row et.
template <int D, bool BF16>
__device__ __forceinline__ void softmax_role(const BlockFlatParams& p, uint8_t* smem, uint64_t* bars, int32_t* err, int et, int b,
                                             uint32_t lane_off) {
    using Sh = Shape<D>;
    const uint32_t ts = kColS + 128 * b + lane_off, to = kColO + 128 * b + lane_off;
    // The rows of the next segment are on their way while this one's sums are written.
    const Rows<D, kSoftWarps> rows(smem + Sh::kQ, 4 * b + (et >> 5), et & 31);
    auto ready = [&](int s) {
        rows.template finish<BF16>(p.scale_log2, reinterpret_cast<int8_t*>(smem + Sh::kPower) + s % kRing * 128);
        mbar_arrive(bars + kQFull + s % kRing);
    };
    int k = 0, seg = 0;
    Walk w(p);
    bool more = w.next();
    if (more) {
        rows.fetch(p, w);
        ready(0);
    }
#pragma unroll 1
    for (; more; ++seg) {
        const int n = p.seqs[w.i].n;
        const int begin = w.j0 + ((b ^ k) & 1);
        float m = kNegInf, l = 0.f, qs = 1.f;
        uint32_t bad = 0;
        k += w.j1 - w.j0;
#pragma unroll 1
        for (int j = begin, kk = k - (w.j1 - begin); j < w.j1; j += 2, kk += 2) {
            if (j == begin) {
                bar_wait(bars + kQFull + seg % kRing, (uint32_t)(seg / kRing & 1), err);
                qs = row_factor(p.scale_log2, reinterpret_cast<const int8_t*>(smem + Sh::kPower)[seg % kRing * 128 + et]);
            }
            bar_wait(bars + kKFull + kk % kRing, (uint32_t)(kk / kRing & 1), err);
            bar_wait(bars + kVHead + kk % kRing, (uint32_t)(kk / kRing & 1), err);
            const float* hk = reinterpret_cast<const float*>(smem + Sh::kHeadK) + kk % kRing * 4;
            const float4* hv = reinterpret_cast<const float4*>(smem + Sh::kHeadV) + kk % kRing * 4;
            bar_wait(bars + kSFull + b, (uint32_t)(kk >> 1 & 1), err);
            __syncwarp();
            tc_fence_after();
            const int lim = n - j * kStep;  // columns that are there
            float mx = kNegInf;
            // logit = S c (+ log2 of V's scale in the weight), c > 0 or NaN, constant in a part's columns. Loops over parts stay rolled: the
            // roles together would not fit the instruction cache (unrolled, with a third of all stalls, 111 us where rolled 77).
            auto part_of = [&](int ch, uint32_t (&r)[32], float& c, float& lv, float& iv) {
                tm_ld32(ts + 32 * ch, r);
                const float4 h = hv[ch];
                c = qs * hk[ch];
                if (c < 1e-37f) c = 1e-37f;  // 0 would make -inf of a masked column NaN
                lv = h.x;
                iv = h.y;
                bad |= __float_as_uint(h.z);
                tm_wait_ld();
                const int left = lim - 32 * ch;
                if (__builtin_expect(left < 32, 0)) {
#pragma unroll
                    for (int z = 0; z < 32; ++z)
                        if (z >= left) r[z] = 0xff800000u;
                    if (left <= 0) c = 1.f, lv = 0.f, iv = 1.f;
                }
            };
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
                uint32_t r[32];
                float c, lv, iv;
                part_of(ch, r, c, lv, iv);
                mx = fmaxf(mx, fmaf(max32(r), c, lv));
            }
            const bool up = mx > m + kRaise;  // also from -inf
            const bool rescale = __any_sync(0xffffffffu, up);
            const float f = up ? ex2f(m - mx) : 1.f;  // 0 from -inf
            if (up) m = mx;
            l *= f;
            const float mm = m == kNegInf ? 0.f : m - kShift;
            // again, for the weights: those of a part lie over logits that are through
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
                uint32_t r[32];
                float c, lv, iv;
                part_of(ch, r, c, lv, iv);
                const float ad = lv - mm;
                const float2 c2 = make_float2(c, c), a2 = make_float2(ad, ad);
                float2 s0 = make_float2(0.f, 0.f), s1 = s0;
                uint32_t o[16];
#pragma unroll
                for (int z = 0; z < 16; ++z) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[2 * z]), __uint_as_float(r[2 * z + 1])), c2, a2);
                    const float2 v = make_float2(ex2f(x.x), ex2f(x.y));
                    if (z & 1) s1 = __fadd2_rn(s1, v);
                    else s0 = __fadd2_rn(s0, v);
                    o[z] = h2u(__float22half2_rn(v));
                }
                s0 = __fadd2_rn(s0, s1);
                l = fmaf(s0.x + s0.y, iv, l);
                tm_st16(ts + 16 * ch, o);
            }
            if (rescale && j > begin) {  // O: the products of two steps before are through, since this step's logits are
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t o[32];
                    tm_ld32(to + 32 * ch, o);
                    tm_wait_ld();
#pragma unroll
                    for (int z = 0; z < 32; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * f);
                    tm_st32(to + 32 * ch, o);
                }
            }
            tm_wait_st();
            tc_fence_before();
            mbar_arrive(bars + kPFull + b);
        }
        // of the pair's part in this CTA (a pair's first CTA is no sooner than the pair before's last)
        float* part = p.parts + (size_t)((p.seqs[w.i].pair_begin + w.pair + blockIdx.x) * 2 + b) * kPart<D>;
        const bool some = begin < w.j1;
        more = w.next();
        if (more) {
            bar_wait(bars + kQEmpty, (uint32_t)(seg & 1), err);
            __syncwarp();
            rows.fetch(p, w);
        }
        bar_wait(bars + kOFull + b, (uint32_t)(seg & 1), err);
        __syncwarp();
        tc_fence_after();
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t o[32];
            tm_ld32(to + 32 * ch, o);
            tm_wait_ld();
#pragma unroll
            for (int z = 0; z < 8; ++z)
                reinterpret_cast<uint4*>(part)[(8 * ch + z) * 128 + et] =
                    some ? make_uint4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]) : make_uint4(0, 0, 0, 0);
        }
        part[128 * D + et] = m;
        part[128 * D + 128 + et] = l;
        part[128 * D + 256 + et] = __uint_as_float(bad);
        tc_fence_before();
        mbar_arrive(bars + kOEmpty + b);
        if (more) ready(seg + 1);
    }
}

template <int D, bool INT8, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) flat_kernel(const __grid_constant__ BlockFlatParams p) {
    using Sh = Shape<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    int32_t* err = reinterpret_cast<int32_t*>(p.c.base + p.c.lay.err);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kBars);
    start_next();
    if (t == 0) {
        for (int k = 0; k < kRing; ++k) {
            mbar_init(bars + kKFull + k, 128);
            mbar_init(bars + kVFull + k, 128);
            mbar_init(bars + kVHead + k, 4);
            mbar_init(bars + kQFull + k, 32 * kSoftWarps);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(bars + kKEmpty + k, 1);
            mbar_init(bars + kVEmpty + k, 1);
            mbar_init(bars + kSFull + k, 1);
            mbar_init(bars + kPFull + k, 128);
            mbar_init(bars + kOFull + k, 1);
            mbar_init(bars + kOEmpty + k, 128);
        }
        mbar_init(bars + kQEmpty, 1);
        mbar_init(bars + kDrain, 1);
        for (int k = 0; k < 2 * kExpWarps; ++k) mbar_init(bars + kRaw + k, 1);
        for (int k = 0; k < 4; ++k) mbar_init(bars + kRaw + 2 * kExpWarps + k, 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (w == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(smem + Sh::kTmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // All of tensor memory is this CTA's, so it starts at address 0, and shared memory on 1024 bytes; both are counted on.
    // Were it ever not so, the launch would do nothing but say so.
    const bool placed = *reinterpret_cast<volatile uint32_t*>(smem + Sh::kTmem) == 0 && (smem_addr(smem) & 1023) == 0;
    if (!placed && t == 0) atomicOr(err, kErrBadSlot);
    const Rings<D> rings = {smem + Sh::kRings, bars + kRaw, bars + kRaw + 2 * kExpWarps, reinterpret_cast<int32_t*>(smem + Sh::kWhat)};
    const int steps = (int)(p.units * (blockIdx.x + 1) / p.grid - p.units * blockIdx.x / p.grid);
    if (!placed) {
    } else if (w < kSoftWarps) {
        softmax_role<D, BF16>(p, smem, bars, err, t & 127, w >> 2, (uint32_t)(32 * (w & 3)) << 16);
    } else if (w & 3) {
        const int x = expansion_warp(w), wp = x & 3;
        if (x < 4)
            expand_steps<D, INT8, BF16, false, 1>(
                rings, x, 0, steps, err, lane,
                [&](int k, float2 h, uint32_t) {
                    if (lane == 0) reinterpret_cast<float*>(smem + Sh::kHeadK)[k % kRing * 4 + wp] = h.x;
                },
                [&](int k) {
                    if (k >= 2) bar_wait(bars + kKEmpty + (k & 1), (uint32_t)(((k >> 1) - 1) & 1), err);
                    return smem + Sh::kK + (k & 1) * Sh::kTileK;
                },
                [&](int k) { mbar_arrive(bars + kKFull + k % kRing); });
        else
            expand_steps<D, INT8, BF16, true, 1>(
                rings, x, 0, steps, err, lane,
                [&](int k, float2 h, uint32_t bad) {  // the weights need no more of V: they are made while its tile waits for a place
                    if (lane == 0) {
                        reinterpret_cast<float4*>(smem + Sh::kHeadV)[k % kRing * 4 + wp] = make_float4(h.x, h.y, __uint_as_float(bad), 0.f);
                        mbar_arrive(bars + kVHead + k % kRing);
                    }
                },
                [&](int k) {
                    if (k >= 2) bar_wait(bars + kVEmpty + (k & 1), (uint32_t)(((k >> 1) - 1) & 1), err);
                    return smem + Sh::kV + (k & 1) * Sh::kTileV;
                },
                [&](int k) { mbar_arrive(bars + kVFull + k % kRing); });
    } else if (w == kIssuer) {
        issue_role<D>(p, smem_addr(smem), bars, err);
    } else {
        fill_rings<D, true>(p, rings, (w - kIssuer) / 4 - 1, steps, err, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == kIssuer) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*reinterpret_cast<volatile uint32_t*>(smem + Sh::kTmem))
                     : "memory");
    }
}

// The parts of a pair (blockIdx.x) for 32 rows of it (blockIdx.y) and 32 channels (blockIdx.z), in the order of the cuts: a lane a row,
// the warps in turns of parts for the maxima and sums, then four channels each.
constexpr int kJoinWarps = 8, kMostParts = 2 * kBlockPrefillGrid;
template <int D, bool BF16>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ BlockFlatParams p) {
    __shared__ float factor[kMostParts][32];
    __shared__ float red[kJoinWarps][32];
    __shared__ uint32_t flags[kJoinWarps];
    before_done();
    start_next();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y * 32 + lane;
    int i = 0;
#pragma unroll 1
    while (i + 1 < p.n_seqs && p.seqs[i + 1].pair_begin <= (int)blockIdx.x) ++i;
    const auto& e = p.seqs[i];
    const int pair = blockIdx.x - e.pair_begin, h = pair / e.row_tiles, tile = pair - h * e.row_tiles;
    if (tile * 128 + (int)blockIdx.y * 32 >= e.rows) return;
    const int64_t u = e.unit_begin + (int64_t)pair * e.steps;
    const int b0 = (int)(((u + 1) * p.grid - 1) / p.units), b1 = (int)(((u + e.steps) * p.grid - 1) / p.units);
    const int parts = 2 * (b1 - b0 + 1);
    const float* at = p.parts + (size_t)(blockIdx.x + b0) * 2 * kPart<D>;
    float m = kNegInf;
    uint32_t bad = 0;
#pragma unroll 4
    for (int z = w; z < parts; z += kJoinWarps) {
        const float* x = at + (size_t)z * kPart<D> + 128 * D + row;
        factor[z][lane] = x[0];
        m = fmaxf(m, x[0]);
        bad |= __float_as_uint(x[256]);
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    red[w][lane] = m;
    if (lane == 0) flags[w] = bad;
    __syncthreads();
#pragma unroll
    for (int z = 0; z < kJoinWarps; ++z) m = fmaxf(m, red[z][lane]), bad |= flags[z];
    __syncthreads();
    float l = 0.f;
#pragma unroll 4
    for (int z = w; z < parts; z += kJoinWarps) {
        const float x = factor[z][lane], f = x == kNegInf ? 1.f : ex2f(x - m);  // -inf: zeros or NaN
        factor[z][lane] = f;
        l = fmaf(at[(size_t)z * kPart<D> + 128 * D + 128 + row], f, l);
    }
    red[w][lane] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int z = 0; z < kJoinWarps; ++z) l += red[z][lane];
    const int all = tile * 128 + row;
    if (all >= e.rows) return;
    const size_t out = (size_t)(e.q_row + all / p.r) * p.hq + h * p.r + all % p.r;
    if (w == 0 && blockIdx.z == 0) {
        p.pre_lse[out] = lse_of(m, l, kShift);
        if (p.totals) p.totals[out] = total_of(m, l, kShift);
    }
    const float inv = kDenomUnit * (l == 0.f ? 0.f : 1.f / l);
    {
        static_assert(kJoinWarps * 4 == 32, "channels of a CTA");
        const int c = blockIdx.z * kJoinWarps + w;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int z = 0; z < parts; ++z) {
            const float4 x = reinterpret_cast<const float4*>(at + (size_t)z * kPart<D>)[c * 128 + row];
            const float f = factor[z][lane];
            o = make_float4(fmaf(x.x, f, o.x), fmaf(x.y, f, o.y), fmaf(x.z, f, o.z), fmaf(x.w, f, o.w));
        }
        float y[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
        if (__builtin_expect(bad, 0)) {  // non-finite V of exact tokens went into the products as 0: each into its own channel
            const int sealed = e.n & ~(p.c.block - 1);
            const uint16_t* v = tail_ptr(p.c, p.c.lay.tail_v, e.seq, h);
#pragma unroll 1
            for (int z = 0; z < 4; ++z)
#pragma unroll 1
                for (int t = 0; t < e.n - sealed; ++t) {
                    const uint32_t x = v[tail_v_off(D, t, 4 * c + z)];
                    if (bad_pair<BF16>(x)) y[z] += unpack2<BF16>(x).x;
                }
        }
        *reinterpret_cast<float4*>(p.pre_o + out * D + 4 * c) = make_float4(y[0], y[1], y[2], y[3]);
    }
}

template <int D, bool INT8, bool BF16>
int launch(const BlockFlatParams& p, int pairs, cudaStream_t s) {
    static SmemOnce once;
    const int e = once.allow(reinterpret_cast<const void*>(flat_kernel<D, INT8, BF16>), Shape<D>::kSmem);
    if (e) return e;
    // (not behind the kernel before: 117 us for the call where it takes 110)
    flat_kernel<D, INT8, BF16><<<p.grid, kThreads, Shape<D>::kSmem, s>>>(p);
    const int rc = (int)cudaGetLastError();
    return rc ? rc : launch_behind(join_kernel<D, BF16>, dim3(pairs, 4, D / 32), 32 * kJoinWarps, 0, s, p);
}

}  // namespace

int launch_block_flat(const BlockFlatParams& p, int pairs, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    switch ((p.c.d == 128 ? 4 : 0) + (p.c.int8 ? 2 : 0) + (p.c.bf16 ? 1 : 0)) {
        case 0: return launch<64, false, false>(p, pairs, s);
        case 1: return launch<64, false, true>(p, pairs, s);
        case 2: return launch<64, true, false>(p, pairs, s);
        case 3: return launch<64, true, true>(p, pairs, s);
        case 4: return launch<128, false, false>(p, pairs, s);
        case 5: return launch<128, false, true>(p, pairs, s);
        case 6: return launch<128, true, false>(p, pairs, s);
        default: return launch<128, true, true>(p, pairs, s);
    }
}

}  // namespace kvarn
