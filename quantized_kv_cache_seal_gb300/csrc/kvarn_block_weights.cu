// Block cache: what each block of a sequence receives of the softmax weights, added up over queries.
//
//   weights[seq][h][b] += sum over the rows (query token, head of KV head h) and the tokens n of block b of p_n,
//   p_n = 2^(x_n) / sum 2^(x_n'), x_n = scale log2(e) (q . k_n), over the tokens that the row sees.
// A row's denominator is known only behind its last key, so it goes in two steps: whoever makes the logits (decode
// attention, or window_kernel for the last queries of a prompt, which reads K alone) leaves of every 32-token tile and row
// a maximum m and the tile's sum s of 2^(x - m), 8 bytes for 32 logits, and of every row its total; weigh_kernel
// adds the tiles' shares to their blocks in a fixed order. Kept as a pair, no rounding of a logit's size
// stands between a weight and its denominator (log2 of the sum in one word would be off by 2^-17 at 128). A prefix that is walked once
// leaves its part of a row's total as such a pair too.
//
// Measured: beside decode (16 sequences of 32k, 32 / 8 heads) the pairs cost nothing that shows, 178 us as without, and weigh_kernel
// 6.4 us. 32 queries of 16 ragged prompts of 1k to 16k, 40 / 10 heads, bf16 (178 MB of codes, 45 MB of pairs written and read): window_kernel 60 us,
// weigh_kernel 14; the former bound by issue slots (61 % busy; a third of them the weights), the latter by its loads' latency.
#include "kvarn_block_ring.cuh"

namespace kvarn {
namespace {

// ---- logits of the last queries ----
// S = Q code^T on tcgen05 (M = 128 rows, N = 128 tokens, f16 operands, exact codes, fp32 sums) as in prefill, and no more: a
// unit of work is a step of 128 tokens for a tile of 128 rows of a (sequence, KV head), and the line of all units is cut evenly over
// the CTAs, one a SM. Roles (736 threads): eight expansion warps that turn K codes into f16 tiles (a warp 32 tokens,
// four warps every other step); one that issues the MMAs into four S buffers (all 512 columns of tensor
// memory: no O is kept); two that fill the code rings; three softmax warpgroups, every third step each, a thread a row. Every wait
// is bounded and sets the error word when it gives up.
constexpr int kWinThreads = 736, kWinStep = 128, kWinStages = 3, kWinRing = 8;
// A step's scales are written before its tile has a place, when the QK of five steps before has been issued and so the softmax of nine
// before is through: eight places would not do.
constexpr int kWinScales = 16;
// warps; behind the softmax ones in turn of four the issuer and the two that fill the rings, and three expansion warps, so that the issuer's
// scheduler has none of those
constexpr int kWinSoftmax = 4 * kWindowParts, kWinExpand = 8, kWinIssuer = kWinSoftmax;
static_assert(kWinThreads == 32 * (kWinSoftmax + kWinExpand + 3), "warps");
// barriers
constexpr int kKFull = 0, kKEmpty = kKFull + kWinRing, kSFull = kKEmpty + kWinStages, kSEmpty = kSFull + 4, kQFull = kSEmpty + 4,
              kQEmpty = kQFull + kWinRing, kDrain = kQEmpty + 2, kRaw = kDrain + 1, kWinBars = kRaw + kWinExpand * 2 + 4;

template <int D>
struct WinShape {
    static constexpr int kTile = D / 64 * kAtom;
    static constexpr int kQ = 0;                                   // 2 tiles
    static constexpr int kK = 2 * kTile;                           // kWinStages tiles
    static constexpr int kRings = kK + kWinStages * kTile;
    static constexpr int kScale = kRings + Rings<D>::kBytes;       // float[kWinScales][4]: K scale of a step's parts
    static constexpr int kPower = kScale + kWinScales * 16;         // int8[kWinRing][128]: of a segment's rows
    static constexpr int kBars = kPower + kWinRing * 128;
    static constexpr int kWhat = kBars + 8 * kWinBars;             // int[8][2]
    static constexpr int kTmem = kWhat + 64;
    static constexpr int kSmem = kTmem + 16;
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

typedef RowWalk<BlockWindowParams> WinWalk;

template <int D>
__device__ __forceinline__ void win_issue(const BlockWindowParams& p, uint32_t sbase, uint64_t* bars, int32_t* err) {
    using Sh = WinShape<D>;
    const bool leader = elect_one();
    const uint32_t base = sbase >> 4;
    int k = 0, seg = 0;
    WinWalk w(p);
#pragma unroll 1
    for (; w.next(); ++seg) {
        const int j1 = __shfl_sync(0xffffffffu, w.j1, 0), j0 = __shfl_sync(0xffffffffu, w.j0, 0);
        bar_wait(bars + kQFull + seg % kWinRing, (uint32_t)(seg / kWinRing & 1), err);
        const uint32_t q = base + ((Sh::kQ + __shfl_sync(0xffffffffu, seg & 1, 0) * Sh::kTile) >> 4);
#pragma unroll 1
        for (int j = j0; j < j1; ++j, ++k) {
            bar_wait(bars + kKFull + k % kWinRing, (uint32_t)(k / kWinRing & 1), err);
            if (k >= 4) bar_wait(bars + kSEmpty + (k & 3), (uint32_t)(((k >> 2) - 1) & 1), err);
            __syncwarp();
            tc_fence_after();
            const int stage = __shfl_sync(0xffffffffu, k % kWinStages, 0), buf = __shfl_sync(0xffffffffu, k & 3, 0);  // seen to be uniform
            const uint32_t kt = base + ((Sh::kK + stage * Sh::kTile) >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = ((ks >> 2) * kAtom + (ks & 3) * 32) >> 4;
                if (leader) mma_ss(128 * buf, desc128(q + off), desc128(kt + off), kIdesc<128>, ks > 0);
            }
            if (leader) mma_commit(bars + kSFull + (k & 3));
            if (leader) mma_commit(bars + kKEmpty + k % kWinStages);
            if (leader && j == j1 - 1) mma_commit(bars + kQEmpty + (seg & 1));
        }
    }
    if (leader) mma_commit(bars + kDrain);
    // every MMA has completed before tensor memory is released
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!mbar_try_wait(bars + kDrain, 0u) && global_ns() - t0 < kWaitLimitNs) {
    }
}

// Warpgroup b takes every third step; thread et owns row et. (32 queries of 16 ragged prompts: two of them 74 us, three
// 72, four, with an S buffer each that the next MMAs wait for, 79; three with rows that several warps bring 60.)
template <int D, bool BF16>
__device__ __forceinline__ void win_softmax(const BlockWindowParams& p, uint8_t* smem, uint64_t* bars, int32_t* err, int et, int b,
                                            uint32_t lane_off) {
    using Sh = WinShape<D>;
    // The first two warpgroups also bring the next segment's rows, which are on their way during a step. (One warp of its own took
    // 13 us to bring the first.)
    int k = 0, seg = 0;
    WinWalk w(p), then(p);
    bool more = then.next(), coming = false;
    auto fetch = [&](int s) {
        const Rows<D, 8> rows(smem + Sh::kQ + (s & 1) * Sh::kTile, 4 * b + (et >> 5), et & 31);
        rows.fetch(p, then);
        coming = true;
    };
    auto ready = [&](int s) {
        const Rows<D, 8> rows(smem + Sh::kQ + (s & 1) * Sh::kTile, 4 * b + (et >> 5), et & 31);
        rows.template finish<BF16>(p.scale_log2, reinterpret_cast<int8_t*>(smem + Sh::kPower) + s % kWinRing * 128);
        mbar_arrive(bars + kQFull + s % kWinRing);
        coming = false;
    };
    if (more && b < 2) {
        fetch(0);
        ready(0);
    }
#pragma unroll 1
    for (; more; ++seg) {
        w = then;
        more = then.next();
        if (more && b < 2) {
            if (seg > 0) bar_wait(bars + kQEmpty + ((seg - 1) & 1), (uint32_t)(((seg - 1) >> 1) & 1), err);
            __syncwarp();
            fetch(seg + 1);
        }
        const BlockRowsSeq& e = p.seqs[w.i];
        const int row = w.tile * 128 + et, tiles = (e.n + kTileTokens - 1) / kTileTokens, pad = e.pad;
        const bool valid = row < e.rows;
        const int pos = valid ? e.n - e.q_len + row / p.r : e.n - 1, before = (e.pre_n + kWinStep - 1) / kWinStep;
        float2* out = p.sums + e.sum_begin + (int64_t)w.h * tiles * pad + row;
        float2 total = make_float2(kNegInf, 0.f);
        float qs = 1.f;
        bool first = true;
        const int j0 = w.j0 + (b + kWindowParts - k % kWindowParts) % kWindowParts;
        k += w.j1 - w.j0;
#pragma unroll 1
        for (int j = j0, kk = k - (w.j1 - j0); j < w.j1; j += kWindowParts, kk += kWindowParts) {
            if (first) {
                bar_wait(bars + kQFull + seg % kWinRing, (uint32_t)(seg / kWinRing & 1), err);
                qs = row_factor(p.scale_log2, reinterpret_cast<const int8_t*>(smem + Sh::kPower)[seg % kWinRing * 128 + et]);
                first = false;
            }
            bar_wait(bars + kKFull + kk % kWinRing, (uint32_t)(kk / kWinRing & 1), err);
            const float* hd = reinterpret_cast<const float*>(smem + Sh::kScale) + kk % kWinScales * 4;
            bar_wait(bars + kSFull + (kk & 3), (uint32_t)(kk >> 2 & 1), err);
            __syncwarp();
            tc_fence_after();
            const int lim = j < before ? e.pre_n - j * kWinStep : pos + 1 - (j - before) * kWinStep;  // visible columns
            const bool plain = __all_sync(0xffffffffu, lim >= kWinStep);
            // (rolled: unrolled, the roles together would not fit the instruction cache)
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
                uint32_t r[32];
                tm_ld32(128 * (kk & 3) + 32 * ch + lane_off, r);
                float c = qs * hd[ch];
                if (c < 1e-37f) c = 1e-37f;  // 0 would make -inf of a masked column NaN
                tm_wait_ld();
                if (ch == 3) {  // S may be written again
                    tc_fence_before();
                    mbar_arrive(bars + kSEmpty + (kk & 3));
                }
                const int left = lim - 32 * ch;
                if (!plain) {
#pragma unroll
                    for (int z = 0; z < 32; ++z)
                        if (z >= left) r[z] = 0xff800000u;
                    if (left <= 0) c = 1.f;
                }
                const float m = max32(r) * c, mm = m == kNegInf ? 0.f : m;
                const float2 c2 = make_float2(c, c), a2 = make_float2(-mm, -mm);
                float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
                for (int z = 0; z < 16; ++z) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[2 * z]), __uint_as_float(r[2 * z + 1])), c2, a2);
                    const float2 v = make_float2(ex2f(x.x), ex2f(x.y));
                    if (z & 1) s1 = __fadd2_rn(s1, v);
                    else s0 = __fadd2_rn(s0, v);
                }
                s0 = __fadd2_rn(s0, s1);
                const float2 part = make_float2(m, s0.x + s0.y);
                const int tile = 4 * (j - before) + ch;  // (of a prefix nothing is noted but the rows' totals)
                if (valid && (unsigned)tile < (unsigned)tiles) out[(int64_t)tile * pad] = part;
                total = joined(total, part);
            }
            if (coming) ready(seg + 1);
        }
        if (coming) ready(seg + 1);
        // of the pair's part in this CTA (a pair's first CTA is no sooner than the pair before's last)
        p.totals[((int64_t)(e.pair_begin + w.pair + blockIdx.x) * kWindowParts + b) * 128 + et] = total;
    }
}

template <int D, bool INT8, bool BF16>
__global__ void __launch_bounds__(kWinThreads, 1) window_kernel(const __grid_constant__ BlockWindowParams p) {
    using Sh = WinShape<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int t = threadIdx.x, w = t >> 5, lane = t & 31;
    int32_t* err = reinterpret_cast<int32_t*>(p.c.base + p.c.lay.err);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kBars);
    before_done();  // (ahead of tensor memory, which the kernel before may hold)
    start_next();
    if (t == 0) {
        for (int k = 0; k < kWinRing; ++k) {
            mbar_init(bars + kKFull + k, 128);
            mbar_init(bars + kQFull + k, 256);
        }
        for (int k = 0; k < kWinStages; ++k) mbar_init(bars + kKEmpty + k, 1);
        for (int k = 0; k < 4; ++k) {
            mbar_init(bars + kSFull + k, 1);
            mbar_init(bars + kSEmpty + k, 128);
        }
        for (int k = 0; k < 2; ++k) mbar_init(bars + kQEmpty + k, 1);
        mbar_init(bars + kDrain, 1);
        for (int k = 0; k < kWinExpand * 2; ++k) mbar_init(bars + kRaw + k, 1);
        for (int k = 0; k < 4; ++k) mbar_init(bars + kRaw + 2 * kWinExpand + k, 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (w == kWinIssuer) {
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
    const Rings<D> rings = {smem + Sh::kRings, bars + kRaw, bars + kRaw + 2 * kWinExpand, reinterpret_cast<int32_t*>(smem + Sh::kWhat)};
    const int steps = (int)(p.units * (blockIdx.x + 1) / p.grid - p.units * blockIdx.x / p.grid);
    if (!placed) {
    } else if (w < kWinSoftmax) {
        win_softmax<D, BF16>(p, smem, bars, err, t & 127, w >> 2, (uint32_t)(32 * (w & 3)) << 16);
    } else if (w & 3) {
        const int x = (w - kWinSoftmax) / 4 * 3 + (w & 3) - 1, odd = x >> 2, wp = x & 3;
        expand_steps<D, INT8, BF16, false, 2>(
            rings, x, odd, steps, err, lane,
            [&](int k, float2 h, uint32_t) {
                if (lane == 0) reinterpret_cast<float*>(smem + Sh::kScale)[k % kWinScales * 4 + wp] = h.x;
            },
            [&](int k) {
                if (k >= kWinStages) bar_wait(bars + kKEmpty + k % kWinStages, (uint32_t)((k / kWinStages - 1) & 1), err);
                return smem + Sh::kK + k % kWinStages * Sh::kTile;
            },
            [&](int k) { mbar_arrive(bars + kKFull + k % kWinRing); });
    } else if (w == kWinIssuer) {
        win_issue<D>(p, smem_addr(smem), bars, err);
    } else {
        fill_rings<D, false>(p, rings, (w - kWinIssuer) / 4 - 1, steps, err, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w == kWinIssuer) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*reinterpret_cast<volatile uint32_t*>(smem + Sh::kTmem))
                     : "memory");
    }
}

// ---- shares of the blocks ----
constexpr int kWeighThreads = 256;
constexpr int kWeighRows = 128 * kBlockMaxRatio;  // rows of a KV head

// The CTA that takes unit u: the last b with units b / grid <= u, that is units b < (u + 1) grid. (No division of 64 bits.)
__device__ __forceinline__ int cta_of(int64_t u, int64_t units, int grid) {
    int64_t b = (int64_t)((float)u / (float)units * (float)grid);
    while (units * b >= (u + 1) * grid) --b;
    while (units * (b + 1) < (u + 1) * grid) ++b;
    return (int)b;
}

// A CTA some blocks of a (KV head, sequence): its rows' totals first, then p.lanes lanes (WIDE: 32) a block.
template <int SEQS, bool WIDE>
__global__ void __launch_bounds__(kWeighThreads) weigh_kernel(const __grid_constant__ BlockWeighArgs<SEQS> p) {
    __shared__ float2 of[kWeighRows];  // of a row: its maximum, 1 / denominator (0: adds nothing)
    __shared__ float2 some[kWeighThreads];
    __shared__ int2 ctas[kWeighRows / 128];
    __shared__ float got[WIDE ? 8 * kWeighThreads / 32 : 8 * kWeighThreads];  // of a block
    before_done();
    const BlockWeighSeq& e = p.seqs[blockIdx.z];
    const int h = blockIdx.y, t = threadIdx.x, blocks = (e.tiles + (1 << p.log2_tiles) - 1) >> p.log2_tiles;
    const int first = blockIdx.x * p.blocks;
    if (first >= blocks) return;
    if (p.grid > 0) {  // the CTAs that share each row tile's pair
        if (t < (e.rows + 127) / 128) {
            const int64_t u = e.unit_begin + (int64_t)(h * ((e.rows + 127) / 128) + t) * e.steps;
            ctas[t] = make_int2(cta_of(u, p.units, p.grid), cta_of(u + e.steps - 1, p.units, p.grid));
        }
        __syncthreads();
    }
    for (int row = e.rows + t; row < e.pad; row += kWeighThreads) of[row] = make_float2(0.f, 0.f);
    int span = 32;  // rows at a time; as many threads as there are to a row, each some of its parts
    while (span < kWeighThreads && span < e.rows) span *= 2;
    for (int row0 = 0; row0 < e.rows; row0 += span) {
        const int row = row0 + t % span, turn = t / span, turns = kWeighThreads / span;
        float2 s = make_float2(kNegInf, 0.f);
        if (row >= e.rows) {
        } else if (p.grid == 0) {
            if (turn == 0) s = p.totals[(int64_t)e.row * p.hq + h * e.rows + row];
        } else {  // the parts of the row's pair, of the CTAs that share it
            const int pair = h * ((e.rows + 127) / 128) + row / 128, b0 = ctas[row / 128].x, b1 = ctas[row / 128].y;
            const float2* at = p.totals + (int64_t)(e.pair_begin + pair) * kWindowParts * 128 + row % 128;
#pragma unroll 4
            for (int b = kWindowParts * b0 + turn; b < kWindowParts * (b1 + 1); b += turns) s = joined(s, at[(int64_t)b * 128]);
        }
        if (turns > 1) {
            some[t] = s;
            __syncthreads();
            for (int z = 1; turn == 0 && z < turns; ++z) s = joined(s, some[z * span + t]);
            __syncthreads();
        }
        if (turn == 0 && row < e.rows) of[row] = make_float2(s.x, s.y > 0.f && s.y < -kNegInf ? 1.f / s.y : 0.f);
    }
    __syncthreads();
    const float2* sums = p.sums + e.sum_begin + ((int64_t)h * e.stride + e.before) * e.pad;
    float* to = p.weights + ((int64_t)e.seq * p.hkv + h) * p.cols + first;
    const int count = min(p.blocks, blocks - first);
    auto share = [](float2 x, float2 f) {  // (a tile out of sight: -inf, 0)
        const float y = x.y * ex2f(x.x - f.x);
        return f.y != 0.f ? y * f.y : 0.f;
    };
    if (WIDE) {
        // A warp a block, 128 rows at a time, four a lane, whose totals stay in registers (looked up row by row, 21 us where this
        // takes 14 for 32 queries of 16 ragged prompts).
        const int w = t >> 5, lane = t & 31;
        for (int r0 = 0; r0 < e.pad; r0 += 128) {
            float2 f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = r0 + 32 * i + lane < e.pad ? of[r0 + 32 * i + lane] : make_float2(0.f, 0.f);
            for (int b = w; b < count; b += kWeighThreads / 32) {
                const int t0 = (first + b) << p.log2_tiles, t1 = min(t0 + (1 << p.log2_tiles), e.tiles);
                const float2* at = sums + (int64_t)t0 * e.pad + r0 + lane;
                float sum = 0.f;
#pragma unroll 2
                for (int k = t0; k < t1; ++k, at += e.pad) {
                    float2 x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = r0 + 32 * i + lane < e.pad ? at[32 * i] : make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum += share(x[i], f[i]);
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (lane == 0) got[b] = r0 == 0 ? sum : got[b] + sum;
            }
        }
    } else {
        const int lane = t % p.lanes, lane0 = lane % e.pad, step = p.lanes % e.pad;
        for (int b = t / p.lanes; b < p.blocks; b += kWeighThreads / p.lanes) {  // whole warps
            const int t0 = (first + b) << p.log2_tiles, n = (min(t0 + (1 << p.log2_tiles), e.tiles) - t0) * e.pad;  // negative: none
            const float2* at = sums + (int64_t)t0 * e.pad;
            float sum = 0.f;
            int row = lane0;
#pragma unroll 4
            for (int k = lane; k < n; k += p.lanes) {
                sum += share(at[k], of[row]);
                row += step;
                row -= row >= e.pad ? e.pad : 0;
            }
            for (int d = p.lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (lane == 0) got[b] = sum;
        }
    }
    __syncthreads();
    for (int b = t; b < count; b += kWeighThreads) to[b] += got[b];
}

template <int D, bool INT8, bool BF16>
int launch(const BlockWindowParams& p, cudaStream_t s) {
    static SmemOnce once;
    const int e = once.allow(reinterpret_cast<const void*>(window_kernel<D, INT8, BF16>), WinShape<D>::kSmem);
    if (e) return e;
    return launch_behind(window_kernel<D, INT8, BF16>, p.grid, kWinThreads, WinShape<D>::kSmem, s, p);
}

}  // namespace

int launch_block_window(const BlockWindowParams& p, void* stream) {
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

int launch_block_weigh(const BlockWeighParams& p, void* stream) {
    const dim3 grid(p.most, p.hkv, p.n_seqs);
    cudaStream_t t = (cudaStream_t)stream;
    if (p.n_seqs <= 16) {
        BlockWeighArgs<16> few;
        static_cast<BlockWeighHead&>(few) = p;
        for (int i = 0; i < p.n_seqs; ++i) few.seqs[i] = p.seqs[i];
        return launch_behind(p.lanes == 32 ? weigh_kernel<16, true> : weigh_kernel<16, false>, grid, kWeighThreads, 0, t, few);
    }
    return launch_behind(p.lanes == 32 ? weigh_kernel<kBlockMaxSeqs, true> : weigh_kernel<kBlockMaxSeqs, false>, grid, kWeighThreads, 0, t, p);
}

}  // namespace kvarn
