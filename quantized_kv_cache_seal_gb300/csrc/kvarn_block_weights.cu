// Block cache: what each block of a sequence receives of the softmax weights, added up over queries.
//
//   weights[seq][h][b] += sum over the rows (query token, head of KV head h) and the tokens n of block b of p_n,
//   p_n = 2^(x_n) / sum 2^(x_n'), x_n = scale log2(e) (q . k_n), over the tokens that the row sees.
// A row's denominator is known only behind its last key, so it goes in two steps: whoever makes the logits (decode
// attention, or window_kernel for the last queries of a prompt, which reads K alone) leaves of every 32-token tile and row
// the running maximum m and the tile's sum s of 2^(x - m), 8 bytes for 32 logits; weigh_kernel joins a row's tiles to the
// denominator, and adds the tiles' shares to their blocks in a fixed order. Kept as a pair, no rounding
// of a logit's size stands between a weight and its denominator (log2 of the sum in one word would be off by 2^-17 at 128).
#include <limits.h>

#include "kvarn_block_dev.cuh"
#include "kvarn_tc.cuh"

namespace kvarn {
namespace {

// ---- logits of the last queries ----
// The pairs of a (sequence, KV head, chunk of kWindowRows rows) and its tiles form one line that is cut evenly over the
// CTAs. A pair's rows lie in shared memory in the order of mma.m16n8k16's B operand; a warp takes a tile's codes as A
// operands (the next tile's are on their way) and goes through the rows, eight at a time.
constexpr int kWinWarps = 12, kWinThreads = 32 * kWinWarps;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, bool INT8, bool BF16>
__global__ void __launch_bounds__(kWinThreads, 1) window_kernel(const __grid_constant__ BlockWindowParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const BlockView& c = p.c;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int kPieces = D / 32;  // 16-byte pieces of a lane for eight rows
    uint4* rows = reinterpret_cast<uint4*>(smem);                                      // [row / 8][piece][lane]
    float* factor = reinterpret_cast<float*>(smem + (size_t)p.smem_rows * (2 * D));    // of a row's logits
    int* last = reinterpret_cast<int*>(factor + p.smem_rows);                          // the last position that it sees
    int* down = last + p.smem_rows;                                                    // the power of two that its values lose
    const int64_t u0 = p.units * blockIdx.x / p.grid, u1 = p.units * (blockIdx.x + 1) / p.grid;
    const int sh = c.log2_block - 5;
    int i = 0;
    for (int64_t from = u0; from < u1;) {
#pragma unroll 1
        while (i + 1 < p.n_seqs && p.seqs[i + 1].unit_begin <= from) ++i;
        const BlockWindowSeq& e = p.seqs[i];
        const int pair = (int)((from - e.unit_begin) / e.tiles), kvh = pair / e.chunks, row0 = pair % e.chunks * kWindowRows;
        const int64_t begin = e.unit_begin + (int64_t)pair * e.tiles;
        const int tile0 = (int)(from - begin), tile1 = (int)min(u1 - begin, (int64_t)e.tiles);
        const int count = min(kWindowRows, e.rows - row0), octets = (count + 7) / 8;
        // the pair's rows
        __syncthreads();
        auto source = [&](int row) {
            const int all = row0 + row;
            return p.q + ((size_t)(e.q_row + all / p.r) * p.hq + kvh * p.r + all % p.r) * D;
        };
        for (int row = threadIdx.x; row < 8 * octets; row += kWinThreads) {
            int ex = 0;
            if (BF16 && row < count) {
                uint32_t top = 0;
                const uint4* at = reinterpret_cast<const uint4*>(source(row));
#pragma unroll 4
                for (int k = 0; k < D / 8; ++k) top = max_of(top, at[k]);
                ex = exponent_of<BF16>(max(top & 0xffffu, top >> 16)) - kExactK;
            }
            down[row] = ex;
            factor[row] = p.scale_log2 * power2(ex);
            last[row] = e.n - e.q_len + min(row0 + row, e.rows - 1) / p.r;
        }
        if (BF16) __syncthreads();
        for (int k = threadIdx.x; k < octets * kPieces * 32; k += kWinThreads) {
            const int l = k & 31, piece = k / 32 % kPieces, row = k / (32 * kPieces) * 8 + (l >> 2);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (row < count) {
                x = *reinterpret_cast<const uint4*>(source(row) + 64 * (piece >> 1) + 16 * (l & 3) + 8 * (piece & 1));
                if (BF16) x = scaled_f16<BF16>(x, power2(-down[row]));
            }
            rows[k] = x;
        }
        __syncthreads();
        float2* sums = p.sums + e.sum_begin + (int64_t)kvh * e.tiles * e.pad + row0;
        const int32_t* table = block_table(c, e.seq);
        const int sealed = e.n >> c.log2_block << sh;
        // codes of the warp's next tile, 16 bytes a lane of each 512
        uint4 next[D / 16];
        float next_scale = 1.f;
        auto fetch = [&](int tile) {
            if (tile >= min(tile1, sealed)) return;
            const uint8_t* rec = sealed_tile(c, table, kvh, tile);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) next[k] = __ldg(reinterpret_cast<const uint4*>(rec + 16 + k * 512) + lane);
            next_scale = __ldg(reinterpret_cast<const float*>(rec));
        };
        fetch(tile0 + w);
        for (int tile = tile0 + w; tile < tile1; tile += kWinWarps) {
            uint32_t a[2][D / 16][4];  // half of 16 tokens, 16 channels, registers of the A operand
            float ks = 1.f;
            if (tile < sealed) {
                ks = next_scale;
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int y = 0; y < D / 64; ++y) {
                        const uint4 u = next[(z * (D / 64) + y) * 2], v = next[(z * (D / 64) + y) * 2 + 1];
                        const uint32_t x4[4] = {u.x, u.y, u.z, u.w}, y4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            a[z][4 * y + j][0] = codes_lo<INT8>(x4[j]);
                            a[z][4 * y + j][1] = codes_lo<INT8>(y4[j]);
                            a[z][4 * y + j][2] = codes_hi<INT8>(x4[j]);
                            a[z][4 * y + j][3] = codes_hi<INT8>(y4[j]);
                        }
                    }
                fetch(tile + kWinWarps);
            } else {  // exact rows
                const uint16_t* k = tail_ptr(c, c.lay.tail_k, e.seq, kvh) + (size_t)(tile - sealed) * (kTileTokens * D);
                const int nv = e.n - tile * kTileTokens;
                uint32_t top = 0;
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int tok = 8 * (g >> 1) + 4 * z + 2 * b + (g & 1);
#pragma unroll
                        for (int y = 0; y < D / 32; ++y) {
                            uint4 x = make_uint4(0, 0, 0, 0);
                            if (tok < nv) x = *reinterpret_cast<const uint4*>(k + tok * D + 64 * (y >> 1) + 16 * t + 8 * (y & 1));
                            if (BF16) top = max_of(top, finite_only<BF16>(x));
                            a[z][2 * y][b] = x.x;
                            a[z][2 * y][2 + b] = x.y;
                            a[z][2 * y + 1][b] = x.z;
                            a[z][2 * y + 1][2 + b] = x.w;
                        }
                    }
                if (BF16) {
                    const int ex = warp_exponent<BF16>(top) - kExactK;
                    ks = power2(ex);
                    const float f = power2(-ex);
#pragma unroll
                    for (int z = 0; z < 2; ++z)
#pragma unroll
                        for (int y = 0; y < D / 16; ++y)
#pragma unroll
                            for (int x = 0; x < 4; ++x) a[z][y][x] = scaled_f16<BF16>(a[z][y][x], f);
                }
            }
            const bool plain = (tile + 1) * kTileTokens <= e.n - e.q_len + row0 / p.r + 1;  // every row sees all of it
            float2* out = sums + (int64_t)tile * e.pad;
#pragma unroll 1
            for (int o = 0; o < octets; ++o) {
                float s[2][4] = {};
#pragma unroll
                for (int y = 0; y < kPieces; ++y) {
                    const uint4 b = rows[(o * kPieces + y) * 32 + lane];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        mma16816(s[z], a[z][2 * y][0], a[z][2 * y][1], a[z][2 * y][2], a[z][2 * y][3], b.x, b.y);
                        mma16816(s[z], a[z][2 * y + 1][0], a[z][2 * y + 1][1], a[z][2 * y + 1][2], a[z][2 * y + 1][3], b.z, b.w);
                    }
                }
                const int r = 8 * o + 2 * t;
                const float2 f = *reinterpret_cast<const float2*>(factor + r);
                const float f0 = f.x * ks, f1 = f.y * ks;
                int2 l = make_int2(INT_MAX, INT_MAX);
                if (!plain) l = *reinterpret_cast<const int2*>(last + r);
                const int pos = tile * kTileTokens + 8 * (g >> 1) + (g & 1);  // of a lane's first token; the others 4 z + 2 b on
                float m0 = kNegInf, m1 = kNegInf;
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        if (pos + 4 * z + 2 * b <= l.x) m0 = fmaxf(m0, s[z][2 * b] * f0);
                        if (pos + 4 * z + 2 * b <= l.y) m1 = fmaxf(m1, s[z][2 * b + 1] * f1);
                    }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
                    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
                }
                const float n0 = m0 == kNegInf ? 0.f : m0, n1 = m1 == kNegInf ? 0.f : m1;
                float l0 = 0.f, l1 = 0.f;
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        if (pos + 4 * z + 2 * b <= l.x) l0 += ex2f(fmaf(s[z][2 * b], f0, -n0));
                        if (pos + 4 * z + 2 * b <= l.y) l1 += ex2f(fmaf(s[z][2 * b + 1], f1, -n1));
                    }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
                    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
                }
                if (g == 0) *reinterpret_cast<float4*>(out + r) = make_float4(m0, l0, m1, l1);
            }
        }
        from = begin + tile1;
    }
}

// ---- shares of the blocks ----
constexpr int kWeighWarps = 16, kWeighThreads = 32 * kWeighWarps;
constexpr int kWeighRows = 128 * kBlockMaxRatio;  // rows of a KV head

struct Sum {
    float m, l;  // 2^m l
    __device__ __forceinline__ void add(float om, float ol) {
        const float top = fmaxf(m, om);
        const float f = m == kNegInf ? 1.f : ex2f(m - top), of = om == kNegInf ? 1.f : ex2f(om - top);  // -inf: 0 or NaN
        l = l * f + ol * of;
        m = top;
    }
};

// A CTA a (KV head, sequence). The rows' denominators first, a lane a row and the warps in turns of tiles; then the
// blocks, a warp each.
__global__ void __launch_bounds__(kWeighThreads) weigh_kernel(const __grid_constant__ BlockWeighParams p) {
    __shared__ float top[kWeighRows], share[kWeighRows];  // of a row: its maximum, 1 / denominator (0: adds nothing)
    __shared__ Sum part[kWeighWarps][32];
    const BlockWeighSeq& e = p.seqs[blockIdx.y];
    const int h = blockIdx.x, w = threadIdx.x >> 5, lane = threadIdx.x & 31, tiles = e.before + e.tiles;
    const float2* sums = p.sums + e.sum_begin + (int64_t)h * tiles * e.pad;
    int span = 1;  // lanes of a tile
    while (span < min(e.rows, 32)) span *= 2;
    for (int row0 = 0; row0 < e.rows; row0 += span) {
        const int row = row0 + lane % span, step = 32 / span;
        Sum s = {kNegInf, 0.f};
        if (row < e.rows) {
#pragma unroll 4
            for (int k = w * step + lane / span; k < tiles; k += kWeighWarps * step) {
                const float2 x = sums[(int64_t)k * e.pad + row];
                s.add(x.x, x.y);
            }
        }
        for (int d = span; d < 32; d *= 2) s.add(__shfl_xor_sync(0xffffffffu, s.m, d), __shfl_xor_sync(0xffffffffu, s.l, d));
        part[w][lane] = s;
        __syncthreads();
        if (w == 0 && lane < span && row < e.rows) {
#pragma unroll
            for (int z = 1; z < kWeighWarps; ++z) s.add(part[z][lane].m, part[z][lane].l);
            if (e.lse_row >= 0) s.add(p.pre_lse[(int64_t)e.lse_row * p.hq + h * e.rows + row] + p.shift, 1.f);
            top[row] = s.m;
            share[row] = s.l > 0.f && s.l < -kNegInf ? 1.f / s.l : 0.f;
        }
        __syncthreads();
    }
    const int blocks = (e.tiles + (1 << p.log2_tiles) - 1) >> p.log2_tiles;
    float* to = p.weights + ((int64_t)e.seq * p.hkv + h) * p.cols;
    for (int b = w; b < blocks; b += kWeighWarps) {
        const int t0 = b << p.log2_tiles, t1 = min(t0 + (1 << p.log2_tiles), e.tiles);
        const float2* at = sums + (int64_t)(e.before + t0) * e.pad;
        float sum = 0.f;
#pragma unroll 4
        for (int k = lane; k < (t1 - t0) * e.pad; k += 32) {
            const int row = k % e.pad;
            if (row >= e.rows || share[row] == 0.f) continue;
            const float2 x = at[k];
            if (x.x != kNegInf) sum += x.y * ex2f(x.x - top[row]) * share[row];
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) to[b] += sum;
    }
}

template <int D, bool INT8, bool BF16>
int launch(const BlockWindowParams& p, cudaStream_t s) {
    static SmemOnce once;
    const int e = once.allow(reinterpret_cast<const void*>(window_kernel<D, INT8, BF16>), kWindowRows * (2 * D + 12));
    if (e) return e;
    window_kernel<D, INT8, BF16><<<p.grid, kWinThreads, (size_t)p.smem_rows * (2 * D + 12), s>>>(p);
    return (int)cudaGetLastError();
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
    weigh_kernel<<<dim3(p.hkv, p.n_seqs), kWeighThreads, 0, (cudaStream_t)stream>>>(p);
    return (int)cudaGetLastError();
}

}  // namespace kvarn
