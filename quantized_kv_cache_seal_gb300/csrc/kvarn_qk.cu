// RMS norm of every query and key head with a weight, then the position rotation, in one
// pass (the cache takes post-rotation keys and queries).
//   y_d = x_d rsqrt(mean x^2 + eps) w_d;  pairs (y_i, y_{i+R/2}) or (y_2i, y_{2i+1}) turned
//   by position * freq_i; channels from R on pass through. fp32 throughout, one rounding.
//
// Norm, weight and rotation are one linear map of a pair: out = rsqrt(..) (y c + partner s), with
// c and s (cos, sin times the weights) made once for all heads of a token that an item holds.
//
// Bound by memory: each value is read once and written once. A group of 8, 16 or 32 lanes
// takes an item (one token, some of its heads), eight head rows in flight, 8 channels a lane, so
// that both halves of a pair sit in one lane and only the norm's sums cross lanes, eight rows'
// together. The angle is kept as a 64-bit fraction of a turn: frac(freq / 2 pi) * 2^64 times the
// position, modulo 2^64, drops whole turns exactly at any position; its top 32 bits then go to
// sincospi. No fp64 arithmetic is used: this chip has little, and the few operations that a lane
// needed of it once an item took twice the time of the memory traffic.
//
// Measured: 49,157 tokens of 40 + 10 heads of 128 in 188 us, 6.7 TB/s (with weights 192 us); 4,096
// tokens of 32 + 8 with weights in 16.5 us, 5.1 TB/s (the kernel; a call from Python takes 19 to 22).
// head_dims of 64 and 256 alike. Others run with sizes known at run time and idle lanes: as many bytes
// at 80, 96 and 192 in 301, 259 and 257 us, with weights 361, 307 and 306.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvarn_block.h"

namespace kvarn {
namespace {

// 96 registers a thread, eight rows in flight (with runtime sizes, 4,096 tokens of 40 heads: 20.8 us; 80 and
// four rows 22.6; with 64, which do not hold four rows and the map, 34; kAny needs 122).
constexpr int kQkThreads = 128, kQkCtas = 5, kAhead = 8;

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// frac(freq / 2 pi) * 2^64, from integers: with freq = M 2^(E - 1086), M of 64 bits, and C = 2^64 * 2 / pi
// rounded, the high half of M C is turns * 2^(1024 - E), to 2^-63 of it (a double product: 2^-53). From 4
// radians on whole turns go out at the top and as many bits come in at the bottom: the next words of M times
// 128 bits of 2 / pi, so that the fraction keeps 2^-64 up to 2^64 radians (and means little beyond 2^53).
__device__ __forceinline__ uint64_t turns(double freq) {
    const int64_t bits = __double_as_longlong(freq);
    const int s = (int)(bits >> 52 & 0x7ff) - 1024;
    const uint64_t m = ((uint64_t)bits << 11) | 1ull << 63;
    uint64_t f;
    if (s <= 0) {
        f = s > -64 ? __umul64hi(m, 0xa2f9836e4e44152aull) >> -s : 0;
    } else {
        constexpr uint64_t c1 = 0xa2f9836e4e441529ull, c0 = 0xfc2757d1f534ddc0ull;
        const uint64_t low = m * c1, next = low + __umul64hi(m, c0), top = __umul64hi(m, c1) + (next < low);
        f = s < 64 ? top << s | next >> (64 - s) : s == 64 ? next : 0;
    }
    return bits < 0 ? 0 - f : f;
}

// Lane l of a group owns channels: interleaved, 8 l .. 8 l + 7; otherwise, for l < R / 8,
// 4 l .. 4 l + 3 and R / 2 + 4 l .. + 3, and from R on 8 l .. 8 l + 7.
// kAny: any head_dim and order; the others: head_dim 8 * LANES, and in the last two rot_dim too. (20,000 tokens
// of 40 heads, rotated whole: 67.5 us as kFullHalves, 68.1 as kHalves; with rot_dim 64 of 128 68.7 as kHalves,
// 89.5 as kAny.)
enum { kAny, kHalves, kPairs, kFullHalves, kFullPairs };

template <bool IN_BF16, int LANES, int MODE>
__global__ void __launch_bounds__(kQkThreads, MODE == kAny ? 4 : kQkCtas) qk_kernel(const __grid_constant__ QkParams p) {
    const int l = threadIdx.x % LANES;
    const unsigned group = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u) << ((threadIdx.x & 31) / LANES * LANES);
    const int d = MODE != kAny ? 8 * LANES : p.d;
    const bool live = MODE != kAny || 8 * l < d;
    constexpr bool kFull = MODE >= kFullHalves, kTwo = MODE == kHalves || MODE == kFullHalves;  // kTwo: two pieces a row
    const bool turned = kFull || 8 * l < p.rot;
    const bool pairs = MODE == kAny ? p.interleaved : !kTwo;
    const bool halves = turned && !pairs;
    const int c0 = halves ? 4 * l : 8 * l;                  // first four channels
    const int c1 = halves ? (kFull ? 4 * LANES : p.rot / 2) + 4 * l : 8 * l + 4;  // last four
    const int item = blockIdx.x * (kQkThreads / LANES) + threadIdx.x / LANES;
    const int64_t tok = item / p.items_per_token;
    if (tok >= p.n_tokens) return;  // whole groups
    const int h0 = item % p.items_per_token * p.heads_per_item, h1 = min(h0 + p.heads_per_item, p.hq + p.hkv);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {  // q, k
        const int first = side ? max(h0 - p.hq, 0) : h0;
        const int rows = (side ? h1 - p.hq : min(h1, p.hq)) - first;
        if (rows <= 0) continue;
        const uint16_t* in = (side ? p.k + tok * p.k_stride : p.q + tok * p.q_stride) + (int64_t)first * d;
        uint16_t* out = (side ? p.k_out + tok * p.k_out_stride : p.q_out + tok * p.q_out_stride) + (int64_t)first * d;
        const float* wt = side ? p.k_weight : p.q_weight;
        float2 c[4], s[4];  // out = y c + partner s
#pragma unroll 1
        for (int hb = 0; hb < rows; hb += kAhead) {
            uint2 a[kAhead], b[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                a[u] = b[u] = make_uint2(0, 0);
                if (hb + u < rows && live) {
                    const uint16_t* x = in + u * d;
                    if (kTwo || halves) {
                        a[u] = *reinterpret_cast<const uint2*>(x + c0);
                        b[u] = *reinterpret_cast<const uint2*>(x + c1);
                    } else {
                        const uint4 w = *reinterpret_cast<const uint4*>(x + c0);
                        a[u] = make_uint2(w.x, w.y);
                        b[u] = make_uint2(w.z, w.w);
                    }
                }
            }
            if (hb == 0) {  // over the loads' latency
                float4 w0 = make_float4(1.f, 1.f, 1.f, 1.f), w1 = w0;
                if (wt && live) {
                    w0 = __ldg(reinterpret_cast<const float4*>(wt + c0));
                    w1 = __ldg(reinterpret_cast<const float4*>(wt + c1));
                }
                float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {};
                if (turned) {
                    const int64_t pos = p.positions[tok];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t top = (int32_t)((turns(p.freqs[4 * l + i]) * (uint64_t)pos) >> 32);
                        sincospif((float)top * 4.656612873077393e-10f, &sn[i], &cs[i]);  // top 2^-32 turns, 2 to a pi
                    }
                }
                if (pairs) {
                    c[0] = make_float2(w0.x * cs[0], w0.y * cs[0]), s[0] = make_float2(-w0.y * sn[0], w0.x * sn[0]);
                    c[1] = make_float2(w0.z * cs[1], w0.w * cs[1]), s[1] = make_float2(-w0.w * sn[1], w0.z * sn[1]);
                    c[2] = make_float2(w1.x * cs[2], w1.y * cs[2]), s[2] = make_float2(-w1.y * sn[2], w1.x * sn[2]);
                    c[3] = make_float2(w1.z * cs[3], w1.w * cs[3]), s[3] = make_float2(-w1.w * sn[3], w1.z * sn[3]);
                } else {
                    c[0] = make_float2(w0.x * cs[0], w0.y * cs[1]), s[0] = make_float2(-w1.x * sn[0], -w1.y * sn[1]);
                    c[1] = make_float2(w0.z * cs[2], w0.w * cs[3]), s[1] = make_float2(-w1.z * sn[2], -w1.w * sn[3]);
                    c[2] = make_float2(w1.x * cs[0], w1.y * cs[1]), s[2] = make_float2(w0.x * sn[0], w0.y * sn[1]);
                    c[3] = make_float2(w1.z * cs[2], w1.w * cs[3]), s[3] = make_float2(w0.z * sn[2], w0.w * sn[3]);
                }
            }
            float rs[kAhead];
            if (wt) {  // the rows' sums cross the lanes together
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    float2 f = unpack2<IN_BF16>(a[u].x), g = __fmul2_rn(f, f);
                    f = unpack2<IN_BF16>(a[u].y), g = __ffma2_rn(f, f, g);
                    f = unpack2<IN_BF16>(b[u].x), g = __ffma2_rn(f, f, g);
                    f = unpack2<IN_BF16>(b[u].y), g = __ffma2_rn(f, f, g);
                    rs[u] = g.x + g.y;
                }
#pragma unroll
                for (int m = LANES / 2; m > 0; m >>= 1)
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) rs[u] += __shfl_xor_sync(group, rs[u], m);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) rs[u] = rsqrtf(rs[u] * p.inv_d + p.eps);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (hb + u >= rows || !live) break;
                const float2 y[4] = {unpack2<IN_BF16>(a[u].x), unpack2<IN_BF16>(a[u].y), unpack2<IN_BF16>(b[u].x),
                                     unpack2<IN_BF16>(b[u].y)};
                float2 o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = __fmul2_rn(y[i], c[i]);
                if (turned) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = __ffma2_rn(pairs ? make_float2(y[i].y, y[i].x) : y[i ^ 2], s[i], o[i]);
                }
                if (wt) {
                    const float2 r = make_float2(rs[u], rs[u]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = __fmul2_rn(o[i], r);
                }
                uint2 lo, hi;
                if (p.out_bf16) {
                    lo = make_uint2(pack2<true>(o[0].x, o[0].y), pack2<true>(o[1].x, o[1].y));
                    hi = make_uint2(pack2<true>(o[2].x, o[2].y), pack2<true>(o[3].x, o[3].y));
                } else {
                    lo = make_uint2(pack2<false>(o[0].x, o[0].y), pack2<false>(o[1].x, o[1].y));
                    hi = make_uint2(pack2<false>(o[2].x, o[2].y), pack2<false>(o[3].x, o[3].y));
                }
                uint16_t* z = out + u * d;
                if (kTwo || halves) {
                    *reinterpret_cast<uint2*>(z + c0) = lo;
                    *reinterpret_cast<uint2*>(z + c1) = hi;
                } else {
                    *reinterpret_cast<uint4*>(z + c0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
            }
            in += kAhead * d;
            out += kAhead * d;
        }
    }
}

template <bool I, int LANES>
int launch_qk(const QkParams& p, cudaStream_t s) {
    constexpr int kPerCta = kQkThreads / LANES;
    const unsigned grid = (unsigned)((p.n_tokens * p.items_per_token + kPerCta - 1) / kPerCta);
    if (p.d != 8 * LANES) qk_kernel<I, LANES, kAny><<<grid, kQkThreads, 0, s>>>(p);
    else if (p.interleaved && p.rot == p.d) qk_kernel<I, LANES, kFullPairs><<<grid, kQkThreads, 0, s>>>(p);
    else if (p.interleaved) qk_kernel<I, LANES, kPairs><<<grid, kQkThreads, 0, s>>>(p);
    else if (p.rot == p.d) qk_kernel<I, LANES, kFullHalves><<<grid, kQkThreads, 0, s>>>(p);
    else qk_kernel<I, LANES, kHalves><<<grid, kQkThreads, 0, s>>>(p);
    return (int)cudaGetLastError();
}
template <bool I>
int launch_lanes(const QkParams& p, cudaStream_t s) {
    return p.d <= 64 ? launch_qk<I, 8>(p, s) : p.d <= 128 ? launch_qk<I, 16>(p, s) : launch_qk<I, 32>(p, s);
}

}  // namespace

int launch_qk_norm_rope(const QkParams& p, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    return p.in_bf16 ? launch_lanes<true>(p, s) : launch_lanes<false>(p, s);
}

}  // namespace kvarn
