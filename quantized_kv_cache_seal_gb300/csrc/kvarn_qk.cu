// RMS norm of every query and key head with a weight, then the position rotation, in one
// pass (the cache takes post-rotation keys and queries).
//   y_d = x_d rsqrt(mean x^2 + eps) w_d;  pairs (y_i, y_{i+R/2}) or (y_2i, y_{2i+1}) turned
//   by position * freq_i; channels from R on pass through. fp32 throughout, one rounding.
//
// Bound by memory: each value is read once and written once. A group of 8, 16 or 32 lanes
// takes items (one token, some of its heads), one head row at a time, 8 channels a lane, so
// that both halves of a pair sit in one lane and only the norm's sum crosses lanes; cos and
// sin are computed once an item and reused for its heads. The angle is kept as a 64-bit
// fraction of a turn: frac(freq / 2 pi) * 2^64 times the position, modulo 2^64, drops
// whole turns exactly at any position; its top 32 bits then go to sincospi. The fraction is
// the only fp64 arithmetic (slow on this chip: done once an item it took twice the time of
// the memory traffic), so in large calls a group takes several items and does it once.
// Measured: 49,157 tokens of 40 + 10 heads of 128 in 204 us, 6.2 TB/s; 4,096 tokens of 32 + 8
// in 26 us, 3.2 TB/s (a single round of groups: latency).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kvarn_block.h"

namespace kvarn {
namespace {

constexpr int kQkThreads = 128;

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

// Lane l of a group owns channels: interleaved, 8 l .. 8 l + 7; otherwise, for l < R / 8,
// 4 l .. 4 l + 3 and R / 2 + 4 l .. + 3, and from R on 8 l .. 8 l + 7.
template <bool IN_BF16, bool OUT_BF16, int LANES>
__global__ void __launch_bounds__(kQkThreads, 8) qk_kernel(const __grid_constant__ QkParams p) {
    constexpr int kAhead = 4;  // rows in flight
    const int l = threadIdx.x % LANES;
    const unsigned group = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u) << ((threadIdx.x & 31) / LANES * LANES);
    const bool live = 8 * l < p.d;
    const bool turned = 8 * l < p.rot;
    const bool halves = turned && !p.interleaved;
    const int c0 = halves ? 4 * l : 8 * l;                  // first four channels
    const int c1 = halves ? p.rot / 2 + 4 * l : 8 * l + 4;  // last four
    uint64_t frac[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        frac[i] = 0;
        if (turned) {
            double f = p.freqs[4 * l + i] * 0.15915494309189533577;  // turns a position
            f -= floor(f);
            frac[i] = (uint64_t)(f * 18446744073709551616.0);
        }
    }
    // a CTA's items are consecutive, its groups take them in turn
    constexpr int kGroups = kQkThreads / LANES;
    const int items = (int)(p.n_tokens * p.items_per_token), first = blockIdx.x * kGroups * p.items_per_group;
    const int end = min(items, first + kGroups * p.items_per_group);
    for (int item = first + threadIdx.x / LANES; item < end; item += kGroups) {  // whole groups
        const int64_t tok = item / p.items_per_token;
        const int h0 = item % p.items_per_token * p.heads_per_item, h1 = min(h0 + p.heads_per_item, p.hq + p.hkv);
        const uint16_t* qr = p.q + tok * p.q_stride;
        const uint16_t* kr = p.k + tok * p.k_stride;
        uint16_t* qo = p.q_out + tok * p.q_out_stride;
        uint16_t* ko = p.k_out + tok * p.k_out_stride;
        float cs[4], sn[4];
        for (int hb = h0; hb < h1; hb += kAhead) {
            uint2 a[kAhead], b[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = hb + u;
                a[u] = b[u] = make_uint2(0, 0);
                if (h < h1 && live) {
                    const uint16_t* x = h < p.hq ? qr + (int64_t)h * p.d : kr + (int64_t)(h - p.hq) * p.d;
                    if (halves) {
                        a[u] = *reinterpret_cast<const uint2*>(x + c0);
                        b[u] = *reinterpret_cast<const uint2*>(x + c1);
                    } else {
                        const uint4 w = *reinterpret_cast<const uint4*>(x + c0);
                        a[u] = make_uint2(w.x, w.y);
                        b[u] = make_uint2(w.z, w.w);
                    }
                }
            }
            if (hb == h0 && turned) {  // over the loads' latency
                const int64_t pos = p.positions[tok];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int32_t top = (int32_t)((frac[i] * (uint64_t)pos) >> 32);
                    sincospif((float)top * 4.656612873077393e-10f, &sn[i], &cs[i]);  // top 2^-32 turns, 2 to a pi
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int h = hb + u;
                if (h >= h1) break;  // the same for the whole group
                float y[8];
                float2 f;
                f = unpack2<IN_BF16>(a[u].x), y[0] = f.x, y[1] = f.y;
                f = unpack2<IN_BF16>(a[u].y), y[2] = f.x, y[3] = f.y;
                f = unpack2<IN_BF16>(b[u].x), y[4] = f.x, y[5] = f.y;
                f = unpack2<IN_BF16>(b[u].y), y[6] = f.x, y[7] = f.y;
                const bool is_q = h < p.hq;
                const float* wt = is_q ? p.q_weight : p.k_weight;
                if (wt) {
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
                    for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(group, ss, m);
                    const float rs = rsqrtf(ss * p.inv_d + p.eps);
                    if (live) {  // 1 KB at most: from the first cache
                        const float4 w0 = __ldg(reinterpret_cast<const float4*>(wt + c0));
                        const float4 w1 = __ldg(reinterpret_cast<const float4*>(wt + c1));
                        y[0] *= rs * w0.x, y[1] *= rs * w0.y, y[2] *= rs * w0.z, y[3] *= rs * w0.w;
                        y[4] *= rs * w1.x, y[5] *= rs * w1.y, y[6] *= rs * w1.z, y[7] *= rs * w1.w;
                    }
                }
                if (turned) {
                    if (p.interleaved) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float u0 = y[2 * i], u1 = y[2 * i + 1];
                            y[2 * i] = u0 * cs[i] - u1 * sn[i];
                            y[2 * i + 1] = u1 * cs[i] + u0 * sn[i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float u0 = y[i], u1 = y[4 + i];
                            y[i] = u0 * cs[i] - u1 * sn[i];
                            y[4 + i] = u1 * cs[i] + u0 * sn[i];
                        }
                    }
                }
                if (live) {
                    uint16_t* o = is_q ? qo + (int64_t)h * p.d : ko + (int64_t)(h - p.hq) * p.d;
                    const uint2 lo = make_uint2(pack2<OUT_BF16>(y[0], y[1]), pack2<OUT_BF16>(y[2], y[3]));
                    const uint2 hi = make_uint2(pack2<OUT_BF16>(y[4], y[5]), pack2<OUT_BF16>(y[6], y[7]));
                    if (halves) {
                        *reinterpret_cast<uint2*>(o + c0) = lo;
                        *reinterpret_cast<uint2*>(o + c1) = hi;
                    } else {
                        *reinterpret_cast<uint4*>(o + c0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    }
                }
            }
        }
    }
}

template <bool I, bool O>
int launch_qk(const QkParams& p, cudaStream_t s) {
    const int lanes = p.d <= 64 ? 8 : p.d <= 128 ? 16 : 32;
    const int64_t per_cta = (int64_t)(kQkThreads / lanes) * p.items_per_group;
    const unsigned grid = (unsigned)((p.n_tokens * p.items_per_token + per_cta - 1) / per_cta);
    if (lanes == 8) qk_kernel<I, O, 8><<<grid, kQkThreads, 0, s>>>(p);
    else if (lanes == 16) qk_kernel<I, O, 16><<<grid, kQkThreads, 0, s>>>(p);
    else qk_kernel<I, O, 32><<<grid, kQkThreads, 0, s>>>(p);
    return (int)cudaGetLastError();
}

}  // namespace

int launch_qk_norm_rope(const QkParams& p, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    if (p.in_bf16) return p.out_bf16 ? launch_qk<true, true>(p, s) : launch_qk<true, false>(p, s);
    return p.out_bf16 ? launch_qk<false, true>(p, s) : launch_qk<false, false>(p, s);
}

}  // namespace kvarn
