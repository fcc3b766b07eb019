// Block cache: writing (quantising) and reading back.
//
// Sealed, per (block, KV head, K or V) with amax = max |x|:
//   e4m3: s = 2^e with the smallest e >= -100 for which amax <= 448 2^e; the code is x / s
//         rounded to nearest even. x / s is exact (a power of two), so the code never
//         depends on how the division was done.
//   int8: s = max(amax / 127 in fp32, 2^-100); the code is the whole number nearest to the
//         real quotient x / s, ties to even, at most 127 in size.
// amax = 0: s = 1. A non-finite value in the block: s = NaN, every value of the block reads
// NaN. The partial newest block stays exact, so the result does not depend on how the
// tokens were cut into calls.
#include "kvarn_block_dev.cuh"

namespace kvarn {
namespace {

constexpr int kWriteThreads = 256;

// Rounds x to the code of the real quotient x / s. n is first taken from x * (1 / s), which is
// within a few ulp of the quotient, then corrected from the remainder r = x - n s: x has at
// most 11 significant bits, so wherever |x| >= s / 2 its last bit is worth more than s's, r is
// a multiple of s's last bit below 2^24 of them, and the fma gives it exactly.
__device__ __forceinline__ int int8_code(float x, float s, float inv) {
    float n = rintf(x * inv);
    const float r = fmaf(-n, s, x), r2 = 2.f * fabsf(r);
    if (r2 > s || (r2 == s && ((int)n & 1))) n += r > 0.f ? 1.f : -1.f;
    return (int)fminf(fmaxf(n, -127.f), 127.f);
}

// Four codes + 128, as bytes. The nearest whole numbers come out of the low bits of a sum with 1.5 * 2^23
// + 128; where every remainder is under half of s they are right, and only otherwise (ties among them)
// taken one by one. |x / s| <= 127 (1 + 2^-22), so nothing needs a clamp. (131,072 tokens of 8 heads,
// normal values: 168 us; one by one throughout 260; e4m3, without the remainders, 144.)
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d, float s, float inv) {
    constexpr float kSum = 12582912.f + 128.f;
    const float2 inv2 = make_float2(inv, inv), less = make_float2(-s, -s);
    const float2 x[2] = {make_float2(a, b), make_float2(c, d)};
    float2 t[2];
    float r = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        t[i] = __ffma2_rn(x[i], inv2, make_float2(kSum, kSum));
        const float2 u = __ffma2_rn(__fadd2_rn(t[i], make_float2(-kSum, -kSum)), less, x[i]);
        asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(r) : "f"(u.x), "f"(u.y));
    }
    uint32_t w = __byte_perm(__byte_perm(__float_as_uint(t[0].x), __float_as_uint(t[0].y), 0x0040),
                             __byte_perm(__float_as_uint(t[1].x), __float_as_uint(t[1].y), 0x0040), 0x5410);
    if (__builtin_expect(r >= 0.5f * s, 0)) {
        w = 0;
#pragma unroll 1
        for (int i = 3; i >= 0; --i)
            w = w << 8 | (uint32_t)(int8_code(i == 0 ? a : i == 1 ? b : i == 2 ? c : d, s, inv) + 128);
    }
    return w;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// One group of B D / 64 threads per (sequence, completed block, K or V, KV head); a thread
// holds 8 tokens x 8 channels, so that the V codes (channel-major) are turned in its
// registers. The group of a sequence's first completed block also moves the tokens behind the
// last block into the exact tail, after it has read the old tail: both use the same rows.
// Bound by memory; the input is read once (16-byte loads, whole rows) and codes leave in
// 32-byte sectors or larger. 64 sequences, ragged, written and read back (read_kernel), e4m3: 1,575
// us, 6.0 TB/s together; smaller calls are bound by the two launches.
template <int D, bool BF16, class P>
__global__ void __launch_bounds__(kWriteThreads) append_kernel(const __grid_constant__ P p) {
    __shared__ uint32_t red[kWriteThreads / 32];
    const BlockView& c = p.c;
    constexpr int d = D;
    const int bt = c.block, lb = c.log2_block;
    const int lg = lb + (D == 128 ? 1 : 0), tpg = 1 << lg;  // threads of a group: 32 .. 256
    const int item = blockIdx.x * (kWriteThreads >> lg) + (threadIdx.x >> lg);
    const int tid = threadIdx.x & (tpg - 1);
    const bool on = item < p.items;
    int i = 0;
    for (int lo = 0, hi = p.n_seqs - 1; on && lo < hi; i = lo) {  // last sequence that begins at or before the item
        const int mid = (lo + hi + 1) / 2;
        if (p.seqs[mid].item_begin <= item) lo = mid; else hi = mid - 1;
    }
    const BlockAppendSeq& e = p.seqs[i];
    const int rel = item - e.item_begin;
    const int h = rel % c.hkv, side = rel / c.hkv % 2, j = rel / (2 * c.hkv);
    const int first = e.n_before >> lb;  // first block that the call touches
    const bool seals = on && j < e.n_blocks;
    const uint16_t* in = side ? p.v : p.k;
    const int64_t stride = side ? p.v_stride : p.k_stride;
    uint16_t* tail = on ? tail_ptr(c, side ? c.lay.tail_v : c.lay.tail_k, e.seq, h) : nullptr;
    const int c8 = tid % (d / 8), oct = tid / (d / 8);  // 8 channels, 8 tokens
    const int p0 = ((first + j) << lb) + 8 * oct;       // first of the 8 positions
    uint4 x[8];
    uint32_t top = 0;
    if (seals) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int pos = p0 + u;
            if (pos >= e.n_before) {
                x[u] = *reinterpret_cast<const uint4*>(in + (e.in_row + (int64_t)(pos - e.n_before)) * stride +
                                                       h * d + 8 * c8);
            } else if (side == 0) {
                x[u] = *reinterpret_cast<const uint4*>(tail + (size_t)(pos & (bt - 1)) * d + 8 * c8);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[q] = (uint32_t)tail[tail_v_off(d, pos & (bt - 1), 8 * c8 + 2 * q)] |
                           ((uint32_t)tail[tail_v_off(d, pos & (bt - 1), 8 * c8 + 2 * q + 1)] << 16);
                x[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                                         __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu)));
        }
        top = max(top & 0xffffu, top >> 16);  // 16-bit patterns without sign order as their values
    }
    for (int m = 16; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();  // also: the old tail has been read
    if (seals) {
        const int w0 = (threadIdx.x - tid) >> 5;
        for (int w = 0; w < tpg / 32; ++w) top = max(top, red[w0 + w]);
        const bool finite = top < (BF16 ? 0x7f80u : 0x7c00u);
        const float amax = unpack2<BF16>(top).x;
        float s = 1.f;
        if (!finite) {
            s = __int_as_float(0x7fc00000);
        } else if (amax > 0.f) {
            if (c.int8) {
                s = fmaxf(__fdiv_rn(amax, 127.f), 7.888609052210118e-31f);
            } else {
                // amax = 1.f 2^x (as fp32 every 16-bit value but a bf16 subnormal is normal, and
                // those fall under the smallest scale): 1.f <= 1.75 gives e = x - 8, else x - 7
                const uint32_t b = __float_as_uint(amax);
                const int ex = (int)(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
                s = __uint_as_float((uint32_t)(max(ex, -100) + 127) << 23);
            }
        }
        const float inv = 1.f / s;
        const int slot = p.slots[e.slot_begin + j];
        const int tile = oct / 4, tok = (8 * oct) % kTileTokens;
        uint8_t* t = tile_ptr(c, slot, h, tile);
        if (tid == 0 && side == 0 && h == 0) {
            reinterpret_cast<int32_t*>(c.base + c.lay.table)[((size_t)e.seq * c.num_layers + c.layer) * c.max_blocks +
                                                             first + j] = slot;
        }
        if (c8 == 0 && tok == 0) {
            float* hd = reinterpret_cast<float*>(t);
            if (side == 0) {
                hd[0] = s;
            } else {
                hd[1] = s;
                hd[2] = amax == 0.f ? (float)kZeroV : log2f(s);
                hd[3] = (amax == 0.f ? power2(-kZeroV) : inv) * kDenomUnit;
            }
        }
        uint2 q[8];  // codes of token u, channel by channel
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            uint32_t o[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const float2 a = unpack2<BF16>(w[2 * z]), b = unpack2<BF16>(w[2 * z + 1]);
                if (!finite) {
                    o[z] = 0;
                } else if (c.int8) {
                    o[z] = int8x4(a.x, a.y, b.x, b.y, s, inv);
                } else {
                    o[z] = e4m3x4(a.x * inv, a.y * inv, b.x * inv, b.y * inv);
                }
            }
            q[u] = make_uint2(o[0], o[1]);
        }
        if (side == 0) {
#pragma unroll
            for (int u = 0; u < 8; ++u) *reinterpret_cast<uint2*>(t + k_code_off(d, tok + u, 8 * c8)) = q[u];
        } else {
            transpose4(q[0].x, q[1].x, q[2].x, q[3].x);
            transpose4(q[0].y, q[1].y, q[2].y, q[3].y);
            transpose4(q[4].x, q[5].x, q[6].x, q[7].x);
            transpose4(q[4].y, q[5].y, q[6].y, q[7].y);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                *reinterpret_cast<uint2*>(t + v_code_off(d, tok, 8 * c8 + z)) = make_uint2(q[z].x, q[4 + z].x);
                *reinterpret_cast<uint2*>(t + v_code_off(d, tok, 8 * c8 + 4 + z)) = make_uint2(q[z].y, q[4 + z].y);
            }
        }
    }
    if (on && j == 0) {  // the tokens behind the last completed block
        const int n1 = e.n_before + e.n_new;
        const int from = e.n_blocks > 0 ? (first + e.n_blocks) << lb : e.n_before;
        for (int z = tid; z < (n1 - from) * (d / 8); z += tpg) {
            const int pos = from + z / (d / 8), ch = 8 * (z % (d / 8));
            const uint4 w = *reinterpret_cast<const uint4*>(in + (e.in_row + (int64_t)(pos - e.n_before)) * stride +
                                                            h * d + ch);
            if (side == 0) {
                *reinterpret_cast<uint4*>(tail + (size_t)(pos & (bt - 1)) * d + ch) = w;
            } else {
                const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int y = 0; y < 8; ++y)
                    tail[tail_v_off(d, pos & (bt - 1), ch + y)] = (uint16_t)(v[y >> 1] >> (16 * (y & 1)));
            }
        }
    }
}

template <class P>
int append_launch(const P& p, cudaStream_t s) {
    const int groups = kWriteThreads / (p.c.block * p.c.d / 64);
    const unsigned grid = (unsigned)((p.items + groups - 1) / groups);
    if (p.c.d == 128) {
        if (p.c.bf16) append_kernel<128, true><<<grid, kWriteThreads, 0, s>>>(p);
        else append_kernel<128, false><<<grid, kWriteThreads, 0, s>>>(p);
    } else {
        if (p.c.bf16) append_kernel<64, true><<<grid, kWriteThreads, 0, s>>>(p);
        else append_kernel<64, false><<<grid, kWriteThreads, 0, s>>>(p);
    }
    return (int)cudaGetLastError();
}

// Reading back: a group of D / 2 threads per (sequence, tile, K or V, KV head); a thread takes
// 8 tokens x 8 channels (V codes turned in its registers) and writes 16 bytes a token (32 in
// fp32). Sealed values are code * s in fp32, rounded once; a finite value beyond the type's
// range becomes its largest. Bound by memory.
template <int D, bool BF16, bool INT8, bool F32>
__global__ void __launch_bounds__(kWriteThreads) read_kernel(const __grid_constant__ BlockReadParams p) {
    const BlockView& c = p.c;
    constexpr int d = D, tpg = D / 2;
    const int64_t item64 = (int64_t)blockIdx.x * (kWriteThreads / tpg) + threadIdx.x / tpg;
    if (item64 >= p.items) return;
    const int item = (int)item64;
    const int tid = threadIdx.x % tpg;
    int lo = 0;
    for (int hi = p.n_seqs - 1; lo < hi;) {
        const int mid = (lo + hi + 1) / 2;
        if (p.seqs[mid].item_begin <= item) lo = mid; else hi = mid - 1;
    }
    const BlockReadSeq& e = p.seqs[lo];
    const int rel = item - e.item_begin;
    const int h = rel % c.hkv, side = rel / c.hkv % 2, tile = e.start / kTileTokens + rel / (2 * c.hkv);
    const int c8 = tid % (d / 8), tok = tid / (d / 8) * 8;
    const int pos0 = tile * kTileTokens + tok;
    const int sealed = e.n & ~(c.block - 1);
    const int end = e.start + e.count;
    if (pos0 >= end || pos0 + 8 <= e.start) return;
    uint8_t* out = reinterpret_cast<uint8_t*>(side ? p.v : p.k);
    const size_t row = (size_t)c.hkv * d, at = (size_t)h * d + 8 * c8;
    if (tile * kTileTokens < sealed) {  // sealed is a multiple of 32
        const uint8_t* t = sealed_tile(c, block_table(c, e.seq), h, tile);
        const float s = reinterpret_cast<const float*>(t)[side];
        uint2 q[8];
        if (side == 0) {
#pragma unroll
            for (int u = 0; u < 8; ++u) q[u] = __ldcs(reinterpret_cast<const uint2*>(t + k_code_off(d, tok + u, 8 * c8)));
        } else {
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const uint2 a = __ldcs(reinterpret_cast<const uint2*>(t + v_code_off(d, tok, 8 * c8 + z)));
                const uint2 b = __ldcs(reinterpret_cast<const uint2*>(t + v_code_off(d, tok, 8 * c8 + 4 + z)));
                q[z].x = a.x, q[4 + z].x = a.y, q[z].y = b.x, q[4 + z].y = b.y;
            }
            transpose4(q[0].x, q[1].x, q[2].x, q[3].x);
            transpose4(q[0].y, q[1].y, q[2].y, q[3].y);
            transpose4(q[4].x, q[5].x, q[6].x, q[7].x);
            transpose4(q[4].y, q[5].y, q[6].y, q[7].y);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int pos = pos0 + u;
            if (pos < e.start || pos >= end) continue;
            const uint32_t w[4] = {codes_lo<INT8>(q[u].x), codes_hi<INT8>(q[u].x), codes_lo<INT8>(q[u].y),
                                   codes_hi<INT8>(q[u].y)};
            float f[8];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const float2 g = unpack2<false>(w[z]);
                f[2 * z] = g.x * s, f[2 * z + 1] = g.y * s;
            }
            const size_t o = ((size_t)e.out_row + (pos - e.start)) * row + at;
            if constexpr (F32) {
                float4* dst = reinterpret_cast<float4*>(out + o * 4);
                __stcs(dst, make_float4(f[0], f[1], f[2], f[3]));
                __stcs(dst + 1, make_float4(f[4], f[5], f[6], f[7]));
            } else {
                constexpr float most = BF16 ? 3.3895313892515355e38f : 65504.f;
                uint32_t r[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    float a = f[2 * z], b = f[2 * z + 1];
                    a = a > most ? most : a < -most ? -most : a;  // NaN passes
                    b = b > most ? most : b < -most ? -most : b;
                    r[z] = pack2<BF16>(a, b);
                }
                __stcs(reinterpret_cast<uint4*>(out + o * 2), make_uint4(r[0], r[1], r[2], r[3]));
            }
        }
    } else {
        const uint16_t* tail = tail_ptr(c, side ? c.lay.tail_v : c.lay.tail_k, e.seq, h);
        for (int u = 0; u < 8; ++u) {
            const int pos = pos0 + u;
            if (pos < e.start || pos >= end) continue;
            uint4 w;
            if (side == 0) {
                w = *reinterpret_cast<const uint4*>(tail + (size_t)(pos - sealed) * d + 8 * c8);
            } else {
                uint32_t v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = (uint32_t)tail[tail_v_off(d, pos - sealed, 8 * c8 + 2 * q)] |
                           ((uint32_t)tail[tail_v_off(d, pos - sealed, 8 * c8 + 2 * q + 1)] << 16);
                w = make_uint4(v[0], v[1], v[2], v[3]);
            }
            const size_t o = ((size_t)e.out_row + (pos - e.start)) * row + at;
            if constexpr (F32) {
                const float2 a = unpack2<BF16>(w.x), b = unpack2<BF16>(w.y), g = unpack2<BF16>(w.z), k = unpack2<BF16>(w.w);
                float4* dst = reinterpret_cast<float4*>(out + o * 4);
                dst[0] = make_float4(a.x, a.y, b.x, b.y);
                dst[1] = make_float4(g.x, g.y, k.x, k.y);
            } else {
                *reinterpret_cast<uint4*>(out + o * 2) = w;
            }
        }
    }
}

template <int D, bool BF16, bool INT8>
int read_launch(const BlockReadParams& p, cudaStream_t s) {
    constexpr int groups = kWriteThreads / (D / 2);
    const unsigned grid = (unsigned)(((int64_t)p.items + groups - 1) / groups);
    if (p.f32) read_kernel<D, BF16, INT8, true><<<grid, kWriteThreads, 0, s>>>(p);
    else read_kernel<D, BF16, INT8, false><<<grid, kWriteThreads, 0, s>>>(p);
    return (int)cudaGetLastError();
}

template <int D>
int read_launch_dim(const BlockReadParams& p, cudaStream_t s) {
    if (p.c.bf16) return p.c.int8 ? read_launch<D, true, true>(p, s) : read_launch<D, true, false>(p, s);
    return p.c.int8 ? read_launch<D, false, true>(p, s) : read_launch<D, false, false>(p, s);
}

}  // namespace

int launch_block_append(const BlockAppendSmall& p, void* stream) { return append_launch(p, (cudaStream_t)stream); }
int launch_block_append(const BlockAppendLarge& p, void* stream) { return append_launch(p, (cudaStream_t)stream); }

int launch_block_read(const BlockReadParams& p, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    return p.c.d == 128 ? read_launch_dim<128>(p, s) : read_launch_dim<64>(p, s);
}

int launch_block_init(const BlockView& c, void* stream) {
    // error word, block table and the split counters
    return (int)cudaMemsetAsync(c.base + c.lay.err, 0, c.lay.partials - c.lay.err, (cudaStream_t)stream);
}

int launch_block_clear_errors(const BlockView& c, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = cudaMemsetAsync(c.base + c.lay.err, 0, 16, s);
    return (int)(e != cudaSuccess ? e : cudaMemsetAsync(c.base + c.lay.counters, 0, kBlockMaxGrid * 4, s));
}

int stream_capturing(void* stream, int* capturing) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    const cudaError_t e = cudaStreamIsCapturing((cudaStream_t)stream, &st);
    *capturing = st != cudaStreamCaptureStatusNone;
    return (int)e;
}

}  // namespace kvarn
