// Device helpers of the block cache: addresses, 8-bit codes, packed 16-bit values.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>

#include "kvarn_block.h"
#include "kvarn_dev.cuh"

namespace kvarn {

// A runtime call's error, which is reported here and no longer stands in the runtime for the next launch to find.
inline int taken(cudaError_t e) {
    if (e != cudaSuccess) (void)cudaGetLastError();
    return (int)e;
}

// A kernel's dynamic shared memory limit, raised once on each device (the attribute is the device's).
struct SmemOnce {
    std::atomic<uint64_t> done{0};
    int allow(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        const uint64_t bit = 1ull << (dev & 63);
        if (e != cudaSuccess || (dev < 64 && (done.load() & bit))) return taken(e);
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && dev < 64) done.fetch_or(bit);
        return taken(e);
    }
};

// A launch that may begin while the stream's kernel before it still runs: its thread blocks take the SMs as they get free and wait
// (before_done) ahead of their first access to global memory, for the other to be complete and seen. All threads of all
// thread blocks call it, so that a kernel behind finds every kernel before complete as well. start_next: from here on the next
// kernel's thread blocks may come. What a kernel before may have written is read by plain loads (read<true>), since it is not
// read-only for as long as this one runs.
__device__ __forceinline__ void before_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <bool BEHIND, class T>
__device__ __forceinline__ T read(const T* p) {
    return BEHIND ? *p : __ldg(p);
}
template <class... Args>
int launch_behind(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s, const Args&... args) {
    cudaLaunchAttribute early = {};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = s;
    config.attrs = &early;
    config.numAttrs = 1;
    return taken(cudaLaunchKernelEx(&config, kernel, args...));
}

__device__ __forceinline__ const int32_t* block_table(const BlockView& c, int seq) {
    return reinterpret_cast<const int32_t*>(c.base + c.lay.table) + ((size_t)seq * c.num_layers + c.layer) * c.max_blocks;
}
// tile `tile` of the sequence for KV head h; the host hands out slots, so an entry of a sealed block is in range
__device__ __forceinline__ uint8_t* tile_ptr(const BlockView& c, int slot, int h, int tile_in_block) {
    return c.base + c.lay.pool + (size_t)slot * c.slot_bytes +
           (size_t)(h * (c.block / kTileTokens) + tile_in_block) * tile_bytes(c.d);
}
__device__ __forceinline__ const uint8_t* sealed_tile(const BlockView& c, const int32_t* table, int h, int tile) {
    const int sh = c.log2_block - 5;
    return tile_ptr(c, __ldg(table + (tile >> sh)), h, tile & ((1 << sh) - 1));
}
__device__ __forceinline__ uint16_t* tail_ptr(const BlockView& c, size_t region, int seq, int h) {
    return reinterpret_cast<uint16_t*>(c.base + region) +
           (((size_t)seq * c.num_layers + c.layer) * c.hkv + h) * ((size_t)c.block * c.d);
}

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

// Two codes (low 16 bits of w) as two f16, exact. e4m3: one conversion. int8 held as value +
// 128: the byte under 0x64 is 1024 + byte, and 1152 is taken off.
template <bool INT8>
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
    uint32_t r;
    if constexpr (INT8) {
        r = __byte_perm(w, 0x64646464u, 0x4140);
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&r), __half2half2(__ushort_as_half(0x6480)));
        r = *reinterpret_cast<const uint32_t*>(&h);
    } else {
        asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(w));
    }
    return r;
}
template <bool INT8>
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
    uint32_t r;
    if constexpr (INT8) {
        r = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&r), __half2half2(__ushort_as_half(0x6480)));
        r = *reinterpret_cast<const uint32_t*>(&h);
    } else {
        asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(r) : "r"(w));
    }
    return r;
}

// mbar_wait with its loop kept rolled: an unrolled one costs 2 KB of code at every place, and the
// kernels here have to fit the instruction cache.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, int32_t* err) {
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
    if (*reinterpret_cast<volatile int32_t*>(err) & kErrTimeout) return false;
    const uint64_t t0 = global_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (global_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, kErrTimeout);
            return false;
        }
    }
    return true;
}

// Exact 16-bit values enter the tensor cores as f16 after an exact power of two for 32 tokens or a
// row. Exponent e (-100 at least) of the largest absolute value `top` (a 16-bit pattern without sign):
// values times 2^(k - e) stay under 2^(k + 1).
template <bool BF16>
__device__ __forceinline__ int exponent_of(uint32_t top) {
    return max((int)(__float_as_uint(unpack2<BF16>(top).x) >> 23) - 127, -100);
}
__device__ __forceinline__ float power2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
template <bool BF16>
__device__ __forceinline__ uint32_t scaled_f16(uint32_t w, float f) {
    const float2 a = unpack2<BF16>(w);
    return pack2<false>(a.x * f, a.y * f);
}
template <bool BF16>
__device__ __forceinline__ uint4 scaled_f16(uint4 w, float f) {
    return make_uint4(scaled_f16<BF16>(w.x, f), scaled_f16<BF16>(w.y, f), scaled_f16<BF16>(w.z, f), scaled_f16<BF16>(w.w, f));
}
__device__ __forceinline__ uint32_t max_of(uint32_t top, uint4 x) {  // of two halves each, without sign
    top = __vmaxu2(top, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu));
    return __vmaxu2(top, __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
}
template <bool BF16>
__device__ __forceinline__ int warp_exponent(uint32_t top) {
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    return exponent_of<BF16>(top);
}
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

// Exact V values are brought to this power of two: near the largest codes (127, 448), so that the
// weights, which carry V's scale, use f16's range alike for sealed and exact tokens.
constexpr int kExactV = 8;
// Exact K values and bf16 queries, whose products only go into fp32 sums, to the top of f16's range.
constexpr int kExactK = 14;
// A V of nothing but zeros has no scale of its own, yet its weights (2^(x + log2 s), with 1 / s in the
// denominator) stand beside the others': with this one they do not set the running maximum, which would
// push the others out of f16, and do not leave fp32 in the denominator either, for other scales
// between 2^-60 and 2^50.
constexpr int kZeroV = -60;
// Denominators count w / s in units of 2^12, times this: with weights of 2^15 at most (2^7 at least for a row's
// largest) and scales from 2^-100 (exact values 2^-108) to 2^121, sums of up to 2^24 tokens and the least of them
// stay in fp32's normal range. Without it 32 exact tokens of 2^-100 already made an infinity.
constexpr float kDenomUnit = 1.f / 4096;
// Exponent of the power of two that stands for a part's V scale.
template <bool BF16>
__device__ __forceinline__ int warp_exponent_v(uint32_t top) {
    return __any_sync(0xffffffffu, top != 0) ? warp_exponent<BF16>(top) - kExactV : kZeroV;
}

#define kNegInf (-__int_as_float(0x7f800000))

// log2 of the sum of 2^logit over a row's keys, from its running maximum m and its denominator l (weights are
// 2^(x + log2 s_V - m + shift) and l adds weight kDenomUnit / s_V).
__device__ __forceinline__ float lse_of(float m, float l, float shift) {
    return l == 0.f ? kNegInf : log2f(l) + (m - shift + 12.f);
}
// The sum itself, as a maximum and a denominator with decode's shift of 15. No logarithm: one word of it would be rounded at
// the logits' size. (Denominators near fp32's end, of V scales near 2^-100, keep some powers of two in the maximum.)
__device__ __forceinline__ float2 total_of(float m, float l, float shift) {
    const int up = l > power2(100) ? 32 : 0;
    return make_float2(m + (float)up, l * power2(15 - (int)shift - up));
}
// A row over some keys and the row over others make the row over all of them: their shares, from the log2 of their
// sums; zeros where there are no keys on either side. NaN stays.
__device__ __forceinline__ float2 merge_factors(float a, float b) {
    const float top = fmaxf(a, b);
    if (top == kNegInf) return make_float2(0.f, 0.f);
    const float x = exp2f(a - top), y = exp2f(b - top), inv = 1.f / (x + y);
    return make_float2(x * inv, y * inv);
}
__device__ __forceinline__ float merge(float a, float b, float2 f) { return fmaf(a, f.x, b * f.y); }

// Sums as a maximum and what is over it, 2^x y: two of them as one. (With a maximum of -inf y is 0 or NaN.)
__device__ __forceinline__ float2 joined(float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x);
    float f, g;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(a.x - top));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(b.x - top));
    return make_float2(top, a.y * (a.x == kNegInf ? 1.f : f) + b.y * (b.x == kNegInf ? 1.f : g));
}

// Bytes of a 4 x 4 square: r[i] = row i; afterwards r[j] = column j.
__device__ __forceinline__ void transpose4(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    const uint32_t a = __byte_perm(r0, r1, 0x5140), b = __byte_perm(r0, r1, 0x7362);
    const uint32_t c = __byte_perm(r2, r3, 0x5140), d = __byte_perm(r2, r3, 0x7362);
    r0 = __byte_perm(a, c, 0x5410);
    r1 = __byte_perm(a, c, 0x7632);
    r2 = __byte_perm(b, d, 0x5410);
    r3 = __byte_perm(b, d, 0x7632);
}

}  // namespace kvarn
