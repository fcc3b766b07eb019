// Device helpers of the block cache: addresses, 8-bit codes, packed 16-bit values.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kvarn_block.h"
#include "kvarn_dev.cuh"

namespace kvarn {

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
