// Pieces of the block cache's tcgen05 kernels: operand tiles in shared memory, MMA issue, and the exact tokens of a
// 32-token part as tile rows.
#pragma once
#include "kvarn_block_dev.cuh"
#include "kvarn_tc.cuh"

namespace kvarn {

constexpr int kAtom = 128 * 128;  // bytes of 128 rows of 64 f16

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
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
    return ok != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float max32(const uint32_t (&r)[32]) {
    float a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
#pragma unroll
    for (int k = 2; k < 30; k += 4) {
        a = max3(a, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
        b = max3(b, __uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]));
    }
    return fmaxf(max3(a, __uint_as_float(r[30]), __uint_as_float(r[31])), b);
}

// Exact tokens of a part (none: zeros) as its K or V tile rows. A later token's infinity or NaN
// must not reach a query that does not see it through 0 x NaN: non-finite V enters as 0, and `bad`
// says that there is some, for add_non_finite at the segment's end. K needs no such care (logits
// of unseen tokens are replaced), but neither may set the part's power of two.
// h: K scale, or log2 of the V scale and kDenomUnit over it. x: registers to use.
template <int D, bool BF16, bool IS_V>
__device__ __forceinline__ void expand_exact(const BlockView& c, int seq, int n, int kvh, int tile, int wp, int lane,
                                             uint8_t* dst, float2& h, uint32_t& bad, uint4 (&x)[D / 16]) {
    const int g = lane >> 2, t = lane & 3;
    const int first = (tile - (n >> c.log2_block << (c.log2_block - 5))) * kTileTokens;  // row of the tail
    const int nv = min(kTileTokens, n - tile * kTileTokens);  // valid tokens, none if <= 0
    h = IS_V ? make_float2(0.f, 1.f) : make_float2(1.f, 0.f);
    bad = 0;
    // D / 8 pieces of 16 bytes a lane, four at a time so that their loads overlap; twice, first for the largest
    constexpr int kTurn = 4;
    if (IS_V) {  // piece i: tokens 8 t .. of channel 8 i + g
        const uint16_t* v = tail_ptr(c, c.lay.tail_v, seq, kvh) + (ptrdiff_t)first * D;
        uint32_t keep[4];
#pragma unroll
        for (int z = 0; z < 4; ++z)
            keep[z] = (8 * t + 2 * z < nv ? 0xffffu : 0u) | (8 * t + 2 * z + 1 < nv ? 0xffff0000u : 0u);
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                x[i] = make_uint4(0, 0, 0, 0);
                if (nv > 0) x[i] = *reinterpret_cast<const uint4*>(v + (8 * (i0 + i) + g) * kTileTokens + 8 * t);
            }
#pragma unroll
            for (int i = 0; i < kTurn; ++i)
                x[i] = make_uint4(x[i].x & keep[0], x[i].y & keep[1], x[i].z & keep[2], x[i].w & keep[3]);
        };
        uint32_t top = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < D / 8; i0 += kTurn) {
            load(i0);
#pragma unroll
            for (int i = 0; i < kTurn; ++i) top = max_of(top, finite_only<BF16>(x[i]));
        }
        const int ex = warp_exponent_v<BF16>(top);
        const float f = power2(-ex);
        h = make_float2((float)ex, f * kDenomUnit);
        uint8_t* atom = dst + (wp >> 1) * (D * 128);
#pragma unroll 1
        for (int i0 = 0; i0 < D / 8; i0 += kTurn) {
            load(i0);
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                const uint4 r = x[i];
                bad |= bad_pair<BF16>(r.x) | bad_pair<BF16>(r.y) | bad_pair<BF16>(r.z) | bad_pair<BF16>(r.w);
                *reinterpret_cast<uint4*>(atom + swz(8 * (i0 + i) + g, 4 * (wp & 1) + t)) =
                    scaled_f16<BF16>(finite_only<BF16>(r), f);
            }
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
    } else {  // piece i: bytes i * 512 + lane * 16 of the part's 32 D values
        const uint16_t* k = tail_ptr(c, c.lay.tail_k, seq, kvh) + (ptrdiff_t)first * D;
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                const int y = (i0 + i) * 32 + lane;
                x[i] = make_uint4(0, 0, 0, 0);
                if (y / (D / 8) < nv) x[i] = *reinterpret_cast<const uint4*>(k + y * 8);
            }
        };
        float f = 1.f;
        if (BF16) {
            uint32_t top = 0;
#pragma unroll 1
            for (int i0 = 0; i0 < D / 8; i0 += kTurn) {
                load(i0);
#pragma unroll
                for (int i = 0; i < kTurn; ++i) top = max_of(top, finite_only<BF16>(x[i]));
            }
            const int ex = warp_exponent<BF16>(top) - kExactK;
            f = power2(-ex);
            h.x = power2(ex);
        }
#pragma unroll 1
        for (int i0 = 0; i0 < D / 8; i0 += kTurn) {
            load(i0);
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                const int y = (i0 + i) * 32 + lane, ch8 = y % (D / 8);
                *reinterpret_cast<uint4*>(dst + (ch8 >> 3) * kAtom + swz(32 * wp + y / (D / 8), ch8 & 7)) =
                    BF16 ? scaled_f16<BF16>(x[i], f) : x[i];
            }
        }
    }
}

}  // namespace kvarn
