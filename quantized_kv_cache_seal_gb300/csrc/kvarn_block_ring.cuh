// Roles that the block cache's row-tile kernels share (window_kernel, flat_kernel): their way along a line of steps, query
// rows as operand tiles, and the expansion of codes that come through rings of bulk copies.
#pragma once
#include "kvarn_block_tc.cuh"

namespace kvarn {

// The segments (a tile of 128 rows of a (sequence, KV head), steps j0 .. j1 - 1 of 128 tokens) of a CTA's part of the line.
template <class P>
struct RowWalk {
    const P& p;
    int64_t u, u1;
    int i, h, tile, j0, j1, pair;
    __device__ __forceinline__ RowWalk& operator=(const RowWalk& o) {  // (of the same p)
        u = o.u, u1 = o.u1, i = o.i, h = o.h, tile = o.tile, j0 = o.j0, j1 = o.j1, pair = o.pair;
        return *this;
    }
    __device__ __forceinline__ explicit RowWalk(const P& p_)
        : p(p_), u(p_.units * blockIdx.x / p_.grid), u1(p_.units * (blockIdx.x + 1) / p_.grid), i(0), j0(0), j1(0) {}
    __device__ __forceinline__ bool next() {
        if (u >= u1) return false;
#pragma unroll 1
        while (i + 1 < p.n_seqs && p.seqs[i + 1].unit_begin <= u) ++i;
        const auto& e = p.seqs[i];
        const int rel = (int)u - e.unit_begin;
        pair = rel / e.steps;
        j0 = rel - pair * e.steps;
        j1 = (int)min((int64_t)e.steps, j0 + (u1 - u));
        h = pair / e.row_tiles;
        tile = pair - h * e.row_tiles;
        u += j1 - j0;
        return true;
    }
};

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// WARPS warps write a segment's rows as its Q tile (K-major, 128-byte swizzle) and the exponents of the powers of two that they
// stand for; warp w of them. All of a warp's rows are on their way together; bf16 values and a scale below 0 (which turns
// the query's sign, so that larger S is always a larger logit) take a second look. A scale of 0 makes the queries zeros: all
// logits are 0.
template <int D, int WARPS>
struct Rows {
    static constexpr int kLanes = D / 8, kRows = 32 / kLanes, kTurns = 128 / kRows / WARPS;
    uint8_t* dst;
    int first, lane;
    __device__ __forceinline__ Rows(uint8_t* dst_, int w, int lane_)
        : dst(dst_), first(w * (128 / WARPS) + lane_ / kLanes), lane(lane_) {}
    __device__ __forceinline__ uint8_t* at(int z) const { return dst + (lane % kLanes >> 3) * kAtom + swz(first + z * kRows, lane & 7); }
    template <class P>
    __device__ __forceinline__ void fetch(const P& p, const RowWalk<P>& s) const {
        const auto& e = p.seqs[s.i];
        const int tok0 = s.tile * 128 / p.r, in0 = s.tile * 128 - tok0 * p.r, inv = 65536 / p.r + 1;
        const uint4* q = reinterpret_cast<const uint4*>(p.q + ((size_t)(e.q_row + tok0) * p.hq + s.h * p.r) * D) + lane % kLanes;
#pragma unroll 4
        for (int z = 0; z < kTurns; ++z) {
            const int row = first + z * kRows, in = in0 + row, tok = in * inv >> 16;  // in / r: in < 136, r <= 8
            if (s.tile * 128 + row < e.rows && p.scale_log2 != 0.f)
                cp_async_16(at(z), q + ((size_t)tok * p.hq + in - tok * p.r) * kLanes);
            else
                *reinterpret_cast<uint4*>(at(z)) = make_uint4(0, 0, 0, 0);
        }
    }
    template <bool BF16>
    __device__ __forceinline__ void finish(float scale_log2, int8_t* power) const {
        const uint32_t sign = scale_log2 < 0.f ? 0x80008000u : 0u;
        cp_async_wait_all();
#pragma unroll 4
        for (int z = 0; z < kTurns; ++z) {
            int ex = 0;  // -114 to 113
            if (BF16 || sign) {
                uint4 r = *reinterpret_cast<const uint4*>(at(z));
                if (BF16) {
                    uint32_t top = max_of(0, r);
                    top = max(top & 0xffffu, top >> 16);
#pragma unroll
                    for (int d = kLanes / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                    ex = exponent_of<BF16>(top) - kExactK;
                    r = scaled_f16<BF16>(r, power2(-ex));
                }
                *reinterpret_cast<uint4*>(at(z)) = make_uint4(r.x ^ sign, r.y ^ sign, r.z ^ sign, r.w ^ sign);
            }
            if (lane % kLanes == 0) power[first + z * kRows] = (int8_t)ex;
        }
        fence_proxy_async_smem();
    }
};

// What a row's S is multiplied with, beside K's scale, for its logits.
__device__ __forceinline__ float row_factor(float scale_log2, int power) {
    return (scale_log2 == 0.f ? 1.f : fabsf(scale_log2)) * power2(power);
}

template <int D>
constexpr int kRingEntry = 16 + kTileTokens * D;  // scales and codes of one side of a tile; two hold an exact part

// Codes of a part as rows 32 wp .. of a K tile, or columns of a V tile.
template <int D, bool INT8, bool IS_V>
__device__ __forceinline__ void expand_codes(const uint8_t* rec, uint8_t* dst, int wp, int lane) {
    auto halves = [&](uint32_t u, uint32_t v) {
        return make_uint4(codes_lo<INT8>(u), codes_hi<INT8>(u), codes_lo<INT8>(v), codes_hi<INT8>(v));
    };
    const int t = lane & 3;
    if (IS_V) {  // lanes take the chunks in an order in which the stores of eight meet eight different banks
        const int g = (lane >> 3) + (lane & 4);
        uint8_t* to = dst + (wp >> 1) * (D * 128) + swz(g, 4 * (wp & 1) + t);
#pragma unroll 2
        for (int i = 0; i < D / 16; ++i) {  // 8 tokens of channels 16 i + g and + 8
            const uint4 x = *reinterpret_cast<const uint4*>(rec + 16 + i * 512 + (4 * g + t) * 16);
            *reinterpret_cast<uint4*>(to + i * 2048) = halves(x.x, x.y);
            *reinterpret_cast<uint4*>(to + i * 2048 + 1024) = halves(x.z, x.w);
        }
    } else {
        const int g = lane >> 2, row0 = 32 * wp + 8 * (g >> 1) + (g & 1);
        // 16 channels of one token: chunk i holds token 4 (i / (D / 32)) + 2 (i & 1), channels 64 (i / 2 % (D / 64)) on. The row's place in
        // its group of eight turns the 16-byte chunks' places by an exclusive or.
#pragma unroll 2
        for (int i = 0; i < D / 16; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(rec + 16 + i * 512 + lane * 16);
            const int row = row0 + 4 * (i / (D / 32)) + 2 * (i & 1);
            uint8_t* to = dst + i / 2 % (D / 64) * kAtom + row * 128;
            const int at = (2 * t) ^ (row & 7);
            *reinterpret_cast<uint4*>(to + (at << 4)) = halves(x.x, x.y);
            *reinterpret_cast<uint4*>(to + ((at ^ 1) << 4)) = halves(x.z, x.w);
        }
    }
}

// 16 bytes of exact tokens (nv of them; none: zeros, and `src` is not read): of V tokens 8 t .. of channel 8 i + g, of K
// bytes i * 512 + lane * 16 of the part's rows.
template <int D, bool IS_V>
__device__ __forceinline__ uint4 exact_piece(const uint8_t* src, int nv, int i, int lane) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (IS_V) {
        const int g = lane >> 2, t = lane & 3;
        if (8 * t < nv) x = *reinterpret_cast<const uint4*>(src + (8 * i + g) * 64 + 16 * t);
        const int left = nv - 8 * t;
        uint32_t keep[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) keep[z] = (2 * z < left ? 0xffffu : 0u) | (2 * z + 1 < left ? 0xffff0000u : 0u);
        return make_uint4(x.x & keep[0], x.y & keep[1], x.z & keep[2], x.w & keep[3]);
    }
    if ((i * 32 + lane) / (D / 8) < nv) x = *reinterpret_cast<const uint4*>(src + (i * 32 + lane) * 16);
    return x;
}
// What a part of exact tokens stands for: K's scale, or log2 of V's and kDenomUnit over it; `bad`: non-finite V, which enters as
// 0. Neither side's non-finite values set the power of two.
template <int D, bool BF16, bool IS_V>
__device__ __forceinline__ float2 exact_head(const uint8_t* src, int nv, int lane, uint32_t& bad) {
    bad = 0;
    if (!IS_V && !BF16) return make_float2(1.f, 0.f);
    uint32_t top = 0;
#pragma unroll 2
    for (int i = 0; i < D / 8; ++i) {
        const uint4 r = exact_piece<D, IS_V>(src, nv, i, lane);
        top = max_of(top, finite_only<BF16>(r));
        if (IS_V) bad |= bad_pair<BF16>(r.x) | bad_pair<BF16>(r.y) | bad_pair<BF16>(r.z) | bad_pair<BF16>(r.w);
    }
    if (!IS_V) return make_float2(power2(warp_exponent<BF16>(top) - kExactK), 0.f);
    bad = __reduce_or_sync(0xffffffffu, bad);
    const int ex = warp_exponent_v<BF16>(top);
    return make_float2((float)ex, power2(-ex) * kDenomUnit);
}
// The tokens as rows of a K tile, or columns of a V tile. h: exact_head's.
template <int D, bool BF16, bool IS_V>
__device__ __forceinline__ void expand_rows(const uint8_t* src, int nv, uint8_t* dst, int wp, int lane, float2 h) {
    const float f = IS_V ? power2(-(int)h.x) : 1.f / h.x;
#pragma unroll 2
    for (int i = 0; i < D / 8; ++i) {
        const uint4 r = exact_piece<D, IS_V>(src, nv, i, lane);
        if (IS_V) {
            uint8_t* atom = dst + (wp >> 1) * (D * 128);
            *reinterpret_cast<uint4*>(atom + swz(8 * i + (lane >> 2), 4 * (wp & 1) + (lane & 3))) =
                scaled_f16<BF16>(finite_only<BF16>(r), f);
        } else {
            const int y = i * 32 + lane, ch8 = y % (D / 8);
            *reinterpret_cast<uint4*>(dst + (ch8 >> 3) * kAtom + swz(32 * wp + y / (D / 8), ch8 & 7)) =
                BF16 ? scaled_f16<BF16>(r, f) : r;
        }
    }
}

// Eight rings of two entries each, one of every expansion warp x: part x & 3 (32 tokens) of every step, K for x < 4 and V
// for the others (SIDES), or K of every other step, the odd ones for x >= 4. The four rings of such a group go in step: turn t is entry
// t & 1 of each. An exact part takes both entries, so a turn with one waits for the turn before to be through, and the turn
// behind it for it.
template <int D>
struct Rings {
    static constexpr int kCount = 8;
    static constexpr int kBytes = kCount * 2 * kRingEntry<D>;
    uint8_t* data;     // [kCount][2][kRingEntry]
    uint64_t* full;    // barriers [kCount][2]
    uint64_t* empty;   // barriers [2 groups][2]
    int32_t* what;     // [kCount][2]: kCodes, or exact tokens, none if 0
    static constexpr int kCodes = -1;
};

// A warp fills a group's rings, a lane each (the way along the line is the same for all, and costs an expansion warp as much as the
// conversion). Pool slots are looked up a turn earlier. (Expansion warps that did it themselves took twice as long for a part: 76 us for
// two prefixes of 32k where it is 60 this way.)
template <int D, bool SIDES, class P>
__device__ __forceinline__ void fill_rings(const P& p, const Rings<D>& rings, int group, int steps, int32_t* err, int lane) {
    const BlockView& c = p.c;
    const int sh = c.log2_block - 5, wp = lane & 3, x = 4 * group + wp;
    const bool v = SIDES && group == 1;
    uint64_t* empty = rings.empty + 2 * group;
    uint8_t* data = rings.data + x * 2 * kRingEntry<D>;
    uint64_t* full = rings.full + 2 * x;
    volatile int32_t* what = rings.what + 2 * x;
    struct Part {
        int seq, n, kvh, tile, slot;  // seq -1: no more; slot -1: exact tokens, or none
    };
    RowWalk<P> w(p);
    bool more = w.next();
    int j = w.j0;
    auto skip = [&]() {
        if (more && ++j == w.j1) {
            more = w.next();
            if (more) j = w.j0;
        }
    };
    if (!SIDES && group == 1) skip();
    auto look = [&]() {
        Part a = {-1, 0, 0, 0, -1};
        if (!more) return a;
        const auto& e = p.seqs[w.i];
        a = Part{e.seq, e.n, w.h, 4 * j + wp, -1};
        if (!SIDES && e.pre_n > 0) {
            const int before = (e.pre_n + 127) / 128;
            if (j < before) a.seq = e.pre, a.n = e.pre_n;
            else a.tile -= 4 * before;
        }
        if (a.tile < a.n >> c.log2_block << sh) a.slot = read<true>(block_table(c, a.seq) + (a.tile >> sh));
        skip();
        if (!SIDES) skip();
        return a;
    };
    const int turns = SIDES ? steps : (steps + 1 - group) / 2;
    bool ok = true, alone = false;  // alone: the turn before has the rings for itself
    Part now = look(), next = look();
    int t = 0;
#pragma unroll 1
    for (; t < turns; ++t) {
        const int y = t & 1, exact = now.slot < 0 && now.seq >= 0 ? max(now.n - now.tile * kTileTokens, 0) : 0;
        const bool was = alone;
        alone = __any_sync(0xffffffffu, exact > 0);
        bool here = t < 2 || bar_wait(empty + y, (uint32_t)(((t >> 1) - 1) & 1), err);
        if (t > 0 && (was || alone)) here = bar_wait(empty + (y ^ 1), (uint32_t)(((t - 1) >> 1) & 1), err) && here;
        ok = __all_sync(0xffffffffu, here);
        if (!ok) break;
        if (lane < 4) {
            if (now.slot >= 0) {
                const uint8_t* rec = tile_ptr(c, now.slot, now.kvh, now.tile & ((1 << sh) - 1));
                uint8_t* to = data + y * kRingEntry<D>;
                what[y] = Rings<D>::kCodes;
                mbar_arrive_expect_tx(full + y, kRingEntry<D>);
                // scales, and K's codes behind them, or V's
                bulk_g2s(to, rec, 16, full + y);
                bulk_g2s(to + 16, rec + 16 + (v ? kTileTokens * D : 0), kTileTokens * D, full + y);
            } else if (exact) {
                constexpr int kBytes = kTileTokens * D * 2;
                static_assert(kBytes <= 2 * kRingEntry<D>, "room for an exact part");
                what[y] = min(exact, kTileTokens);
                mbar_arrive_expect_tx(full + y, kBytes);
                bulk_g2s(data, tail_ptr(c, v ? c.lay.tail_v : c.lay.tail_k, now.seq, now.kvh) +
                                   (size_t)(now.tile - (now.n >> c.log2_block << sh)) * (kTileTokens * D), kBytes, full + y);
            } else {
                what[y] = 0;
                mbar_arrive(full + y);
            }
        }
        __syncwarp();
        now = next;
        next = look();
    }
    // What is in flight lands (which a wait that gave up did not see to) before the CTA's shared memory goes away.
    const uint64_t t0 = global_ns();
#pragma unroll 1
    for (int z = max(t - 2, 0); z < t; ++z)
        while (!mbar_try_wait(full + (z & 1), (uint32_t)(z >> 1 & 1)) && global_ns() - t0 < kWaitLimitNs) {
        }
}

// Expansion warp x: its part of steps first, first + STRIDE .. of the CTA's `steps`. head(step, h, bad): what the part stands for, known
// before there is a place for it; place(step): the tile to write, once it is free; publish(step): the tile is there.
template <int D, bool INT8, bool BF16, bool IS_V, int STRIDE, class Head, class Place, class Publish>
__device__ __forceinline__ void expand_steps(const Rings<D>& rings, int x, int first, int steps, int32_t* err, int lane, Head head,
                                             Place place, Publish publish) {
    const uint8_t* data = rings.data + x * 2 * kRingEntry<D>;
    const volatile int32_t* what = rings.what + 2 * x;
    int t = 0;
#pragma unroll 1
    for (int k = first; k < steps; k += STRIDE, ++t) {
        const int y = t & 1;
        bar_wait(rings.full + 2 * x + y, (uint32_t)(t >> 1 & 1), err);
        const int is = __shfl_sync(0xffffffffu, what[y], 0);  // one answer for the warp, also after a wait that gave up
        const uint8_t* rec = data + y * kRingEntry<D>;
        float2 h;
        uint32_t bad = 0;
        if (is < 0) {
            const float4 hd = *reinterpret_cast<const float4*>(rec);
            h = IS_V ? make_float2(hd.z, hd.w) : make_float2(hd.x, 0.f);
        } else {
            h = exact_head<D, BF16, IS_V>(data, is, lane, bad);
        }
        head(k, h, bad);
        uint8_t* dst = place(k);
        if (is < 0) expand_codes<D, INT8, IS_V>(rec, dst, x & 3, lane);
        else expand_rows<D, BF16, IS_V>(data, is, dst, x & 3, lane, h);
        __syncwarp();
        if (lane == 0) mbar_arrive(rings.empty + (x >> 2) * 2 + y);
        fence_proxy_async_smem();
        publish(k);
    }
}

}  // namespace kvarn
