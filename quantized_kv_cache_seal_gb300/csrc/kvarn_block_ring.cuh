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

// WARPS warps write a segment's rows as its Q tile (K-major, 128-byte swizzle) and the exponents of the powers of two
// that they stand for; warp w.
// All of a warp's rows are on their way together; bf16 values and a scale below 0 (which turns the query's sign, so
// that larger S is always a larger logit) take a second look. A scale of 0 makes the queries zeros: all logits are 0.
template <int D, bool BF16, int WARPS, class P>
__device__ __forceinline__ void make_rows(const P& p, const RowWalk<P>& s, uint8_t* dst, int8_t* power, int w, int lane) {
    const bool zero = p.scale_log2 == 0.f;
    const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kTurns = 128 / kRows / WARPS;
    const auto& e = p.seqs[s.i];
    const int first = w * (128 / WARPS) + lane / kLanes;
    auto at = [&](int z) { return dst + (lane % kLanes >> 3) * kAtom + swz(first + z * kRows, lane & 7); };
#pragma unroll 4
    for (int z = 0; z < kTurns; ++z) {
        const int all = s.tile * 128 + first + z * kRows;
        if (all < e.rows && !zero)
            cp_async_16(at(z), reinterpret_cast<const uint4*>(p.q + ((size_t)(e.q_row + all / p.r) * p.hq + s.h * p.r + all % p.r) * D) +
                                   lane % kLanes);
        else
            *reinterpret_cast<uint4*>(at(z)) = make_uint4(0, 0, 0, 0);
    }
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

// What a row's S is multiplied with, beside K's scale, for its logits.
__device__ __forceinline__ float row_factor(float scale_log2, int power) {
    return (scale_log2 == 0.f ? 1.f : fabsf(scale_log2)) * power2(power);
}

// A 32-token part of a step: of sequence `seq` with n tokens. step -1: none; slot -1: exact tokens, or none.
struct RowPart {
    int step, seq, n, kvh, tile, slot;
    __device__ __forceinline__ int exact() const { return slot < 0 ? n - tile * kTileTokens : 0; }  // tokens, none if <= 0
};

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

// Exact tokens (nv of them; none: zeros, and `src` is not read) as the same. Non-finite V enters as 0, and `bad` says that there is
// some; neither side's sets the part's power of two. h: K scale, or log2 of the V scale and kDenomUnit over it.
template <int D, bool BF16, bool IS_V>
__device__ __forceinline__ void expand_rows(const uint8_t* src, int nv, uint8_t* dst, int wp, int lane, float2& h, uint32_t& bad) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int kPieces = D / 8;
    h = IS_V ? make_float2(0.f, 1.f) : make_float2(1.f, 0.f);
    bad = 0;
    if (IS_V) {  // piece i: tokens 8 t .. of channel 8 i + g
        uint32_t keep[4];
#pragma unroll
        for (int z = 0; z < 4; ++z)
            keep[z] = (8 * t + 2 * z < nv ? 0xffffu : 0u) | (8 * t + 2 * z + 1 < nv ? 0xffff0000u : 0u);
        auto piece = [&](int i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (nv > 0) x = *reinterpret_cast<const uint4*>(src + (8 * i + g) * 64 + 16 * t);
            return make_uint4(x.x & keep[0], x.y & keep[1], x.z & keep[2], x.w & keep[3]);
        };
        uint32_t top = 0;
#pragma unroll 2
        for (int i = 0; i < kPieces; ++i) top = max_of(top, finite_only<BF16>(piece(i)));
        const int ex = warp_exponent_v<BF16>(top);
        const float f = power2(-ex);
        h = make_float2((float)ex, f * kDenomUnit);
        uint8_t* atom = dst + (wp >> 1) * (D * 128);
#pragma unroll 2
        for (int i = 0; i < kPieces; ++i) {
            const uint4 r = piece(i);
            bad |= bad_pair<BF16>(r.x) | bad_pair<BF16>(r.y) | bad_pair<BF16>(r.z) | bad_pair<BF16>(r.w);
            *reinterpret_cast<uint4*>(atom + swz(8 * i + g, 4 * (wp & 1) + t)) = scaled_f16<BF16>(finite_only<BF16>(r), f);
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
    } else {  // piece i: bytes i * 512 + lane * 16 of the part's rows
        auto piece = [&](int i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if ((i * 32 + lane) / kPieces < nv) x = *reinterpret_cast<const uint4*>(src + (i * 32 + lane) * 16);
            return x;
        };
        float f = 1.f;
        if (BF16) {
            uint32_t top = 0;
#pragma unroll 2
            for (int i = 0; i < kPieces; ++i) top = max_of(top, finite_only<BF16>(piece(i)));
            const int ex = warp_exponent<BF16>(top) - kExactK;
            f = power2(-ex);
            h.x = power2(ex);
        }
#pragma unroll 2
        for (int i = 0; i < kPieces; ++i) {
            const int y = i * 32 + lane, ch8 = y % kPieces;
            const uint4 x = piece(i);
            *reinterpret_cast<uint4*>(dst + (ch8 >> 3) * kAtom + swz(32 * wp + y / kPieces, ch8 & 7)) = BF16 ? scaled_f16<BF16>(x, f) : x;
        }
    }
}

// One expansion warp: part wp of every STRIDE-th step from `first` on, K or V. Codes come by bulk copies into a ring of the warp's own (two
// entries at `ring`, a barrier each), two parts ahead of the one that is expanded, pool slots a part earlier; an exact
// part takes both entries. place(step): the tile to write, once it is free (null: the wait gave up); publish(step, h, bad):
// the tile is there.
template <int D, bool INT8, bool BF16, bool IS_V, int STRIDE, class P, class Place, class Publish>
__device__ __forceinline__ void expand_line(const P& p, uint8_t* ring, uint64_t* landed, int32_t* err, int first, int wp, int lane,
                                            Place place, Publish publish) {
    const BlockView& c = p.c;
    const int sh = c.log2_block - 5;
    RowWalk<P> w(p);
    bool more = w.next();
    int j = w.j0, k = 0;  // the next step to look at
    auto skip = [&]() {
        ++k;
        if (more && ++j == w.j1) {
            more = w.next();
            if (more) j = w.j0;
        }
    };
    if (first) skip();
    auto look = [&]() {
        RowPart x = {-1, 0, 0, 0, 0, -1};
        if (!more) return x;
        const auto& e = p.seqs[w.i];
        x = RowPart{k, e.seq, e.n, w.h, 4 * j + wp, -1};
        if (x.tile < e.n >> c.log2_block << sh) x.slot = __ldg(block_table(c, e.seq) + (x.tile >> sh));
#pragma unroll
        for (int z = 0; z < STRIDE; ++z) skip();
        return x;
    };
    int issued = 0, done = 0;  // entries; entry x is place x & 1, phase x >> 1 of its barrier
    bool ok = true;            // no wait has given up
    // the part's copy, where there is room for it
    auto fetch = [&](const RowPart& a) {
        if (!ok) return false;
        if (a.slot >= 0) {
            if (issued - done >= 2) return false;
            if (lane == 0) {
                const uint8_t* rec = tile_ptr(c, a.slot, a.kvh, a.tile & ((1 << sh) - 1));
                uint8_t* to = ring + (issued & 1) * kRingEntry<D>;
                mbar_arrive_expect_tx(landed + (issued & 1), kRingEntry<D>);
                if (IS_V) {
                    bulk_g2s(to, rec, 16, landed + (issued & 1));
                    bulk_g2s(to + 16, rec + 16 + kTileTokens * D, kTileTokens * D, landed + (issued & 1));
                } else {
                    bulk_g2s(to, rec, kRingEntry<D>, landed + (issued & 1));
                }
            }
            ++issued;
        } else if (a.exact() > 0) {
            if (issued != done) return false;
            const bool odd = issued & 1;
            if (lane == 0) {
                if (odd) mbar_arrive(landed + 1);  // from the ring's start on
                constexpr int kBytes = kTileTokens * D * 2;
                static_assert(kBytes <= 2 * kRingEntry<D>, "room for an exact part");
                mbar_arrive_expect_tx(landed, kBytes);
                bulk_g2s(ring, tail_ptr(c, IS_V ? c.lay.tail_v : c.lay.tail_k, a.seq, a.kvh) +
                                   (size_t)(a.tile - (a.n >> c.log2_block << sh)) * (kTileTokens * D), kBytes, landed);
                mbar_arrive(landed + 1);
            }
            if (odd) ++issued, ++done;
            issued += 2;
        }
        return true;
    };
    RowPart now = look(), next = look(), then = look();
    int ahead = 0;  // of the first two, on their way
    auto pump = [&]() {
        if (ahead == 0 && fetch(now)) ahead = 1;
        if (ahead == 1 && fetch(next)) ahead = 2;
    };
    pump();
#pragma unroll 1
    while (now.step >= 0) {
        uint8_t* dst = place(now.step);
        bool here = __all_sync(0xffffffffu, dst != nullptr);  // (the expansion of exact rows is warp-wide)
        float2 h = make_float2(1.f, 1.f);
        uint32_t bad = 0;
        int used = 0;
        if (here && ok) {
            if (now.slot >= 0) {
                here = bar_wait(landed + (done & 1), (uint32_t)(done >> 1 & 1), err);
                const uint8_t* rec = ring + (done & 1) * kRingEntry<D>;
                const float4 hd = *reinterpret_cast<const float4*>(rec);
                h = IS_V ? make_float2(hd.z, hd.w) : make_float2(hd.x, 0.f);
                expand_codes<D, INT8, IS_V>(rec, dst, wp, lane);
                used = 1;
            } else {
                if (now.exact() > 0) {
                    here = __all_sync(0xffffffffu, bar_wait(landed, (uint32_t)(done >> 1 & 1), err));
                    used = 2;
                }
                expand_rows<D, BF16, IS_V>(ring, now.exact(), dst, wp, lane, h, bad);
            }
        }
        ok = __all_sync(0xffffffffu, here) && ok;  // one answer for the warp; also: all lanes have read
        if (ok) done += used;
        fence_proxy_async_smem();
        publish(now.step, h, bad);
        now = next;
        next = then;
        ahead = max(ahead - 1, 0);
        pump();
        then = look();  // its slot is there by the time it is fetched, a turn from now
    }
    // Normally every copy was waited for above. After a wait that gave up nothing more was issued, and what is in flight
    // lands (a bounded wait again) before the CTA's shared memory goes away.
    if (!ok) {
        const uint64_t t0 = global_ns();
#pragma unroll 1
        for (; done < issued; ++done)
            while (!mbar_try_wait(landed + (done & 1), (uint32_t)(done >> 1 & 1)) && global_ns() - t0 < kWaitLimitNs) {
            }
    }
}

}  // namespace kvarn
