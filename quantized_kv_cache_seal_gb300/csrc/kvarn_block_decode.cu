// Block cache: decode attention, one query token per sequence.
//
//   o = sum_n w_n v_n / sum_n w_n, w_n = 2^(x_n), x_n = scale log2(e) (q . code_n) s_K,n.
// Codes are exact in f16, so q . code runs on the tensor cores with fp32 sums (bf16 queries
// enter as f16 after an exact power of two brings the head's largest value under 2^15: what
// that drops is 2^-39 of it). V's scale is folded into the weight: w'_n = 2^(x_n + log2 s_V,n
// - m' + 15), m' the running maximum of x + log2 s_V, so that weights are at most 2^15 in f16
// whatever V's range, and keep all its bits down to 2^-29 of the largest; the denominator adds
// w' / s_V in fp32, in units of 2^12 (kDenomUnit). Rounding w' to f16 is off by at most 2^-11 of
// each weight, less in sum than the output's own rounding; bf16 would cost eight times that.
//
// Bound by memory: 4 r operations of a KV head's r query heads per 2 code bytes. All (sequence,
// KV head) pairs form one line of 32-token tiles that is cut evenly over the CTAs, one a SM;
// the warps of a CTA take its tiles in turn. A tile is one contiguous record (two where it is
// exact) that a warp fetches with one bulk copy into a ring of its own (three deep at head_dim
// 128: 197 KB in flight a SM, which covers the latency four times), so that the warps meet only
// at the end of a (sequence, KV head), and without a barrier. Codes lie in the order of
// mma.m16n8k16's A operand:
// K (tokens x channels) x q gives S^T, whose accumulators become the weights' B operand for
// V^T (channels x tokens) by one movmatrix each; heads are the 8 columns, so up to 8 query
// heads cost the same. Warps join in shared memory and CTAs that share a pair through a
// workspace, each added in a fixed order by whichever comes last: results do not depend on
// timing. mma.sync suits it better than tcgen05: M = 128 of the latter would be 4 query heads
// and 124 rows of nothing, and the tensor pipe is idle four fifths of the time as it is.
//
// 16 sequences of 32k tokens, 32 / 8 heads, e4m3: 176 us, 6.1 TB/s of code bytes, 0.90 of a plain
// copy's rate; 64 ragged sequences of 1k..16k, 40 / 10 heads, int8, bf16: 262 us, 5.7 TB/s.
//
// KVARN_BLOCK_MORE: the variant with prefixes and weights, a translation unit of its own (kvarn_block_decode_more.cu), so that
// calls without them keep their code. A prefix's tiles stand in front of a sequence's own in its line, or its row over a
// prefix walked once for many sequences is joined at the end; each tile's maximum and sum of weights go to `sums`.
#include "kvarn_block_dev.cuh"

namespace kvarn {
namespace {

#ifdef KVARN_BLOCK_MORE
constexpr bool kMore = true;
#define KVARN_MORE_PARAM , const __grid_constant__ BlockDecodeMore x
typedef BlockDecodeMore More;
#else
constexpr bool kMore = false;
#define KVARN_MORE_PARAM
// (nothing of it is read)
struct More {
    float2 *sums, *totals;
    const float *pre_o, *pre_lse;
    uint32_t merged[1];
    int32_t pre[1], pre_n[1];
};
#endif

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr float kShift = 15.f;  // weights are at most 2^15 (total_of counts on it)

template <int D>
struct Shape {
    static constexpr int kTile = 16 + 2 * kTileTokens * D;  // a sealed tile; an exact one's K or V is 16 bytes less
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kHeadStride = D + 8;  // floats of a head in the join buffer: the two heads of a lane pair sit 16 banks apart
    static constexpr int kRing = kWarps * kStages * kTile;
    static constexpr int kJoin = kRing;                                    // float[warps][4][D + 8]
    static constexpr int kM = kJoin + kWarps * 4 * kHeadStride * 4;        // float[warps][4]
    static constexpr int kL = kM + kWarps * 4 * 4;
    static constexpr int kBars = kL + kWarps * 4 * 4;
    static constexpr int kFree = kBars + kWarps * kStages * 8;             // barrier: the join buffer may be written again
    static constexpr int kCount = kFree + 8;                               // int: warps that have written it
    static constexpr int kSmem = kCount + 8;
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A position on the line of tiles: the (sequence, KV head) that unit u belongs to.
struct Cursor {
    int i, h, begin, end;
    __device__ __forceinline__ void start(const BlockDecodeParams& p, int u) {
        int lo = 0;
#pragma unroll 1
        for (int hi = p.n_seqs - 1; lo < hi;) {
            const int mid = (lo + hi + 1) / 2;
            if (p.seqs[mid].unit_begin <= u) lo = mid; else hi = mid - 1;
        }
        i = lo;
        h = (u - p.seqs[lo].unit_begin) / p.seqs[lo].units;
        begin = p.seqs[lo].unit_begin + h * p.seqs[lo].units;
        end = begin + p.seqs[lo].units;
    }
    __device__ __forceinline__ void advance(const BlockDecodeParams& p, int u) {
        while (u >= end) {
            if (++h == p.c.hkv) h = 0, ++i;
            begin = end;
            end += p.seqs[i].units;
        }
    }
};

// The warp's state for one (sequence, KV head); lane 4 g + t holds heads 2 t, 2 t + 1.
template <int D>
struct State {
    float m[2], l[2];
    float o[D / 16][4];  // O^T: channels 16 i + g (+ 8), heads 2 t, 2 t + 1
};

// Tile t of a sequence's line: of the prefix in front of it (where it has one here), then its own.
struct TilePlace {
    int seq, n, tile;
};
__device__ __forceinline__ TilePlace place_of(const BlockDecodeParams& p, const More& x, int i, int t) {
    const BlockDecodeSeq& e = p.seqs[i];
    if (!kMore) return TilePlace{e.seq, e.n, t};
    const int before = (x.pre_n[i] + kTileTokens - 1) / kTileTokens;
    return t < before ? TilePlace{x.pre[i], x.pre_n[i], t} : TilePlace{e.seq, e.n, t - before};
}

// Weights of 32 tokens from S^T (rows g, g + 8 of the two 16-token halves).
// sums: where the tile's maximum and sum of each head go, or null.
template <int D>
__device__ __forceinline__ void weigh(State<D>& st, const float (&s)[2][4], float f0, float f1, float lv, float ivs, int nv,
                                      int lane, int r, float2* sums, uint32_t (&w)[2][2]) {
    const int g = lane >> 2;
    float x[2][4];
    float m0 = kNegInf, m1 = kNegInf;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const bool in = 8 * (g >> 1) + 4 * a + 2 * b + (g & 1) < nv;
            x[a][2 * b] = in ? fmaf(s[a][2 * b], f0, lv) : kNegInf;
            x[a][2 * b + 1] = in ? fmaf(s[a][2 * b + 1], f1, lv) : kNegInf;
            m0 = fmaxf(m0, x[a][2 * b]);
            m1 = fmaxf(m1, x[a][2 * b + 1]);
        }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
    }
    if (__any_sync(0xffffffffu, m0 > st.m[0] || m1 > st.m[1])) {
        m0 = fmaxf(m0, st.m[0]);
        m1 = fmaxf(m1, st.m[1]);
        const float r0 = m0 > st.m[0] ? ex2(st.m[0] - m0) : 1.f, r1 = m1 > st.m[1] ? ex2(st.m[1] - m1) : 1.f;
        st.m[0] = m0;
        st.m[1] = m1;
        st.l[0] *= r0;
        st.l[1] *= r1;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            st.o[i][0] *= r0;
            st.o[i][1] *= r1;
            st.o[i][2] *= r0;
            st.o[i][3] *= r1;
        }
    }
    // a head without a finite logit so far keeps m = -inf; its weights must not be 2^(inf - inf)
    const float n0 = st.m[0] == kNegInf ? 0.f : st.m[0] - kShift, n1 = st.m[1] == kNegInf ? 0.f : st.m[1] - kShift;
    float l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float p0 = ex2(x[a][2 * b] - n0), p1 = ex2(x[a][2 * b + 1] - n1);
            l0 += p0;
            l1 += p1;
            w[a][b] = movmatrix(pack2<false>(p0, p1));
        }
    st.l[0] = fmaf(l0, ivs, st.l[0]);
    st.l[1] = fmaf(l1, ivs, st.l[1]);
    if (kMore && sums) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, d);
            l1 += __shfl_xor_sync(0xffffffffu, l1, d);
        }
        const int h = 2 * (lane & 3);
        if (g == 0 && h < r) sums[h] = make_float2(st.m[0], l0 * ivs);
        if (g == 0 && h + 1 < r) sums[h + 1] = make_float2(st.m[1], l1 * ivs);
    }
}

template <int D, bool INT8>
__device__ __forceinline__ void sealed_unit(State<D>& st, const uint8_t* t, const uint32_t (&q)[D / 64][4][2], float c0, float c1,
                                            int lane, int r, float2* sums) {
    const float4 hd = *reinterpret_cast<const float4*>(t);
    float s[2][4] = {};
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const uint8_t* at = t + 16 + (a * (D / 64) + c) * 1024 + lane * 16;
            const uint4 u = *reinterpret_cast<const uint4*>(at), v = *reinterpret_cast<const uint4*>(at + 512);
            const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                mma16816(s[a], codes_lo<INT8>(x[j]), codes_lo<INT8>(y[j]), codes_hi<INT8>(x[j]), codes_hi<INT8>(y[j]),
                         q[c][j][0], q[c][j][1]);
        }
    uint32_t w[2][2];
    weigh<D>(st, s, c0 * hd.x, c1 * hd.x, hd.z, hd.w, kTileTokens, lane, r, sums, w);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(t + 16 + kTileTokens * D + i * 512 + lane * 16);
        mma16816(st.o[i], codes_lo<INT8>(x.x), codes_lo<INT8>(x.z), codes_hi<INT8>(x.x), codes_hi<INT8>(x.z), w[0][0], w[0][1]);
        mma16816(st.o[i], codes_lo<INT8>(x.y), codes_lo<INT8>(x.w), codes_hi<INT8>(x.y), codes_hi<INT8>(x.w), w[1][0], w[1][1]);
    }
}

// 32 exact tokens (nv of them valid) from the tail: rows k, channel rows v of 32 tokens. bf16
// values become f16 after the tile's own exact powers of two, as the queries do.
template <int D, bool BF16>
__device__ __forceinline__ void exact_unit(State<D>& st, const uint16_t* k, const uint16_t* v, int nv,
                                           const uint32_t (&q)[D / 64][4][2], float c0, float c1, int lane, int heads,
                                           float2* sums) {
    const int g = lane >> 2, t = lane & 3;
    float ks = 1.f;
    float s[2][4] = {};
    {
        uint4 x[2][D / 64][2][2];  // half, 64-channel part, rows g / g + 8, 16 channels
        uint32_t top = 0;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int tok = 8 * (g >> 1) + 4 * a + 2 * b + (g & 1);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint4 r = make_uint4(0, 0, 0, 0);
                        if (tok < nv) r = *reinterpret_cast<const uint4*>(k + tok * D + 64 * c + 16 * t + 8 * z);
                        x[a][c][b][z] = r;
                        if (BF16) top = max_of(top, finite_only<BF16>(r));  // an infinity must not scale the others away
                    }
            }
        float f = 1.f;
        if (BF16) {
            top = max(top & 0xffffu, top >> 16);
            for (int d = 16; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
            const int e = exponent_of<BF16>(top) - kExactK;
            f = power2(-e);
            ks = power2(e);
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const uint4 u = x[a][c][0][z], w = x[a][c][1][z];
                    const uint32_t lo[4] = {u.x, u.y, u.z, u.w}, hi[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t r[4] = {lo[2 * j], hi[2 * j], lo[2 * j + 1], hi[2 * j + 1]};
                        if (BF16)
#pragma unroll
                            for (int y = 0; y < 4; ++y) r[y] = scaled_f16<BF16>(r[y], f);
                        mma16816(s[a], r[0], r[1], r[2], r[3], q[c][2 * z + j][0], q[c][2 * z + j][1]);
                    }
                }
    }
    uint4 y[D / 16][2];
    uint32_t top = 0;
    uint32_t keep[4];  // tokens of the lane's four words that are valid
#pragma unroll
    for (int z = 0; z < 4; ++z)
        keep[z] = (8 * t + 2 * z < nv ? 0xffffu : 0u) | (8 * t + 2 * z + 1 < nv ? 0xffff0000u : 0u);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint4 r = *reinterpret_cast<const uint4*>(v + (16 * i + g + 8 * b) * kTileTokens + 8 * t);
            r = make_uint4(r.x & keep[0], r.y & keep[1], r.z & keep[2], r.w & keep[3]);
            y[i][b] = r;
            top = max_of(top, finite_only<BF16>(r));
        }
    const int e = warp_exponent_v<BF16>(top);
    const float f = power2(-e);
    uint32_t w[2][2];
    weigh<D>(st, s, c0 * ks, c1 * ks, (float)e, f * kDenomUnit, nv, lane, heads, sums, w);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            uint32_t r[4] = {a ? y[i][0].z : y[i][0].x, a ? y[i][1].z : y[i][1].x, a ? y[i][0].w : y[i][0].y,
                             a ? y[i][1].w : y[i][1].y};
#pragma unroll
            for (int z = 0; z < 4; ++z) r[z] = scaled_f16<BF16>(r[z], f);
            mma16816(st.o[i], r[0], r[1], r[2], r[3], w[a][0], w[a][1]);
        }
}

// Heads h0 .. h0 + heads - 1 (four at most) of one (sequence, KV head) from the warps' states in the join
// buffer, by one warp, a lane 4 channels (at head_dim 64 half the lanes). Where the CTA holds only a part of
// the pair, the part goes to the workspace, and whichever part comes last adds them all in the order of the
// cuts. row: of the pair's first head in q and out.
// ALONE: a warp's own state instead (w: this one), and parts of the warps' own.
template <int D, bool BF16, bool ALONE>
__device__ void join_heads(const BlockDecodeParams& p, const More& x, const uint8_t* smem, const Cursor& cur, bool whole,
                           bool starts, int half, size_t row, int w, int lane) {
    using Sh = Shape<D>;
    const float* join = reinterpret_cast<const float*>(smem + Sh::kJoin);
    const float* sm = reinterpret_cast<const float*>(smem + Sh::kM);
    const float* sl = reinterpret_cast<const float*>(smem + Sh::kL);
    const int heads = min(4, p.r - 4 * half), b = ALONE ? blockIdx.x * kWarps + w : blockIdx.x, workers = ALONE ? p.grid * kWarps : p.grid;
    const int z0 = ALONE ? w : 0, z1 = ALONE ? w + 1 : kWarps;
    const bool live = 4 * lane < D;
    constexpr size_t kPart = 8 * (D + 2);  // floats: O [8][D], m [8], l [8]
    float* partials = reinterpret_cast<float*>(p.c.base + p.c.lay.partials);
    float* mine = partials + (size_t)(2 * b + (starts ? 1 : 0)) * kPart;
    const bool merged = kMore && x.pre_lse && (x.merged[cur.i >> 5] >> (cur.i & 31) & 1);
    auto give = [&](int head, float4 o, float m, float l) {
        const float inv = l == 0.f ? 0.f : 1.f / l, u = kDenomUnit;
        float4 y = make_float4(o.x * u * inv, o.y * u * inv, o.z * u * inv, o.w * u * inv);
        if (kMore && x.totals && lane == 0) {
            float2 t = make_float2(m, l);
            if (merged) t = joined(t, x.totals[row + head]);
            x.totals[row + head] = t;
        }
        if (kMore && merged) {  // with the finished row over the shared prefix
            const float2 f = merge_factors(lse_of(m, l, kShift), x.pre_lse[row + head]);
            float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            if (live) z = *reinterpret_cast<const float4*>(x.pre_o + (row + head) * D + 4 * lane);
            y = make_float4(merge(y.x, z.x, f), merge(y.y, z.y, f), merge(y.z, z.z, f), merge(y.w, z.w, f));
        }
        if (live)
            *reinterpret_cast<uint2*>(p.out + (row + head) * D + 4 * lane) =
                make_uint2(pack2<BF16>(y.x, y.y), pack2<BF16>(y.z, y.w));
    };
    // (alone there is nothing else to do while a head's loads are on their way)
#pragma unroll(ALONE ? 4 : 1)
    for (int h = 0; h < (ALONE ? 4 : heads); ++h) {
        if (ALONE && h >= heads) break;
        float big = kNegInf, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int z = z0; z < z1; ++z) big = fmaxf(big, sm[z * 4 + h]);
#pragma unroll
        for (int z = z0; z < z1; ++z) {
            const float mz = sm[z * 4 + h], f = mz == kNegInf ? 1.f : ex2(mz - big);  // -inf: zeros or NaN
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (live) x = *reinterpret_cast<const float4*>(join + (z * 4 + h) * Sh::kHeadStride + 4 * lane);
            o.x = fmaf(x.x, f, o.x);
            o.y = fmaf(x.y, f, o.y);
            o.z = fmaf(x.z, f, o.z);
            o.w = fmaf(x.w, f, o.w);
            l = fmaf(sl[z * 4 + h], f, l);
        }
        if (whole) {
            give(4 * half + h, o, big, l);
        } else {
            if (live) *reinterpret_cast<float4*>(mine + (4 * half + h) * D + 4 * lane) = o;
            if (lane == 0) mine[8 * D + 4 * half + h] = big, mine[8 * D + 8 + 4 * half + h] = l;
        }
    }
    if (whole || 4 * half + heads < p.r) return;
    // CTAs first .. last share the pair; its first one's counter takes the arrivals
    int32_t* counters = reinterpret_cast<int32_t*>(p.c.base + (ALONE ? p.c.lay.warp_counters : p.c.lay.counters));
    const int first = (int)((((int64_t)cur.begin + 1) * workers - 1) / p.units);
    const int last = (int)(((int64_t)(cur.end - (ALONE ? kPairCost : 0)) * workers - 1) / p.units);
    __threadfence();
    __syncwarp();
    int n = 0;
    if (lane == 0) n = atomicAdd(counters + first, 1);
    if (__shfl_sync(0xffffffffu, n, 0) != last - first) return;
    if (lane == 0) counters[first] = 0;
    __threadfence();
    // part z of CTA first + z: slot 1 of the first, slot 0 of the others
    auto part = [&](int z) { return partials + (size_t)(2 * (first + z) + (z == 0 ? 1 : 0)) * kPart; };
#pragma unroll 1
    for (int h0 = 0; h0 < p.r; h0 += 4) {
        float big[4], l[4];
        float4 o[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) big[y] = kNegInf, l[y] = 0.f, o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int z0 = 0; z0 <= last - first; z0 += 32) {  // 32 parts at a time, a lane their m and l
            const int parts = min(32, last - first + 1 - z0);
            float f[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int h = min(h0 + y, p.r - 1);
                float m = kNegInf, s = 0.f;
                if (lane < parts) {
                    m = __ldcg(part(z0 + lane) + 8 * D + h);
                    s = __ldcg(part(z0 + lane) + 8 * D + 8 + h);
                }
                float top = m;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                top = fmaxf(top, big[y]);
                f[y] = m == kNegInf ? 1.f : ex2(m - top);
                s *= f[y];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                const float g = big[y] == kNegInf ? 1.f : ex2(big[y] - top);
                l[y] = fmaf(l[y], g, s);
                o[y].x *= g, o[y].y *= g, o[y].z *= g, o[y].w *= g;
                big[y] = top;
            }
#pragma unroll 4
            for (int z = 0; z < parts; ++z) {
                const float* at = part(z0 + z) + 4 * lane;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int h = min(h0 + y, p.r - 1);
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (live) x = __ldcg(reinterpret_cast<const float4*>(at + h * D));
                    const float w = __shfl_sync(0xffffffffu, f[y], z);
                    o[y].x = fmaf(x.x, w, o[y].x);
                    o[y].y = fmaf(x.y, w, o[y].y);
                    o[y].z = fmaf(x.z, w, o[y].z);
                    o[y].w = fmaf(x.w, w, o[y].w);
                }
            }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
            if (h0 + y < p.r) give(h0 + y, o[y], big[y], l[y]);
    }
}

// ALONE: the line is cut over the warps, not over the CTAs, and a warp ends its pairs by itself: where pairs are short, eight
// warps would spend more time on joining than on their few tiles each.
template <int D, bool INT8, bool BF16, bool ALONE>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ BlockDecodeParams p KVARN_MORE_PARAM) {
    using Sh = Shape<D>;
#ifndef KVARN_BLOCK_MORE
    const More x = {};
#endif
    extern __shared__ __align__(128) uint8_t smem[];
    const BlockView& c = p.c;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + w * Sh::kStages * Sh::kTile;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kBars) + w * Sh::kStages;
    float* join = reinterpret_cast<float*>(smem + Sh::kJoin);
    float* sm = reinterpret_cast<float*>(smem + Sh::kM);
    float* sl = reinterpret_cast<float*>(smem + Sh::kL);
    uint64_t* free_bar = reinterpret_cast<uint64_t*>(smem + Sh::kFree);
    int* count = reinterpret_cast<int*>(smem + Sh::kCount);
    int32_t* err = reinterpret_cast<int32_t*>(c.base + c.lay.err);
    const int b = ALONE ? blockIdx.x * kWarps + w : blockIdx.x, workers = ALONE ? p.grid * kWarps : p.grid;
    constexpr int kTurn = ALONE ? 1 : kWarps;
    const int mine = ALONE ? 0 : w;
    const int u0 = (int)(p.units * b / workers), u1 = (int)(p.units * (b + 1) / workers);
    if (lane < Sh::kStages) mbar_init(bars + lane, 1);
    if (threadIdx.x == 0) {
        mbar_init(free_bar, 1);
        *count = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    if (kMore) {
        before_done();
        start_next();
    }

    // Copies run ahead of the work: a sealed tile takes one ring entry, an exact one two (K rows, V
    // channel rows), an empty sequence's unit none. The next tile's slot is loaded a step early.
    Cursor ahead;
    int ua = u0 + mine, slot = 0, issued = 0, done = 0;  // issued, done: ring entries
    bool ok = true;                                   // no wait for a copy has given up
    const int sh = c.log2_block - 5;
    auto seek = [&]() {
        if (ua >= u1) return;
        ahead.advance(p, ua);
        const TilePlace e = place_of(p, x, ahead.i, ua - ahead.begin);
        slot = -1;
        if (e.tile < e.n >> c.log2_block << sh) slot = read<kMore>(block_table(c, e.seq) + (e.tile >> sh));
    };
    auto entry = [&](const void* src, uint32_t bytes) {
        if (lane == 0) {
            const int st = issued % Sh::kStages;
            mbar_arrive_expect_tx(bars + st, bytes);
            bulk_g2s(ring + st * Sh::kTile, src, bytes, bars + st);
        }
        ++issued;
    };
    auto pump = [&]() {
#pragma unroll 1
        while (ok && ua < u1 && issued - done + (slot < 0 ? 2 : 1) <= Sh::kStages) {
            const TilePlace e = place_of(p, x, ahead.i, ua - ahead.begin);
            const int tile = e.tile, sealed = e.n >> c.log2_block << sh;
            if (slot >= 0) {
                entry(tile_ptr(c, slot, ahead.h, tile & ((1 << sh) - 1)), Sh::kTile);
            } else if (tile * kTileTokens < e.n) {
                constexpr uint32_t kSide = kTileTokens * D * 2;
                const size_t at = (size_t)(tile - sealed) * (kTileTokens * D);
                entry(tail_ptr(c, c.lay.tail_k, e.seq, ahead.h) + at, kSide);
                entry(tail_ptr(c, c.lay.tail_v, e.seq, ahead.h) + at, kSide);
            }
            ua += kTurn;
            seek();
        }
    };
    Cursor cur;
    cur.start(p, u0);
    ahead = cur;
    seek();
    pump();

    int u = u0 + mine, joins = 0;
    for (int begin = u0; begin < u1; begin = min(cur.end, u1)) {
        cur.advance(p, begin);
        const int tiles_end = cur.end - (ALONE ? kPairCost : 0);
        if (ALONE && begin >= tiles_end) {  // of the pair nothing but its cost
            u = min(cur.end, u1);
            continue;
        }
        const int end = min(tiles_end, u1);
        const int h0 = cur.h * p.r;
        // the queries of the pair's r heads as B operands: lane 4 g + t holds head g, channels
        // 64 c + 16 t + 4 j + {0, 1} and {2, 3}
        uint32_t q[D / 64][4][2];
        float c0 = p.scale_log2, c1 = p.scale_log2;
        {
            const uint16_t* src = p.q + ((size_t)cur.i * p.hq + h0 + g) * D + 16 * t;
            uint32_t top = 0;
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (g < p.r) x = *reinterpret_cast<const uint4*>(src + 64 * a + 8 * z);
                    if (BF16) top = max_of(top, x);
                    q[a][2 * z][0] = x.x;
                    q[a][2 * z][1] = x.y;
                    q[a][2 * z + 1][0] = x.z;
                    q[a][2 * z + 1][1] = x.w;
                }
            if (BF16) {
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ex = exponent_of<BF16>(top) - kExactK;
                const float f = power2(-ex);
#pragma unroll
                for (int a = 0; a < D / 64; ++a)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        q[a][j][0] = scaled_f16<BF16>(q[a][j][0], f);
                        q[a][j][1] = scaled_f16<BF16>(q[a][j][1], f);
                    }
                c0 *= power2(__shfl_sync(0xffffffffu, ex, 8 * t));
                c1 *= power2(__shfl_sync(0xffffffffu, ex, 8 * t + 4));
            }
        }
        State<D> st;
        st.m[0] = st.m[1] = kNegInf;
        st.l[0] = st.l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int z = 0; z < 4; ++z) st.o[i][z] = 0.f;
        for (; u < end; u += kTurn) {
            if (!ok) continue;
            const TilePlace e = place_of(p, x, cur.i, u - cur.begin);
            const int tile = e.tile, sealed = e.n >> c.log2_block << sh;
            float2* sums = kMore && x.sums ? x.sums + (size_t)u * p.r : nullptr;
            bool landed = true;
            int entries = 0;
            if (tile < sealed) {
                const int s = done % Sh::kStages;
                landed = bar_wait(bars + s, (uint32_t)(done / Sh::kStages & 1), err);
                sealed_unit<D, INT8>(st, ring + s * Sh::kTile, q, c0, c1, lane, p.r, sums);
                entries = 1;
            } else if (const int nv = min(kTileTokens, e.n - tile * kTileTokens); nv > 0) {
                const int s = done % Sh::kStages, s2 = (done + 1) % Sh::kStages;
                landed = bar_wait(bars + s, (uint32_t)(done / Sh::kStages & 1), err);
                landed = bar_wait(bars + s2, (uint32_t)((done + 1) / Sh::kStages & 1), err) && landed;
                exact_unit<D, BF16>(st, reinterpret_cast<const uint16_t*>(ring + s * Sh::kTile),
                                    reinterpret_cast<const uint16_t*>(ring + s2 * Sh::kTile), nv, q, c0, c1, lane, p.r, sums);
                entries = 2;
            } else if (kMore && sums && lane < p.r) {
                sums[lane] = make_float2(kNegInf, 0.f);  // an empty sequence
            }
            // one answer for the warp, after the products that need not wait for it; also: all lanes have read
            ok = __all_sync(0xffffffffu, landed);
            if (!ok) continue;
            done += entries;
            pump();
        }
        // Join the warps, four heads at a time: each puts its state into the buffer and goes on; the last
        // one to come adds them. (A barrier here left the memory idle at every pair's end.)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], d);
            st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], d);
        }
        const bool whole = begin == cur.begin && end == tiles_end;
        if (ALONE) u = min(cur.end, u1);
#pragma unroll 1
        for (int half = 0; half < (p.r > 4 ? 2 : 1); ++half, ++joins) {
            if (!ALONE && joins > 0) bar_wait(free_bar, (uint32_t)((joins - 1) & 1), err);
            if (t >> 1 == half) {
                const int h = 2 * (t & 1);
                float* at = join + (w * 4 + h) * Sh::kHeadStride + g;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    at[16 * i] = st.o[i][0];
                    at[16 * i + 8] = st.o[i][2];
                    at[16 * i + Sh::kHeadStride] = st.o[i][1];
                    at[16 * i + 8 + Sh::kHeadStride] = st.o[i][3];
                }
                if (g == 0) {
                    sm[w * 4 + h] = st.m[0];
                    sm[w * 4 + h + 1] = st.m[1];
                    sl[w * 4 + h] = st.l[0];
                    sl[w * 4 + h + 1] = st.l[1];
                }
            }
            if (ALONE) {
                __syncwarp();
                join_heads<D, BF16, ALONE>(p, x, smem, cur, whole, begin == cur.begin, half, (size_t)cur.i * p.hq + h0, w, lane);
                __syncwarp();
                continue;
            }
            __threadfence_block();
            __syncwarp();
            int n = 0;
            if (lane == 0) n = atomicAdd(count, 1);
            if (__shfl_sync(0xffffffffu, n, 0) == kWarps - 1) {
                __threadfence_block();
                join_heads<D, BF16, ALONE>(p, x, smem, cur, whole, begin == cur.begin, half, (size_t)cur.i * p.hq + h0, w, lane);
                __syncwarp();
                if (lane == 0) {
                    *count = 0;
                    __threadfence_block();
                    mbar_arrive(free_bar);
                }
            }
        }
    }
    // Normally every copy was waited for above. After a wait that gave up nothing more was issued, and what is
    // in flight lands (a bounded wait again) before the CTA's shared memory goes away.
    if (!ok) {
        const uint64_t t0 = global_ns();
#pragma unroll 1
        for (; done < issued; ++done)
            while (!mbar_try_wait(bars + done % Sh::kStages, (uint32_t)(done / Sh::kStages & 1)) && global_ns() - t0 < kWaitLimitNs) {
            }
    }
}

#ifdef KVARN_BLOCK_MORE
#define KVARN_ARGS p, x
#define KVARN_PARAMS const BlockDecodeParams &p, const BlockDecodeMore &x
#else
#define KVARN_ARGS p
#define KVARN_PARAMS const BlockDecodeParams& p
#endif

template <int D, bool INT8, bool BF16, bool ALONE = false>
int launch(KVARN_PARAMS, cudaStream_t s) {
#ifdef KVARN_BLOCK_MORE
    if (!ALONE && x.alone) return launch<D, INT8, BF16, true>(p, x, s);
#endif
    static SmemOnce once;
    const int e = once.allow(reinterpret_cast<const void*>(decode_kernel<D, INT8, BF16, ALONE>), Shape<D>::kSmem);
    if (e) return e;
#ifdef KVARN_BLOCK_MORE
    return launch_behind(decode_kernel<D, INT8, BF16, ALONE>, p.grid, kThreads, Shape<D>::kSmem, s, p, x);
#else
    decode_kernel<D, INT8, BF16, ALONE><<<p.grid, kThreads, Shape<D>::kSmem, s>>>(p);
    return (int)cudaGetLastError();
#endif
}

}  // namespace

int launch_block_decode(KVARN_PARAMS, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    switch ((p.c.d == 128 ? 4 : 0) + (p.c.int8 ? 2 : 0) + (p.c.bf16 ? 1 : 0)) {
        case 0: return launch<64, false, false>(KVARN_ARGS, s);
        case 1: return launch<64, false, true>(KVARN_ARGS, s);
        case 2: return launch<64, true, false>(KVARN_ARGS, s);
        case 3: return launch<64, true, true>(KVARN_ARGS, s);
        case 4: return launch<128, false, false>(KVARN_ARGS, s);
        case 5: return launch<128, false, true>(KVARN_ARGS, s);
        case 6: return launch<128, true, false>(KVARN_ARGS, s);
        default: return launch<128, true, true>(KVARN_ARGS, s);
    }
}

}  // namespace kvarn
