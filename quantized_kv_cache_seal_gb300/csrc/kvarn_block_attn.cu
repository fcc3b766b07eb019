// Block cache: attention.
#include "kvarn_block_dev.cuh"

namespace kvarn {
namespace {

// One warp per (query token, query head): logits and the weighted sum in fp32, token by token.
template <bool BF16, bool INT8>
__global__ void __launch_bounds__(128) simple_kernel(const __grid_constant__ BlockPrefillParams p) {
    const BlockView& c = p.c;
    const int64_t w = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    int i = 0;
    while (i + 1 < p.n_seqs && p.seqs[i + 1].cta_begin <= w) ++i;
    const BlockPrefillSeq& e = p.seqs[i];
    const int rel = (int)(w - e.cta_begin);
    if (rel >= e.q_len * p.hq) return;
    const int tok = rel / p.hq, h = rel % p.hq, kh = h / p.r, d = c.d;
    const uint16_t* q = p.q + ((size_t)(e.q_row + tok) * p.hq + h) * d;
    uint16_t* out = p.out + ((size_t)(e.q_row + tok) * p.hq + h) * d;
    const int seen = e.n - e.q_len + tok + 1;  // visible tokens
    const int sealed = e.n & ~(c.block - 1);
    const uint16_t* tk = tail_ptr(c, c.lay.tail_k, e.seq, kh);
    const uint16_t* tv = tail_ptr(c, c.lay.tail_v, e.seq, kh);
    float m = -__int_as_float(0x7f800000), l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int n = 0; n < seen; ++n) {
        float dot = 0.f, v[4];
        const uint8_t* t = n < sealed ? sealed_tile(c, block_table(c, e.seq), kh, n / kTileTokens) : nullptr;
        const int tt = n % kTileTokens;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const int ch = lane + 32 * z;
            v[z] = 0.f;
            if (ch >= d) continue;
            float k;
            if (t) {
                const float ks = reinterpret_cast<const float*>(t)[0], vs = reinterpret_cast<const float*>(t)[1];
                k = unpack2<false>(codes_lo<INT8>(t[k_code_off(d, tt, ch & ~7) + (ch & 7)])).x * ks;
                v[z] = unpack2<false>(codes_lo<INT8>(t[v_code_off(d, tt & ~7, ch) + (tt & 7)])).x * vs;
            } else {
                k = unpack2<BF16>(tk[(size_t)(n - sealed) * d + ch]).x;
                v[z] = unpack2<BF16>(tv[(size_t)ch * c.block + (n - sealed)]).x;
            }
            dot += k * unpack2<BF16>(q[ch]).x;
        }
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        dot *= p.scale_log2;
        const float m1 = fmaxf(m, dot), f = exp2f(m - m1), w1 = exp2f(dot - m1);
        l = l * f + w1;
#pragma unroll
        for (int z = 0; z < 4; ++z) acc[z] = acc[z] * f + w1 * v[z];
        m = m1;
    }
    for (int z = 0; z < 4; ++z)
        if (lane + 32 * z < d) out[lane + 32 * z] = (uint16_t)pack2<BF16>(seen > 0 ? acc[z] / l : 0.f, 0.f);
}

}  // namespace

int launch_block_prefill(const BlockPrefillParams& p, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    const unsigned grid = (unsigned)((p.grid + 3) / 4);
    if (p.c.bf16) {
        if (p.c.int8) simple_kernel<true, true><<<grid, 128, 0, s>>>(p);
        else simple_kernel<true, false><<<grid, 128, 0, s>>>(p);
    } else {
        if (p.c.int8) simple_kernel<false, true><<<grid, 128, 0, s>>>(p);
        else simple_kernel<false, false><<<grid, 128, 0, s>>>(p);
    }
    return (int)cudaGetLastError();
}

}  // namespace kvarn
