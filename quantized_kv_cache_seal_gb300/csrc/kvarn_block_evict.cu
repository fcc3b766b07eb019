// Block cache: eviction. Each KV head of a sequence keeps `keep` of its full blocks: the first and last ones asked for,
// and of the others those with the largest weights (ties: the lowest index), in their order; the partial block stays.
// All heads keep as many, so that the sequence stays one of whole blocks: a head's j-th block moves into its place
// in the j-th slot, record by record as it is (no code is made anew), and the host knows which slots are free without
// asking the GPU.
//
// select_kernel, a CTA a (KV head, sequence): the smallest weight that stays by radix (four turns of eight bits over the
// weights' bit patterns in order), then the blocks in order, 1024 at a time, with their weights moved along.
// move_kernel, a thread 16 bytes of a slot: its pieces in order, eight loads ahead of their stores. Places only go
// down (block s_j to j <= s_j, s_j rising), and all that a thread writes it alone reads, so nothing is read after it
// has been written over: a load s_i follows a store to j < i only where s_i >= i > j.
//
// Measured: 16 ragged sequences of up to 16k, 10 heads, int8, cut to 64 blocks of 64: select 8 us, move 40 us for 124 MB read and written (6.2 TB/s).
#include "kvarn_block_dev.cuh"

namespace kvarn {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kMoveThreads = 256, kMoveAhead = 8;

// Weights as whole numbers of the same order; NaN below all.
__device__ __forceinline__ uint32_t rank_of(float w) {
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);  // -0 is 0
    return w != w ? 0u : u >> 31 ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ BlockEvictParams p) {
    __shared__ int counts[kSelWarps][256];
    __shared__ int found[2];
    __shared__ int warp_sum[2][kSelWarps];
    before_done();
    start_next();
    const BlockEvictSeq& e = p.seqs[blockIdx.y];
    const int h = blockIdx.x, t = threadIdx.x, w = t >> 5, lane = t & 31, full = e.full;
    int32_t* kept = p.kept + ((int64_t)e.row * p.c.hkv + h) * p.keep;
    if (full <= p.keep) {
        for (int i = t; i < p.keep; i += kSelThreads) kept[i] = i < full ? i : -1;
        return;
    }
    float* weights = p.weights + ((int64_t)e.seq * p.c.hkv + h) * p.cols;
    // the need-th largest of the blocks between the first and the last ones
    const int lo = p.first, hi = full - p.last;
    int need = p.keep - p.first - p.last;
    uint32_t at = 0;  // its leading bits
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = t; i < kSelWarps * 256; i += kSelThreads) (&counts[0][0])[i] = 0;
            __syncthreads();
            for (int i = lo + t; i < hi; i += kSelThreads) {
                const uint32_t k = rank_of(weights[i]);
                if (shift == 24 || (k ^ at) >> (shift + 8) == 0) atomicAdd(&counts[w][k >> shift & 255], 1);
            }
            __syncthreads();
            if (t < 256) {
                int n = 0;
                for (int z = 0; z < kSelWarps; ++z) n += counts[z][t];
                counts[0][t] = n;
            }
            __syncthreads();
            if (w == 0) {  // bins from the top, eight a lane
                int n[8], sum = 0;
#pragma unroll
                for (int z = 0; z < 8; ++z) sum += n[z] = counts[0][255 - 8 * lane - z];
                int before = sum;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, before, d);
                    if (lane >= d) before += x;
                }
                before -= sum;
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                    if (before < need && before + n[z] >= need) {
                        found[0] = 255 - 8 * lane - z;
                        found[1] = need - before;
                    }
                    before += n[z];
                }
            }
            __syncthreads();
            at |= (uint32_t)found[0] << shift;
            need = found[1];
            __syncthreads();
        }
    }
    // the blocks that stay, in order: weights above `at`, and the first `need` of those at it
    const float rest = weights[full];  // the partial block's (full < cols: there is a place for it)
    int kept_before = 0, same_before = 0;
    for (int i0 = 0; i0 < full; i0 += kSelThreads) {
        const int i = i0 + t;
        const bool in = i < full, middle = in && i >= lo && i < hi;
        const float x = in ? weights[i] : 0.f;
        const uint32_t k = rank_of(x);
        const bool same = middle && k == at && need > 0;
        const unsigned sm = __ballot_sync(0xffffffffu, same);
        if (lane == 0) warp_sum[0][w] = __popc(sm);
        __syncthreads();
        int before = same_before, all = same_before;
#pragma unroll
        for (int z = 0; z < kSelWarps; ++z) {
            if (z < w) before += warp_sum[0][z];
            all += warp_sum[0][z];
        }
        same_before = all;
        before += __popc(sm & ((1u << lane) - 1));
        const bool stays = in && (!middle || (p.keep > p.first + p.last && (k > at || (same && before < need))));
        const unsigned km = __ballot_sync(0xffffffffu, stays);
        if (lane == 0) warp_sum[1][w] = __popc(km);
        __syncthreads();
        int place = kept_before + __popc(km & ((1u << lane) - 1));
        all = kept_before;
#pragma unroll
        for (int z = 0; z < kSelWarps; ++z) {
            if (z < w) place += warp_sum[1][z];
            all += warp_sum[1][z];
        }
        kept_before = all;
        if (stays) {  // place <= i: of these 1024 weights all are read, of later ones none is touched
            kept[place] = i;
            weights[place] = x;
        }
        __syncthreads();
    }
    for (int i = p.keep + t; i <= full; i += kSelThreads) weights[i] = i == p.keep ? rest : 0.f;
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ BlockEvictParams p) {
    before_done();
    const BlockEvictSeq& e = p.seqs[blockIdx.y];
    const int per = (p.c.block / kTileTokens) * tile_bytes(p.c.d) / 16;  // pieces of a head's record
    const int piece = blockIdx.x * kMoveThreads + threadIdx.x;
    if (piece >= per * p.c.hkv) return;
    const int32_t* kept = p.kept + ((int64_t)e.row * p.c.hkv + piece / per) * p.keep;
    const int32_t* table = block_table(p.c, e.seq);
    uint4* pool = reinterpret_cast<uint4*>(p.c.base + p.c.lay.pool) + piece;
    const int64_t slot = p.c.slot_bytes / 16;
#pragma unroll 1
    for (int j0 = 0; j0 < p.keep; j0 += kMoveAhead) {
        uint4 x[kMoveAhead];
        int to[kMoveAhead];  // -1: stays
#pragma unroll
        for (int z = 0; z < kMoveAhead; ++z) {
            const int from = j0 + z < p.keep ? kept[j0 + z] : j0 + z;
            to[z] = -1;
            if (from != j0 + z) {
                to[z] = read<true>(table + j0 + z);
                x[z] = pool[read<true>(table + from) * slot];
            }
        }
#pragma unroll
        for (int z = 0; z < kMoveAhead; ++z)
            if (to[z] >= 0) pool[to[z] * slot] = x[z];
    }
}

}  // namespace

int launch_block_evict(const BlockEvictParams& p, void* stream) {
    cudaStream_t s = (cudaStream_t)stream;
    const int rc = launch_behind(select_kernel, dim3(p.c.hkv, p.n_all), kSelThreads, 0, s, p);
    if (rc == 0 && p.n_seqs > 0) {
        const int pieces = p.c.hkv * ((p.c.block / kTileTokens) * tile_bytes(p.c.d) / 16);
        return launch_behind(move_kernel, dim3((pieces + kMoveThreads - 1) / kMoveThreads, p.n_seqs), kMoveThreads, 0, s, p);
    }
    return rc;
}

}  // namespace kvarn
