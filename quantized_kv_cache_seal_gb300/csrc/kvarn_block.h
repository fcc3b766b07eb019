// Internal declarations of the block cache (8-bit codes, one scale per block of tokens and
// KV head) and of the query/key norm + rotation, shared by their host side and kernels.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <vector_types.h>

#include "kvarn_internal.h"

namespace kvarn {

constexpr int kTileTokens = 32;      // tokens of a code tile; a block is 1, 2 or 4 tiles
constexpr int kBlockMaxSeqs = 256;   // sequences per call (kernel parameter tables)
constexpr int kBlockMaxRatio = 8;    // query heads per KV head
constexpr int kBlockMaxGrid = 256;   // CTAs of a decode launch
constexpr int kBlockPrefillGrid = 152;  // CTAs of a prefill launch that cuts segments: one a SM

// One code tile: 32 tokens of one KV head, K and V, in the order in which a warp loads the
// A operands of mma.m16n8k16 (16 bytes a lane, 512 contiguous bytes a load):
//   [0,16)             f32 K scale, V scale, log2(V scale), kDenomUnit / V scale
//   [16, 16 + 32 D)    K codes: 512-byte chunk (s D/64 + c) 2 + h, lane 4 g + t: token
//                      8 (g >> 1) + 4 s + 2 h + (g & 1), channels 64 c + 16 t .. + 15
//   [16 + 32 D, ...)   V codes: 512-byte chunk m, lane 4 g + t: tokens 8 t .. 8 t + 7 of
//                      channel 16 m + g, then of channel 16 m + g + 8
KVARN_HD inline int tile_bytes(int d) { return 16 + 2 * kTileTokens * d; }
// byte of K codes for (token of the tile, channel), channel a multiple of 8: 8 codes follow
KVARN_HD inline int k_code_off(int d, int tok, int ch) {
    const int g = ((tok >> 3) << 1) | (tok & 1), s = (tok >> 2) & 1, h = (tok >> 1) & 1;
    const int c16 = ch >> 4, t = c16 & 3, c = c16 >> 2;
    return 16 + ((s * (d >> 6) + c) * 2 + h) * 512 + (g * 4 + t) * 16 + (ch & 15);
}
// byte of V codes for (token of the tile, a multiple of 8; channel): 8 tokens follow
KVARN_HD inline int v_code_off(int d, int tok, int ch) {
    return 16 + kTileTokens * d + (ch >> 4) * 512 + ((ch & 7) * 4 + (tok >> 3)) * 16 + ((ch >> 3) & 1) * 8;
}

// element of the exact V of (row of the block, channel)
KVARN_HD inline int tail_v_off(int d, int row, int ch) { return ((row >> 5) * d + ch) * kTileTokens + (row & 31); }

struct BlockLayout {
    size_t err;       // int32[4]
    size_t table;     // int32[max_seqs][num_layers][max_blocks]: pool slot of each sealed block
    size_t counters;  // int32[kBlockMaxGrid], zero between calls: arrivals at a split (sequence, KV head) of a
                      // decode call; segments taken and CTAs done of a prefill call
    size_t warp_counters;  // int32[kBlockMaxGrid * 8]: the same of a decode call that cuts the line over warps
    size_t partials;  // float[kBlockMaxGrid][2][8 (D + 2)] of a decode call, or
                      // float[kBlockPrefillGrid][2][256 (D + 2)] of a prefill call
    size_t tail_k;    // T[max_seqs][num_layers][Hkv][B][D]: exact rows of the partial block
    size_t tail_v;    // T[max_seqs][num_layers][Hkv][B / 32][D][32]: the same for V, channel rows of each 32 tokens
    size_t pool;      // slots of Hkv * (B / 32) tiles
    size_t total;
};

// What every kernel of the cache is told about it.
struct BlockView {
    uint8_t* base;
    BlockLayout lay;
    int64_t slot_bytes;
    int32_t hkv, d, block, log2_block, num_layers, layer, max_blocks;
    int32_t int8;  // codes: 0 = e4m3, 1 = int8 held as value + 128
    int32_t bf16;  // exact values, inputs and outputs: 0 = fp16, 1 = bf16
};

struct BlockAppendSeq {
    int32_t seq, n_before, n_new;
    int32_t n_blocks;    // blocks this call completes
    int32_t in_row;      // first input row
    int32_t item_begin;  // prefix of max(n_blocks, 1) * Hkv * 2
    int32_t slot_begin;  // first of its entries in slots
};

template <int SEQS, int SLOTS>
struct BlockAppendParams {
    BlockView c;
    const uint16_t *k, *v;
    int64_t k_stride, v_stride;  // elements between tokens
    int32_t n_seqs, items;
    BlockAppendSeq seqs[SEQS];
    int32_t slots[SLOTS];
};
// Kernel parameters are copied at every launch: a call for few sequences passes the small
// form. The large one fits the 32,764 bytes that parameters may take.
using BlockAppendSmall = BlockAppendParams<16, 128>;
using BlockAppendLarge = BlockAppendParams<kBlockMaxSeqs, 5000>;
static_assert(sizeof(BlockAppendLarge) <= 32764, "kernel parameter size");

struct BlockReadSeq {
    int32_t seq, n;            // tokens in the cache
    int32_t start, count;
    int32_t out_row;
    int32_t item_begin;        // prefix of tiles touched * Hkv * 2
};
struct BlockReadParams {
    BlockView c;
    void *k, *v;               // [rows][Hkv][D] of the cache's type, or f32
    int32_t n_seqs, items, f32;
    BlockReadSeq seqs[kBlockMaxSeqs];
};

struct BlockDecodeSeq {
    int32_t seq, n;
    int32_t unit_begin;        // prefix of Hkv * units; a unit is one tile
    int32_t units;             // of each KV head, at least 1
};
struct BlockDecodeParams {
    BlockView c;
    const uint16_t* q;
    uint16_t* out;
    int32_t n_seqs, hq, r, grid;
    int64_t units;
    float scale_log2;          // softmax scale * log2(e)
    BlockDecodeSeq seqs[kBlockMaxSeqs];
};
// Units that a (sequence, KV head) counts beside its tiles where the line is cut over warps: its end, in tiles.
// (64 sequences of 1 to 1,024 tokens, bf16, int8: 42 us with 4, 38 with 8, 40 with 12; fp16, e4m3: 28, 29, 31.)
constexpr int kPairCost = 8;
// What a decode launch with prefixes or weights has beside.
struct BlockDecodeMore {
    int32_t alone;             // 1: the line is cut over the warps
    float2* sums;              // [units][r] or null: maximum and sum of each tile's weights, by head
    float2* totals;            // [rows][Hq] (with sums): of each row over all its keys, a prefix's among them; where merged says, it holds the prefix's before
    const float *pre_o, *pre_lse;  // rows finished over shared prefixes (pre_lse null: none), [rows][Hq][D] and [rows][Hq]
    uint32_t merged[kBlockMaxSeqs / 32];  // bit i: sequence entry i takes its row from there
    int32_t pre[kBlockMaxSeqs], pre_n[kBlockMaxSeqs];  // sequence whose pre_n tokens come before entry i's own (0: none)
};

struct BlockPrefillSeq {
    int32_t seq, n, q_len, q_row;
    int32_t pairs;       // pairs of query tiles (256 / r query tokens at most)
    int32_t seg_begin;   // prefix of pairs * Hkv: segments
    int32_t step_begin;  // prefix of Hkv * head_steps
    int32_t head_steps;  // steps of 128 keys over the pairs of one KV head
};
struct BlockPrefillParams {
    BlockView c;
    const uint16_t* q;
    uint16_t* out;
    int32_t n_seqs, hq, r, grid;
    int32_t line;        // 1: the steps of all segments are cut evenly over the CTAs; 0: CTAs take whole segments
    int32_t steps, segs; // of all sequences and KV heads
    float scale_log2;    // softmax scale * log2(e)
    BlockPrefillSeq seqs[kBlockMaxSeqs];
};
// What a prefill launch with prefixes has beside.
struct BlockPrefillMore {
    int32_t flat;        // 1: every query sees all of the entry's n tokens, and finished rows go to pre_o and pre_lse
    float *pre_o, *pre_lse;  // f32 [rows][Hq][D], [rows][Hq]: written if flat; else added where merged says
    float2* totals;      // [rows][Hq] or null, if flat: a row's maximum and sum, in decode's units
    uint32_t merged[kBlockMaxSeqs / 32];  // bit i: entry i
    int32_t pre[kBlockMaxSeqs];    // a prefix whose steps come first in the segments of entry i (not if flat)
    int32_t pre_n[kBlockMaxSeqs];  // its tokens, 0: none
};

// Queries as tiles of 128 rows (query, head of a KV head) over a sequence in steps of 128 tokens, for each KV head.
struct BlockRowsSeq {
    int32_t seq, n, q_len, q_row;
    int32_t rows;        // q_len * r
    int32_t pad;         // rows rounded up to 8 (window)
    int32_t row_tiles;   // of 128 rows
    int32_t steps;       // of 128 tokens
    int32_t unit_begin;  // prefix of Hkv * row_tiles * steps
    int32_t pair_begin;  // prefix of Hkv * row_tiles
    int64_t sum_begin;   // prefix of Hkv * tiles * pad (window)
    int32_t pre, pre_n;  // window: sequence whose pre_n tokens the rows see before its own, in steps of their own (0: none)
};

// Queries of all sequences behind a shared prefix, which see all of it.
struct BlockFlatParams {
    BlockView c;
    const uint16_t* q;
    float* parts;            // [pairs + grid][2][128 (D + 3)]
    float *pre_o, *pre_lse;  // f32 [rows][Hq][D], [rows][Hq]
    float2* totals;          // [rows][Hq] or null: a row's maximum and sum, in decode's units
    int32_t n_seqs, hq, r, grid;
    int64_t units;           // steps of all sequences, KV heads and row tiles
    float scale_log2;
    BlockRowsSeq seqs[kBlockMaxSeqs];
};
inline size_t flat_part_floats(int d) { return 128 * ((size_t)d + 3); }

// Weights of the last queries of sequences (K alone is read).
constexpr int kWindowParts = 3;  // softmax warpgroups of a launch
struct BlockWindowParams {
    BlockView c;
    const uint16_t* q;
    float2* sums;        // of each sequence [Hkv][tiles][pad]: a tile's maximum and sum, by row
    float2* totals;      // [pairs + grid][kWindowParts][128]: a row's maximum and sum over part of its tokens
    int32_t n_seqs, hq, r, grid;
    int64_t units;
    float scale_log2;
    BlockRowsSeq seqs[kBlockMaxSeqs];
};

// Adds the tiles' weights to what their blocks have received.
struct BlockWeighSeq {
    int32_t seq, rows, pad;   // rows of a KV head, and places for them in a tile's sums
    int32_t before, tiles;    // tiles of a prefix in front, its own
    int32_t stride;           // places for them
    int32_t row;              // decode: of totals
    int32_t unit_begin, pair_begin, steps;  // window: as there
    int64_t sum_begin;
};
struct BlockWeighHead {
    const float2* sums;
    const float2* totals;     // decode (grid 0): [rows][Hq]; window: as there
    float* weights;           // [max_seqs][Hkv][cols]
    int64_t units;            // of the window's line
    int32_t grid;
    int32_t n_seqs, hq, hkv, log2_tiles, cols;  // tiles of a block; places of a (sequence, KV head)
    int32_t lanes, blocks;    // lanes that add up a block, blocks of a CTA
    int32_t most;             // CTAs of a (sequence, KV head)
};
template <int SEQS>
struct BlockWeighArgs : BlockWeighHead {
    BlockWeighSeq seqs[SEQS];
};
// (parameters are copied at every launch: few sequences pass a small form)
using BlockWeighParams = BlockWeighArgs<kBlockMaxSeqs>;

struct BlockEvictSeq {
    int32_t seq, full;        // full blocks, more than keep
    int32_t row;              // of kept
};
struct BlockEvictParams {
    BlockView c;
    float* weights;           // [max_seqs][Hkv][cols]
    int32_t* kept;            // [sequences of the call][Hkv][keep]
    int32_t keep, first, last, cols;
    int32_t n_seqs, n_all;    // entries to cut; of all in the call, which come first in seqs
    BlockEvictSeq seqs[kBlockMaxSeqs];
};

struct QkParams {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;  // elements between tokens
    const float *q_weight, *k_weight;
    const int32_t* positions;
    const double* freqs;
    int64_t n_tokens;
    int32_t hq, hkv, d, rot, interleaved, in_bf16, out_bf16;
    int32_t heads_per_item, items_per_token;
    float eps, inv_d;
    int32_t several;      // 1: pair i turns by positions[axes[i] * axis_stride + token], axes a byte a pair
    int64_t axis_stride;  // elements
    uint32_t axes[32];
};

// Launchers: 0 on success, else a cudaError_t value.
int launch_block_append(const BlockAppendSmall& p, void* stream);
int launch_block_append(const BlockAppendLarge& p, void* stream);
int launch_block_read(const BlockReadParams& p, void* stream);
int launch_block_decode(const BlockDecodeParams& p, void* stream);
int launch_block_decode(const BlockDecodeParams& p, const BlockDecodeMore& more, void* stream);
int launch_block_prefill(const BlockPrefillParams& p, void* stream);
int launch_block_prefill(const BlockPrefillParams& p, const BlockPrefillMore& more, void* stream);
int launch_block_flat(const BlockFlatParams& p, int pairs, void* stream);
int launch_block_window(const BlockWindowParams& p, void* stream);
int launch_block_weigh(const BlockWeighParams& p, void* stream);
int launch_block_evict(const BlockEvictParams& p, void* stream);
int launch_block_init(const BlockView& c, void* stream);
int launch_block_clear_errors(const BlockView& c, void* stream);  // the error word and the counters
int launch_qk_norm_rope(const QkParams& p, void* stream);
int stream_capturing(void* stream, int* capturing);

// the calling thread's kvarn_last_error text (kvarn_host.cpp)
void set_last_error(const char* text);

}  // namespace kvarn
