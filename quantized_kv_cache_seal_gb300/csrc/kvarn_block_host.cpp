// Host side of the block cache and of the query/key norm + rotation: argument checks, the
// host mirror of sequence lengths and pool slots, launch parameters, and the C ABI.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <memory>
#include <new>
#include <vector>

#include "../../include/kvarn.h"
#include "kvarn_block.h"

using namespace kvarn;

struct kvarn_block_cache {
    kvarn_block_config cfg;
    BlockView view;
    int r = 1;
    std::vector<int32_t> len;         // [max_seqs][num_layers]
    std::vector<int32_t> table;       // [max_seqs][num_layers][max_blocks]
    std::vector<int32_t> free_slots;  // stack of free pool slots
    std::vector<char> seen;           // scratch of check_ids, all zero between calls
    bool initialized = false;
    bool host_only = false;
    int device = -1;
    int sms = 152;

    int32_t& L(int seq, int layer) { return len[(size_t)seq * cfg.num_layers + layer]; }
    int32_t* T(int seq, int layer) { return &table[((size_t)seq * cfg.num_layers + layer) * view.max_blocks]; }
};

namespace {

kvarn_status fail(kvarn_status st, const char* text) {
    set_last_error(text);
    return st;
}

kvarn_status cuda_fail(int rc, const char* what) {
    char text[256];
    std::snprintf(text, sizeof(text), "%s: %s (%d)", what, cuda_error_string(rc), rc);
    return fail(KVARN_ECUDA, text);
}

constexpr int kWindowTokens = 128;   // queries of a sequence in window_weights
constexpr int kSmallRows = 1 << 22;  // bytes
constexpr int kOwnSteps = 18;        // of each SM: what a pass over the prefixes takes beside its steps
constexpr int kChangeSteps = 4;      // of an SM: what a change of segment takes
constexpr float kLog2e = 1.4426950408889634f;

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Device layout of a cache; false if the sizes leave what an address can hold.
bool make_view(const kvarn_block_config& c, BlockView* v) {
    std::memset(v, 0, sizeof(*v));
    v->hkv = c.num_kv_heads;
    v->d = c.head_dim;
    v->block = c.block_tokens;
    v->log2_block = c.block_tokens == 32 ? 5 : c.block_tokens == 64 ? 6 : 7;
    v->num_layers = c.num_layers;
    v->max_blocks = std::max(1, c.max_seq_len / c.block_tokens);
    v->int8 = c.code == KVARN_CODE_INT8;
    v->bf16 = c.type == KVARN_TYPE_BF16;
    v->slot_bytes = (int64_t)c.num_kv_heads * (c.block_tokens / kTileTokens) * tile_bytes(c.head_dim);
    unsigned __int128 off = 0;
    auto take = [&](unsigned __int128 n) {
        const unsigned __int128 o = off;
        off = (off + n + 255) / 256 * 256;
        return (size_t)o;
    };
    typedef unsigned __int128 U;
    const U seq_layers = (U)c.max_seqs * c.num_layers;
    const U tail = seq_layers * c.num_kv_heads * c.block_tokens * c.head_dim * 2;
    v->lay.err = take(16);
    v->lay.table = take(seq_layers * v->max_blocks * 4);
    v->lay.counters = take(kBlockMaxGrid * 4);
    v->lay.warp_counters = take(kBlockMaxGrid * 8 * 4);
    v->lay.partials = take((U)std::max(kBlockMaxGrid * kBlockMaxRatio, kBlockPrefillGrid * 256) * 2 * (c.head_dim + 2) * 4);
    v->lay.tail_k = take(tail);
    v->lay.tail_v = take(tail);
    v->lay.pool = take((U)c.pool_blocks * (U)v->slot_bytes);
    v->lay.total = (size_t)off;
    return off < ((U)1 << 46);
}

kvarn_status check_config(const kvarn_block_config* c) {
    if (!c) return fail(KVARN_EINVAL, "no configuration");
    if (c->num_layers <= 0 || c->max_seqs <= 0 || c->num_kv_heads <= 0 || c->num_q_heads <= 0 || c->max_seq_len <= 0 ||
        c->pool_blocks < 0)
        return fail(KVARN_EINVAL, "sizes must be positive");
    if (c->head_dim != 64 && c->head_dim != 128) return fail(KVARN_EINVAL, "head_dim must be 64 or 128");
    if (c->block_tokens != 32 && c->block_tokens != 64 && c->block_tokens != 128)
        return fail(KVARN_EINVAL, "block_tokens must be 32, 64 or 128");
    if (c->code != KVARN_CODE_E4M3 && c->code != KVARN_CODE_INT8) return fail(KVARN_EINVAL, "unknown code");
    if (c->type != KVARN_TYPE_F16 && c->type != KVARN_TYPE_BF16) return fail(KVARN_EINVAL, "unknown type");
    if (c->num_q_heads % c->num_kv_heads || c->num_q_heads / c->num_kv_heads > kBlockMaxRatio)
        return fail(KVARN_EINVAL, "num_q_heads must be 1 to 8 times num_kv_heads");
    if ((c->flags & ~KVARN_FLAG_HOST_ONLY) != 0) return fail(KVARN_EINVAL, "unknown flag");
    if ((int64_t)c->max_seqs * c->num_layers > (1ll << 31) - 1 || c->num_kv_heads > (1 << 16) || c->max_seq_len > (1 << 30))
        return fail(KVARN_EINVAL, "too many sequences, layers or heads, or max_seq_len above 2^30");
    return KVARN_OK;
}

// A call's layer and sequences; `changes`: the call moves the cache on, which a captured
// graph would do again at each replay without the host's lengths following.
kvarn_status check_call(kvarn_block_cache* c, int32_t layer, int32_t n, const int32_t* ids, void* stream, bool changes) {
    if (!c) return fail(KVARN_EINVAL, "no cache");
    if (layer < 0 || layer >= c->cfg.num_layers) return fail(KVARN_EINVAL, "no such layer");
    if (n < 0 || (n > 0 && !ids)) return fail(KVARN_EINVAL, "bad sequence list");
    if (n > kBlockMaxSeqs) return fail(KVARN_ECAPACITY, "more than 256 sequences in a call");
    kvarn_status st = KVARN_OK;
    int i = 0;
    for (; i < n; ++i) {
        if (ids[i] < 0 || ids[i] >= c->cfg.max_seqs || c->seen[ids[i]]) {
            st = fail(KVARN_EINVAL, "a sequence id is out of range or given twice");
            break;
        }
        c->seen[ids[i]] = 1;
    }
    for (int j = 0; j < i; ++j) c->seen[ids[j]] = 0;
    if (st || c->host_only) return st;
    int dev = -1;
    int rc = current_device(&dev);
    if (rc) return cuda_fail(rc, "current device");
    if (dev != c->device) return fail(KVARN_EINVAL, "the current device is not the one that holds the cache");
    if (changes || !c->initialized) {
        int capturing = 0;
        rc = stream_capturing(stream, &capturing);
        if (rc) return cuda_fail(rc, "capture state");
        if (capturing) return fail(KVARN_ESTATE, "a call that changes the cache (or is its first) cannot be captured");
    }
    return KVARN_OK;
}

kvarn_status ensure_init(kvarn_block_cache* c, void* stream) {
    if (c->host_only || c->initialized) return KVARN_OK;
    const int rc = launch_block_init(c->view, stream);
    if (rc) return cuda_fail(rc, "cache init");
    c->initialized = true;
    return KVARN_OK;
}

kvarn_status check_append(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* n_tokens,
                          const void* k, const void* v, int64_t k_stride, int64_t v_stride) {
    if (n_seqs > 0 && !n_tokens) return fail(KVARN_EINVAL, "no token counts");
    const int bt = c->cfg.block_tokens;
    int64_t total = 0, blocks = 0;
    for (int i = 0; i < n_seqs; ++i) {
        if (n_tokens[i] < 0) return fail(KVARN_EINVAL, "a token count is negative");
        const int64_t n0 = c->L(ids[i], layer), n1 = n0 + n_tokens[i];
        if (n1 > c->cfg.max_seq_len) return fail(KVARN_ECAPACITY, "a sequence would exceed max_seq_len");
        total += n_tokens[i];
        blocks += n1 / bt - n0 / bt;
    }
    if (total >= 1ll << 31) return fail(KVARN_ECAPACITY, "2^31 tokens or more in a call");
    if ((size_t)blocks > c->free_slots.size()) return fail(KVARN_ECAPACITY, "the pool has too few free blocks");
    if (total == 0) return KVARN_OK;
    const int64_t row = (int64_t)c->cfg.num_kv_heads * c->cfg.head_dim;
    if (!k || !v || !aligned16(k) || !aligned16(v)) return fail(KVARN_EINVAL, "k and v must be 16-byte aligned");
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8)
        return fail(KVARN_EINVAL, "token strides must hold a token's heads and be multiples of 8 elements");
    return KVARN_OK;
}

template <class P>
kvarn_status launch_append(kvarn_block_cache* c, const P& p, void* stream) {
    if (c->host_only || p.items == 0) return KVARN_OK;
    const int rc = launch_block_append(p, stream);
    return rc ? cuda_fail(rc, "append launch") : KVARN_OK;
}

// Append after its checks: launches of as many tokens as the parameters hold slots for. A
// sequence may be cut between launches at any token (the result does not depend on it).
template <class P>
kvarn_status run_append(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* n_tokens,
                        const void* k, const void* v, int64_t k_stride, int64_t v_stride, void* stream, int max_slots) {
    const int bt = c->cfg.block_tokens;
    static thread_local P p;
    p.c = c->view;
    p.c.layer = layer;
    p.k = (const uint16_t*)k;
    p.v = (const uint16_t*)v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_seqs = p.items = 0;
    int slots = 0;
    int64_t row = 0;
    for (int i = 0; i < n_seqs; ++i) {
        int32_t left = n_tokens[i];
        while (left > 0) {
            int32_t& n0 = c->L(ids[i], layer);
            const int room = max_slots - slots;
            // blocks and items that fit (items stay far below 2^31: max_slots * Hkv * 2)
            const int32_t take = (int32_t)std::min<int64_t>(left, (int64_t)(n0 / bt + room) * bt + bt - 1 - n0);
            BlockAppendSeq& e = p.seqs[p.n_seqs++];
            e.seq = ids[i];
            e.n_before = n0;
            e.n_new = take;
            e.n_blocks = (n0 + take) / bt - n0 / bt;
            e.in_row = (int32_t)row;
            e.item_begin = p.items;
            e.slot_begin = slots;
            int32_t* t = c->T(ids[i], layer) + n0 / bt;
            for (int j = 0; j < e.n_blocks; ++j) {
                p.slots[slots++] = t[j] = c->free_slots.back();
                c->free_slots.pop_back();
            }
            p.items += std::max(e.n_blocks, 1) * c->cfg.num_kv_heads * 2;
            n0 += take;
            row += take;
            left -= take;
            if (left > 0) {  // the parameters are full
                const kvarn_status st = launch_append(c, p, stream);
                if (st) return st;
                p.n_seqs = p.items = slots = 0;
            }
        }
    }
    return launch_append(c, p, stream);
}

kvarn_status append(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* n_tokens,
                    const void* k, const void* v, int64_t k_stride, int64_t v_stride, void* stream) {
    kvarn_status st = ensure_init(c, stream);
    if (st) return st;
    const int bt = c->cfg.block_tokens;
    int64_t blocks = 0;
    for (int i = 0; i < n_seqs; ++i) {
        const int64_t n0 = c->L(ids[i], layer);
        blocks += (n0 + n_tokens[i]) / bt - n0 / bt;
    }
    if (n_seqs <= 16 && blocks <= 128)
        return run_append<BlockAppendSmall>(c, layer, n_seqs, ids, n_tokens, k, v, k_stride, v_stride, stream, 128);
    return run_append<BlockAppendLarge>(c, layer, n_seqs, ids, n_tokens, k, v, k_stride, v_stride, stream, 5000);
}

// The work of a sequence of n tokens in an attention launch: tiles of a KV head for the single-token kernel,
// query tile pairs of a KV head and their steps of 128 keys for the many-query one.
int32_t tiles_of(int64_t n) { return (int32_t)((n + kTileTokens - 1) / kTileTokens); }
int32_t head_tiles(int64_t n) { return (int32_t)std::max<int64_t>(1, (n + kTileTokens - 1) / kTileTokens); }
int64_t key_steps(int64_t n) { return (n + 127) / 128; }
int64_t head_pairs(const kvarn_block_cache* c, int64_t q_len) {
    const int pair_tokens = 2 * (128 / c->r);
    return (q_len + pair_tokens - 1) / pair_tokens;
}
int64_t head_steps(const kvarn_block_cache* c, int64_t n, int64_t q_len) {
    const int64_t pair_tokens = 2 * (128 / c->r);
    int64_t steps = 0;
    for (int64_t end = pair_tokens; end < q_len + pair_tokens; end += pair_tokens)
        steps += (n - q_len + std::min(end, q_len) - 1) / 128 + 1;
    return steps;
}
// Flags as a mask of bits.
void mark(uint32_t* mask, const uint8_t* flags, int n) {
    std::memset(mask, 0, kBlockMaxSeqs / 8);
    for (int i = 0; flags && i < n; ++i) mask[i / 32] |= (uint32_t)(flags[i] != 0) << i % 32;
}
// One query a sequence at most: the single-token kernel, whose rows are these queries.
bool single_queries(int32_t n_seqs, const int32_t* q_lens) {
    return std::all_of(q_lens, q_lens + n_seqs, [](int32_t m) { return m <= 1; });
}

kvarn_status check_attention(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* q_lens,
                             const int32_t* added, const void* q, const void* out, float scale) {
    if (!std::isfinite(scale * kLog2e)) return fail(KVARN_EINVAL, "softmax_scale must be finite, below 2^127");
    const bool single = !q_lens || single_queries(n_seqs, q_lens);
    int64_t rows = 0, work = 0;  // work: tiles or steps of a KV head
    for (int i = 0; i < n_seqs; ++i) {
        const int64_t n = c->L(ids[i], layer) + (added ? (int64_t)added[i] : 0);
        const int64_t m = q_lens ? q_lens[i] : 1;
        if (q_lens && (m < 0 || m > n)) return fail(KVARN_EINVAL, "a query count is negative or above the sequence's length");
        rows += m;
        if (single) work += m > 0 ? head_tiles(n) : 0;
        else work += m > 0 ? head_pairs(c, m) * ((n - 1) / 128 + 1) : 0;
    }
    if (rows * c->cfg.num_q_heads >= 1ll << 31) return fail(KVARN_ECAPACITY, "2^31 query rows or more in a call");
    if (!single && work * c->cfg.num_kv_heads >= 1ll << 31) {  // every pair counted as long as the last: now exactly
        work = 0;
        for (int i = 0; i < n_seqs; ++i)
            work += head_steps(c, c->L(ids[i], layer) + (added ? (int64_t)added[i] : 0), q_lens[i]);
    }
    if (work * c->cfg.num_kv_heads >= 1ll << 31)
        return fail(KVARN_ECAPACITY, single ? "2^31 tiles of 32 tokens or more in a call"
                                            : "2^31 steps of 128 keys or more in a call");
    if (rows > 0 && (!q || !out || !aligned16(q) || !aligned16(out)))
        return fail(KVARN_EINVAL, "q and out must be 16-byte aligned");
    // A row of out is written once every reader of the same row of q is through with it, and only then.
    const uint64_t bytes = (uint64_t)rows * c->cfg.num_q_heads * c->cfg.head_dim * 2;
    if (q != out && (uintptr_t)q < (uintptr_t)out + bytes && (uintptr_t)out < (uintptr_t)q + bytes)
        return fail(KVARN_EINVAL, "out overlaps q (it may only be q itself)");
    return KVARN_OK;
}

// What an attention call may have beside its own tokens, sequence by sequence.
struct Beside {
    const int32_t* before = nullptr;   // a prefix whose tokens come first in the sequence's line, -1 for none
    const uint8_t* finished = nullptr; // 1: its rows over a prefix are in pre_o and pre_lse
    float *pre_o = nullptr, *pre_lse = nullptr;
    float2 *sums = nullptr, *totals = nullptr;  // decode: the tiles' sums, the rows' (the prefixes' pass leaves its part there)
    float* weights = nullptr;          // decode: what the blocks have received, added to
};

size_t columns(const kvarn_block_cache* c) { return (size_t)(c->cfg.max_seq_len / c->cfg.block_tokens) + 1; }

kvarn_status run_weigh(kvarn_block_cache* c, BlockWeighParams& p, void* stream) {
    p.hq = c->cfg.num_q_heads;
    p.hkv = c->cfg.num_kv_heads;
    p.log2_tiles = c->view.log2_block - 5;
    p.cols = (int32_t)columns(c);
    // Lanes enough for a block's sums two at a time; a CTA one round of blocks, or more where that still makes four CTAs
    // a SM: every CTA looks its rows' totals up.
    int32_t pad = 1, tiles = 1;
    int64_t blocks = 0;
    for (int i = 0; i < p.n_seqs; ++i) {
        pad = std::max(pad, p.seqs[i].pad);
        tiles = std::max(tiles, p.seqs[i].tiles);
        blocks += (int64_t)p.hkv * (((p.seqs[i].tiles - 1) >> p.log2_tiles) + 1);
    }
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes * 2 < pad << p.log2_tiles) p.lanes *= 2;
    p.blocks = 256 / p.lanes;
    while (p.blocks < 8 * 256 / p.lanes && blocks / (2 * p.blocks) > 4 * c->sms) p.blocks *= 2;
    p.most = (((tiles - 1) >> p.log2_tiles) + p.blocks) / p.blocks;
    const int rc = launch_block_weigh(p, stream);
    return rc ? cuda_fail(rc, "weights launch") : KVARN_OK;
}

kvarn_status run_decode(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const void* q, void* out,
                        float scale, void* stream, const Beside& beside = Beside()) {
    static thread_local BlockDecodeParams p;
    static thread_local BlockDecodeMore x;
    const bool more = beside.before || beside.finished || beside.sums;
    p.c = c->view;
    p.c.layer = layer;
    p.q = (const uint16_t*)q;
    p.out = (uint16_t*)out;
    p.n_seqs = n_seqs;
    p.hq = c->cfg.num_q_heads;
    p.r = c->r;
    p.scale_log2 = scale * kLog2e;
    int64_t units = 0;
    for (int i = 0; i < n_seqs; ++i) {
        BlockDecodeSeq& e = p.seqs[i];
        e.seq = ids[i];
        e.n = c->L(ids[i], layer);
        e.unit_begin = (int32_t)units;
        e.units = head_tiles(e.n);
        if (more) {
            x.pre[i] = beside.before ? beside.before[i] : -1;
            x.pre_n[i] = x.pre[i] >= 0 ? c->L(x.pre[i], layer) : 0;
            if (x.pre_n[i] > 0) e.units = tiles_of(x.pre_n[i]) + tiles_of(e.n);
        }
        units += (int64_t)e.units * c->cfg.num_kv_heads;
    }
    p.units = units;
    if (more) {
        x.sums = beside.sums;
        x.totals = beside.totals;
        x.pre_o = beside.pre_o;
        x.pre_lse = beside.pre_lse;
        mark(x.merged, beside.finished, n_seqs);
    }
    // One CTA a SM, each of its eight warps a unit at least. Equal short sequences: whole (sequence, KV
    // head) pairs, so that nothing is joined across CTAs (which takes about as long as four rounds).
    const int64_t pairs = (int64_t)n_seqs * c->cfg.num_kv_heads, most = std::min(c->sms, kBlockMaxGrid);
    const bool equal = std::all_of(p.seqs, p.seqs + n_seqs, [](const BlockDecodeSeq& e) { return e.units == p.seqs[0].units; });
    p.grid = (int32_t)(equal && p.seqs[0].units <= 32 && pairs <= most ? pairs : std::min((units + 7) / 8, most));
    // Short pairs, a tile a warp at least: the line is cut over the warps. (Measured with weights, 32 / 8 heads of 128, us
    // over warps and over CTAs: 64 ragged sequences of up to 1,024 tokens 28 and 87, of up to 256 21 and 44; 200 of up to 40 26 and 42;
    // 64 of 2,048 57 and 59; 8 of 4,096 22 and 23; 16 of 8,192 59 and 58, of 32,768 195 and 182.)
    x.alone = more && units >= 8 * most && units < 128 * pairs;
    if (x.alone) {
        units = 0;
        for (int i = 0; i < n_seqs; ++i) {
            p.seqs[i].unit_begin = (int32_t)units;
            p.seqs[i].units += kPairCost;
            units += (int64_t)p.seqs[i].units * c->cfg.num_kv_heads;
        }
        p.units = units;
        p.grid = (int32_t)most;
    }
    if (c->host_only) return KVARN_OK;
    const kvarn_status st = ensure_init(c, stream);
    if (st) return st;
    const int rc = more ? launch_block_decode(p, x, stream) : launch_block_decode(p, stream);
    if (rc) return cuda_fail(rc, "decode launch");
    if (!beside.weights) return KVARN_OK;
    static thread_local BlockWeighParams wp;
    wp.sums = beside.sums;
    wp.totals = beside.totals;
    wp.weights = beside.weights;
    wp.units = wp.grid = 0;
    wp.n_seqs = n_seqs;
    for (int i = 0; i < n_seqs; ++i) {
        const BlockDecodeSeq& e = p.seqs[i];
        BlockWeighSeq& s = wp.seqs[i];
        s.seq = e.seq;
        s.rows = s.pad = c->r;
        s.before = tiles_of(x.pre_n[i]);
        s.tiles = e.units - s.before - (x.alone ? kPairCost : 0);
        s.stride = e.units;
        s.row = i;
        s.unit_begin = s.pair_begin = s.steps = 0;
        s.sum_begin = (int64_t)e.unit_begin * c->r;
    }
    return run_weigh(c, wp, stream);
}

// Queries in rows of their own order, each entry's `q_len` of them over `n` tokens of sequence `seq`: all of them if
// `flat` (rows go to pre_o and pre_lse), else causally.
struct Entry {
    int32_t seq, n, q_len, q_row;
    int32_t before;  // as Beside's
    uint8_t finished;
};

kvarn_status run_tiles(kvarn_block_cache* c, int32_t layer, int32_t n_entries, const Entry* entries, bool flat, const void* q,
                       void* out, float scale, void* stream, const Beside& beside);

kvarn_status run_prefill(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* q_lens,
                         const void* q, void* out, float scale, void* stream, const Beside& beside = Beside()) {
    if (single_queries(n_seqs, q_lens)) {
        int32_t one[kBlockMaxSeqs], before[kBlockMaxSeqs];
        uint8_t finished[kBlockMaxSeqs];
        int32_t n = 0;
        for (int i = 0; i < n_seqs; ++i)
            if (q_lens[i] == 1) {
                if (beside.before) before[n] = beside.before[i];
                if (beside.finished) finished[n] = beside.finished[i];
                one[n++] = ids[i];
            }
        Beside b = beside;
        if (b.before) b.before = before;
        if (b.finished) b.finished = finished;
        return n ? run_decode(c, layer, n, one, q, out, scale, stream, b) : KVARN_OK;
    }
    Entry entries[kBlockMaxSeqs];
    int64_t row = 0;
    for (int i = 0; i < n_seqs; ++i) {
        entries[i] = Entry{ids[i], c->L(ids[i], layer), q_lens[i], (int32_t)row, beside.before ? beside.before[i] : -1,
                           (uint8_t)(beside.finished && beside.finished[i])};
        row += q_lens[i];
    }
    return run_tiles(c, layer, n_seqs, entries, false, q, out, scale, stream, beside);
}

// The prefixes' pass on single row tiles, where its parts have room; `done` says so.
kvarn_status run_flat(kvarn_block_cache* c, int32_t layer, int32_t n_entries, const Entry* entries, const void* q, float scale,
                      void* stream, const Beside& beside, bool* done) {
    static thread_local BlockFlatParams p;
    const int hkv = c->cfg.num_kv_heads;
    int64_t units = 0, pairs = 0;
    for (int i = 0; i < n_entries; ++i) {
        BlockRowsSeq& e = p.seqs[i];
        const int64_t rows = (int64_t)entries[i].q_len * c->r, tiles = (rows + 127) / 128, steps = ((int64_t)entries[i].n + 127) / 128;
        e = BlockRowsSeq{entries[i].seq, entries[i].n, entries[i].q_len, entries[i].q_row, (int32_t)rows, 0, (int32_t)tiles,
                         (int32_t)steps, (int32_t)units, (int32_t)pairs, 0};
        units += hkv * tiles * steps;
        pairs += hkv * tiles;
        if (units >= 1ll << 31 || pairs > kBlockPrefillGrid) return KVARN_OK;
    }
    p.grid = (int32_t)std::min<int64_t>(std::min(c->sms, kBlockPrefillGrid), units);
    const size_t room = (size_t)kBlockPrefillGrid * 2 * 256 * (c->cfg.head_dim + 2);
    if ((size_t)(pairs + p.grid) * 2 * flat_part_floats(c->cfg.head_dim) > room) return KVARN_OK;
    *done = true;
    if (c->host_only) return KVARN_OK;
    const kvarn_status st = ensure_init(c, stream);
    if (st) return st;
    p.c = c->view;
    p.c.layer = layer;
    p.q = (const uint16_t*)q;
    p.parts = (float*)(c->view.base + c->view.lay.partials);
    p.pre_o = beside.pre_o;
    p.pre_lse = beside.pre_lse;
    p.totals = beside.totals;
    p.n_seqs = n_entries;
    p.hq = c->cfg.num_q_heads;
    p.r = c->r;
    p.units = units;
    p.scale_log2 = scale * kLog2e;
    const int rc = launch_block_flat(p, (int)pairs, stream);
    return rc ? cuda_fail(rc, "prefix launch") : KVARN_OK;
}

kvarn_status run_tiles(kvarn_block_cache* c, int32_t layer, int32_t n_entries, const Entry* entries, bool flat, const void* q,
                       void* out, float scale, void* stream, const Beside& beside) {
    if (flat) {
        bool done = false;
        const kvarn_status st = run_flat(c, layer, n_entries, entries, q, scale, stream, beside, &done);
        if (st || done) return st;
    }
    static thread_local BlockPrefillParams p;
    static thread_local BlockPrefillMore x;
    p.c = c->view;
    p.c.layer = layer;
    p.q = (const uint16_t*)q;
    p.out = (uint16_t*)out;
    p.hq = c->cfg.num_q_heads;
    p.r = c->r;
    p.scale_log2 = scale * kLog2e;
    p.n_seqs = 0;
    const int hkv = c->cfg.num_kv_heads;
    for (int i = 0; i < n_entries; ++i) {
        if (entries[i].q_len == 0) continue;
        BlockPrefillSeq& e = p.seqs[p.n_seqs++];
        e.seq = entries[i].seq;
        e.n = entries[i].n;
        e.q_len = entries[i].q_len;
        e.q_row = entries[i].q_row;
        // (until they are counted below)
        e.pairs = entries[i].finished;
        e.seg_begin = flat ? -1 : entries[i].before;
        e.step_begin = e.seg_begin >= 0 ? c->L(e.seg_begin, layer) : 0;
    }
    if (p.n_seqs == 0) return KVARN_OK;
    // the longest sequences first: their segments are the longest
    std::sort(p.seqs, p.seqs + p.n_seqs, [](const BlockPrefillSeq& a, const BlockPrefillSeq& b) {
        return (int64_t)a.n + a.step_begin > (int64_t)b.n + b.step_begin;
    });
    const bool more = beside.pre_lse || beside.before;
    uint8_t finished[kBlockMaxSeqs];
    int64_t segs = 0, steps = 0, longest = 0, n_long = 0;
    for (int i = 0; i < p.n_seqs; ++i) {
        BlockPrefillSeq& e = p.seqs[i];
        finished[i] = (uint8_t)e.pairs;
        x.pre[i] = e.seg_begin;
        x.pre_n[i] = e.step_begin;
        const int32_t before = (e.step_begin + 127) / 128;
        e.pairs = (int32_t)head_pairs(c, e.q_len);
        e.seg_begin = (int32_t)segs;
        e.step_begin = (int32_t)steps;
        e.head_steps = flat ? e.pairs * ((e.n - 1) / 128 + 1) : (int32_t)head_steps(c, e.n, e.q_len) + e.pairs * before;
        longest = std::max<int64_t>(longest, before + (e.n - 1) / 128 + 1);
        segs += (int64_t)e.pairs * hkv;
        steps += (int64_t)e.head_steps * hkv;
        if (2 * (e.head_steps / e.pairs) > longest) n_long += (int64_t)e.pairs * hkv;  // (the longest come first)
    }
    x.flat = flat;
    x.pre_o = beside.pre_o;
    x.pre_lse = beside.pre_lse;
    x.totals = flat ? beside.totals : nullptr;
    mark(x.merged, finished, p.n_seqs);
    // Whole segments, the longest first, end when the longest does or the SMs have shared out all;
    // the line of all steps cut evenly ends a share of the steps later, and then costs about four more
    // for the partial results and the kernel that adds them (6 us where a step takes 1.5); eight with prefixes, whose
    // rows are fp32 or are joined (15 to 20 us where it takes 1.9).
    const int64_t sms = std::min(c->sms, kBlockPrefillGrid);
    const int64_t share = (steps + sms - 1) / sms;
    if (more) {
        // Segments can be of very different length here, where some sequences have a prefix in front: changes of segment count as well,
        // as many as the line's last CTA has, whose are the shortest, and of whole ones only those that cannot share an SM count as the longest.
        // (16 sequences, half of them behind a prefix of 8k: 493 us by the rule below.)
        int64_t left = share, last = 0;
        for (int i = p.n_seqs - 1; i >= 0 && left > 0; left -= (int64_t)p.seqs[i--].head_steps * hkv) {
            const BlockPrefillSeq& e = p.seqs[i];
            last += std::min<int64_t>((int64_t)e.pairs * hkv, left / std::max(1, e.head_steps / e.pairs) + 1);
        }
        const int64_t whole = std::max(share, longest * ((n_long + sms - 1) / sms)) + kChangeSteps * (segs / sms);
        p.line = whole > share + 8 + kChangeSteps * last;
    } else {
        const int64_t whole = segs >= 2 * sms ? share : std::max(share, longest * ((segs + sms - 1) / sms));
        p.line = whole > share + 4;
    }
    p.steps = (int32_t)steps;
    p.segs = (int32_t)segs;
    p.grid = (int32_t)std::min<int64_t>(sms, p.line ? steps : segs);
    if (c->host_only) return KVARN_OK;
    const kvarn_status st = ensure_init(c, stream);
    if (st) return st;
    const int rc = more ? launch_block_prefill(p, x, stream) : launch_block_prefill(p, stream);
    return rc ? cuda_fail(rc, "prefill launch") : KVARN_OK;
}

// ---- prefixes and weights ----

// The prefix of each sequence (-1 for none) and that none of them is a sequence of the call.
kvarn_status check_prefix_ids(kvarn_block_cache* c, int32_t n_seqs, const int32_t* ids, const int32_t* prefix_ids) {
    if (!prefix_ids) return KVARN_OK;
    kvarn_status st = KVARN_OK;
    for (int i = 0; i < n_seqs; ++i) c->seen[ids[i]] = 1;
    for (int i = 0; i < n_seqs && !st; ++i) {
        const int32_t pre = prefix_ids[i];
        if (pre < -1 || pre >= c->cfg.max_seqs) st = fail(KVARN_EINVAL, "no such prefix");
        else if (pre >= 0 && c->seen[pre]) st = fail(KVARN_EINVAL, "a prefix is a sequence of the call");
    }
    for (int i = 0; i < n_seqs; ++i) c->seen[ids[i]] = 0;
    return st;
}

// The prefixes of an attention call, and that its work with them can be counted.
kvarn_status check_prefixes(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* prefix_ids,
                            const int32_t* q_lens, const int32_t* added) {
    if (!prefix_ids) return KVARN_OK;
    kvarn_status st = check_prefix_ids(c, n_seqs, ids, prefix_ids);
    if (st) return st;
    int64_t tiles = 0, steps = 0;
    for (int i = 0; i < n_seqs; ++i) {
        const int32_t pre = prefix_ids[i];
        const int64_t own = c->L(ids[i], layer) + (added ? (int64_t)added[i] : 0), most_pairs = head_pairs(c, q_lens ? q_lens[i] : 1);
        tiles += head_tiles(own);
        steps += most_pairs * ((own + 127) / 128);
        if (pre < 0) continue;
        const int64_t n = c->L(pre, layer);
        tiles += tiles_of(n);
        steps += most_pairs * ((n + 127) / 128);
    }
    if ((tiles + n_seqs * (1 + kPairCost)) * c->cfg.num_kv_heads >= 1ll << 31) return fail(KVARN_ECAPACITY, "2^31 tiles of 32 tokens or more in a call");
    if (steps * c->cfg.num_kv_heads >= 1ll << 31) {  // every pair counted as long as the last: now exactly
        steps = 0;
        for (int i = 0; i < n_seqs; ++i) {
            const int64_t own = c->L(ids[i], layer) + (added ? (int64_t)added[i] : 0), m = q_lens ? q_lens[i] : 1;
            steps += head_steps(c, own, m) + head_pairs(c, m) * (prefix_ids[i] >= 0 ? key_steps(c->L(prefix_ids[i], layer)) : 0);
        }
    }
    if (steps * c->cfg.num_kv_heads >= 1ll << 31) return fail(KVARN_ECAPACITY, "2^31 steps of 128 keys or more in a call");
    return KVARN_OK;
}

// Is a prefix of a group of single queries better walked once, as tiles of 128 rows (two more launches), than by each
// sequence? (Measured, 32 / 8 heads of 128, us once and each: 4 sequences behind 32k 42 and 45; 8 behind 8k 30 and 28, behind
// 32k 42 and 79; 16 behind 2k 24 and 20, behind 8k 31 and 45; 64 behind 512 41 and 28, behind 2k 47 and 52, behind 32k 83 and 543. With
// 16 / 2 heads: 32 behind 8k 35 and 32, 64 behind 8k 34 and 49.) Each group is judged by itself, as if it paid for the two launches
// alone, and all measurements are of one group or two: many groups in a call, each under the limit, are walked by every
// sequence although one pass would do for all. Nor does the limit know head_dim (half the bytes at 64).
bool walked_once(const kvarn_block_cache* c, const Entry& g) {
    const int64_t each = (int64_t)g.q_len * g.n, once = head_pairs(c, g.q_len) * (int64_t)g.n;
    return each >= 4 * once && each * c->cfg.num_kv_heads > 600000;
}

// The same for more queries, whose row tiles are filled by each sequence's own: `extra` steps of all KV heads are what the prefixes
// take more that way. Walked once they take a launch of their own and fp32 rows that are joined. (Measured, 32 / 8 heads of 128, us once
// and each: 8 sequences of 17 to 200 queries behind 2k, 2.5 extra steps a SM, 57 and 42; 4 of 400 to 700 behind 16k, 6.7, 421 and
// 398; 32 of 2 to 16 behind 1k, 11.4, 60 and 43; 8 of 30 to 100 behind 8k, 16.8, 123 and 114; 8 of 2 to 16 behind 8k, 20.2, 54 and 63;
// 16 of 40 to 64 behind 16k, 20.2, 197 and 225; 64 behind four of 2k, 22.7, 137 and 154.) One answer for all prefixes of a call, also
// where one has many short questions and another a long prompt.
bool stacked(const kvarn_block_cache* c, int64_t extra) { return extra > (int64_t)kOwnSteps * c->sms; }

// How an attention call with prefixes goes: its sequences with queries, and the runs of them whose prefix is walked once. (Depends
// on query counts and the prefixes' lengths alone.)
struct AttendPlan {
    int32_t ids[kBlockMaxSeqs], lens[kBlockMaxSeqs], before[kBlockMaxSeqs];  // before: a prefix that the sequence walks itself, -1 for none
    uint8_t finished[kBlockMaxSeqs];  // 1: its prefix is walked once
    Entry once[kBlockMaxSeqs];        // rows behind such a prefix
    int32_t n, n_once;
    bool single;
};
void plan_attend(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* prefix_ids,
                 const int32_t* q_lens, AttendPlan& a) {
    Entry groups[kBlockMaxSeqs];
    int64_t extra = 0, row = 0;
    int32_t n_groups = 0;
    a.single = !q_lens || single_queries(n_seqs, q_lens);
    a.n = a.n_once = 0;
    // Sequences without queries leave; runs of one prefix become groups of rows.
    for (int i = 0; i < n_seqs; ++i) {
        const int32_t m = q_lens ? q_lens[i] : 1;
        if (m == 0) continue;
        const int32_t pre = prefix_ids && prefix_ids[i] >= 0 && c->L(prefix_ids[i], layer) > 0 ? prefix_ids[i] : -1;
        a.ids[a.n] = ids[i];
        a.before[a.n] = pre;
        a.lens[a.n] = m;
        if (pre >= 0) {
            if (a.n == 0 || a.before[a.n - 1] != pre) groups[n_groups++] = Entry{pre, c->L(pre, layer), 0, (int32_t)row, -1, 0};
            groups[n_groups - 1].q_len += m;
            extra += head_pairs(c, m) * key_steps(c->L(pre, layer));
        }
        ++a.n;
        row += m;
    }
    // Sequences can also walk a prefix each by itself, in the one launch that takes their own tokens. The groups whose
    // prefix is better walked once are those where that takes longer than the tiles' steps.
    for (int g = 0; g < n_groups; ++g) extra -= head_pairs(c, groups[g].q_len) * key_steps(groups[g].n);
    const bool together = stacked(c, extra * c->cfg.num_kv_heads);
    auto walked = [&](int g) { return a.single ? walked_once(c, groups[g]) : together; };
    for (int i = 0, g = -1, last = -1; i < a.n; ++i) {
        const int32_t pre = a.before[i];
        if (pre >= 0 && pre != last) ++g;
        last = pre;
        a.finished[i] = pre >= 0 && walked(g);
        if (a.finished[i]) a.before[i] = -1;
    }
    for (int g = 0; g < n_groups; ++g)
        if (walked(g)) a.once[a.n_once++] = groups[g];
}

// The parts of an attention call's workspace.
struct Workspace {
    size_t pre_o = 0, pre_lse = 0, sums = 0, totals = 0, total = 0;
};
bool make_workspace(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* prefix_ids,
                    const int32_t* q_lens, const int32_t* added, bool weights, Workspace* w) {
    unsigned __int128 rows = 0, tiles = 0, off = 0;
    bool any = false;
    for (int i = 0; i < n_seqs; ++i) {
        const bool pre = prefix_ids && prefix_ids[i] >= 0;
        any = any || pre;
        rows += q_lens ? q_lens[i] : 1;
        tiles += head_tiles(c->L(ids[i], layer) + (added ? added[i] : 0)) + (pre ? tiles_of(c->L(prefix_ids[i], layer)) : 0) + kPairCost;
    }
    auto take = [&](unsigned __int128 n) {
        const unsigned __int128 o = off;
        off = (off + n + 255) / 256 * 256;
        return (size_t)o;
    };
    // Rows over prefixes: where one is walked once; small ones in any case, so that the workspace of a batch's steps goes by its
    // counts alone.
    const unsigned __int128 rows_o = rows * c->cfg.num_q_heads * c->cfg.head_dim * 4;
    if (any && rows_o > kSmallRows && rows < 1ll << 31) {
        AttendPlan a;
        plan_attend(c, layer, n_seqs, ids, prefix_ids, q_lens, a);
        any = a.n_once > 0;
    }
    w->pre_o = take(any ? rows_o : 0);
    w->pre_lse = take(any ? rows * c->cfg.num_q_heads * 4 : 0);
    w->sums = take(weights ? tiles * c->cfg.num_q_heads * 8 : 0);
    w->totals = take(weights ? rows * c->cfg.num_q_heads * 8 : 0);
    w->total = (size_t)off;
    return off < (unsigned __int128)1 << 46;
}

// Two ranges of memory that meet.
bool meet(const void* a, size_t na, const void* b, size_t nb) {
    return na && nb && (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

// Arguments that attend, append_attend and window_weights share, once the sequences are known to be good.
kvarn_status check_beside(kvarn_block_cache* c, int64_t rows, const void* q, const void* out, const float* weights,
                          const void* workspace, size_t bytes, const Workspace& w) {
    if (w.total > bytes || (w.total && !workspace)) return fail(KVARN_EINVAL, "the workspace is too small");
    if (!aligned16(workspace)) return fail(KVARN_EINVAL, "the workspace must be 16-byte aligned");
    const size_t io = (size_t)rows * c->cfg.num_q_heads * c->cfg.head_dim * 2;
    const size_t held = weights ? (size_t)c->cfg.max_seqs * c->cfg.num_kv_heads * columns(c) * 4 : 0;
    if (weights && ((uintptr_t)weights & 3)) return fail(KVARN_EINVAL, "weights must be 4-byte aligned");
    if (weights && c->cfg.num_kv_heads > 65535) return fail(KVARN_ECAPACITY, "weights of more than 65,535 KV heads");
    if (meet(weights, held, q, io) || meet(weights, held, out, out ? io : 0) || meet(workspace, w.total, q, io) ||
        meet(workspace, w.total, out, out ? io : 0) || meet(workspace, w.total, weights, held))
        return fail(KVARN_EINVAL, "weights or workspace overlap another argument");
    return KVARN_OK;
}

// All arguments of an attention call beyond check_call's, check_append's and check_attention's.
kvarn_status check_attend(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* prefix_ids,
                          const int32_t* q_lens, const int32_t* added, const void* q, const void* out, const float* weights,
                          const void* workspace, size_t bytes, Workspace* w) {
    if (weights && q_lens && !single_queries(n_seqs, q_lens))
        return fail(KVARN_EINVAL, "weights are noted for single queries (window_weights takes more)");
    kvarn_status st = check_prefixes(c, layer, n_seqs, ids, prefix_ids, q_lens, added);
    if (st) return st;
    if (!make_workspace(c, layer, n_seqs, ids, prefix_ids, q_lens, added, weights != nullptr, w))
        return fail(KVARN_ECAPACITY, "the workspace is too large");
    int64_t rows = 0;
    for (int i = 0; i < n_seqs; ++i) rows += q_lens ? q_lens[i] : 1;
    return check_beside(c, rows, q, out, weights, workspace, bytes, *w);
}

// The line of a window_weights call and its workspace. (Prefixes are known to be sequences of the cache.)
kvarn_status plan_window(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* prefix_ids,
                         const int32_t* q_lens, BlockWindowParams& p, Workspace* w) {
    const int hkv = c->cfg.num_kv_heads;
    int64_t rows = 0, units = 0, pairs = 0, sums = 0;
    p.n_seqs = 0;
    for (int i = 0; i < n_seqs; ++i) {
        const int64_t n = c->L(ids[i], layer), m = q_lens[i];
        if (m < 0 || m > n) return fail(KVARN_EINVAL, "a query count is negative or above the sequence's length");
        if (m > kWindowTokens) return fail(KVARN_EINVAL, "more than 128 queries of a sequence");
        if (m > 0) {
            BlockRowsSeq& e = p.seqs[p.n_seqs++];
            e.seq = ids[i];
            e.n = (int32_t)n;
            e.q_len = (int32_t)m;
            e.q_row = (int32_t)rows;
            e.rows = (int32_t)m * c->r;
            e.pad = (e.rows + 7) / 8 * 8;
            e.row_tiles = (e.rows + 127) / 128;
            e.pre = prefix_ids ? prefix_ids[i] : -1;
            e.pre_n = e.pre >= 0 ? c->L(e.pre, layer) : 0;
            e.steps = (int32_t)(key_steps(e.pre_n) + key_steps(n));
            e.unit_begin = (int32_t)units;
            e.pair_begin = (int32_t)pairs;
            e.sum_begin = sums;
            units += (int64_t)hkv * e.row_tiles * e.steps;
            pairs += (int64_t)hkv * e.row_tiles;
            sums += (int64_t)hkv * tiles_of(n) * e.pad;
        }
        rows += m;
        if (units >= 1ll << 31) return fail(KVARN_ECAPACITY, "2^31 steps of 128 keys or more in a call");
    }
    p.units = units;
    p.grid = (int32_t)std::min<int64_t>(c->sms, units);
    w->totals = (size_t)(sums * 8 + 255) / 256 * 256;
    w->total = p.n_seqs ? w->totals + (size_t)(pairs + p.grid) * kWindowParts * 128 * 8 : 0;
    return KVARN_OK;
}

kvarn_status run_attend(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* prefix_ids,
                        const int32_t* q_lens, const void* q, void* out, float scale, float* weights, void* workspace,
                        const Workspace& w, void* stream) {
    AttendPlan a;
    plan_attend(c, layer, n_seqs, ids, prefix_ids, q_lens, a);
    if (a.n == 0) return KVARN_OK;
    Beside b;
    if (weights) {
        b.weights = weights;
        b.sums = (float2*)((uint8_t*)workspace + w.sums);
        b.totals = (float2*)((uint8_t*)workspace + w.totals);
    }
    if (a.n_once > 0) {
        b.pre_o = (float*)((uint8_t*)workspace + w.pre_o);
        b.pre_lse = (float*)((uint8_t*)workspace + w.pre_lse);
        const kvarn_status st = run_tiles(c, layer, a.n_once, a.once, true, q, nullptr, scale, stream, b);
        if (st) return st;
    }
    b.finished = a.finished;
    if (a.single || std::any_of(a.before, a.before + a.n, [](int32_t pre) { return pre >= 0; })) b.before = a.before;
    if (!a.single) return run_prefill(c, layer, a.n, a.ids, a.lens, q, out, scale, stream, b);
    return run_decode(c, layer, a.n, a.ids, q, out, scale, stream, b);
}

// Do any of the n rows of `len` values at a, `stride` apart, touch one of b's? (Values of 16 bits.)
struct Rows {
    const void* at;
    int64_t len, stride;
};
bool rows_meet(const Rows& a, const Rows& b, int64_t n) {
    typedef __int128 I;
    const I d = (I)(uintptr_t)b.at - (I)(uintptr_t)a.at;
    const I sa = (I)a.stride * 2, sb = (I)b.stride * 2, la = a.len * 2, lb = b.len * 2;
    if (d >= (n - 1) * sa + la || -d >= (n - 1) * sb + lb) return false;  // apart as a whole
    if (n == 1) return true;
    if (sa == sb) {  // where b's rows lie between two of a's
        const I in = (d % sa + sa) % sa;
        return in < la || in + lb > sa;
    }
    for (int64_t t = 0; t < n; ++t) {  // row t of a, and the rows of b that start before its end, the last one or two
        const I from = t * sa - d, end = from + la;
        if (end <= 0) continue;
        const I u = (end - 1) / sb;
        if (u < n ? u * sb + lb > from : (n - 1) * sb + lb > from) return true;
    }
    return false;
}

}  // namespace

// Host allocations are made by kvarn_block_create alone; every other entry works in memory
// that it reserved, so that no C++ exception can reach a C caller.
extern "C" {

kvarn_status kvarn_block_required_bytes(const kvarn_block_config* cfg, size_t* bytes) {
    kvarn_status st = check_config(cfg);
    if (st) return st;
    if (!bytes) return fail(KVARN_EINVAL, "no place for the size");
    BlockView v;
    if (!make_view(*cfg, &v)) return fail(KVARN_EINVAL, "the cache is too large");
    *bytes = v.lay.total;
    return KVARN_OK;
}

kvarn_status kvarn_block_create(const kvarn_block_config* cfg, void* dev_mem, size_t bytes, kvarn_block_cache** out) {
    kvarn_status st = check_config(cfg);
    if (st) return st;
    if (!out || !dev_mem || ((uintptr_t)dev_mem & 255)) return fail(KVARN_EINVAL, "dev_mem must be 256-byte aligned");
    std::unique_ptr<kvarn_block_cache> c(new (std::nothrow) kvarn_block_cache());
    if (!c) return fail(KVARN_ENOMEM, "out of host memory");
    c->cfg = *cfg;
    if (!make_view(*cfg, &c->view)) return fail(KVARN_EINVAL, "the cache is too large");
    if (bytes < c->view.lay.total) return fail(KVARN_ENOMEM, "the device block is too small");
    c->view.base = (uint8_t*)dev_mem;
    c->r = cfg->num_q_heads / cfg->num_kv_heads;
    c->host_only = (cfg->flags & KVARN_FLAG_HOST_ONLY) != 0;
    try {
        c->len.assign((size_t)cfg->max_seqs * cfg->num_layers, 0);
        c->table.assign((size_t)cfg->max_seqs * cfg->num_layers * c->view.max_blocks, -1);
        c->free_slots.resize(cfg->pool_blocks);
        c->seen.assign(cfg->max_seqs, 0);
    } catch (...) {
        return fail(KVARN_ENOMEM, "out of host memory");
    }
    for (int i = 0; i < cfg->pool_blocks; ++i) c->free_slots[i] = cfg->pool_blocks - 1 - i;  // pop gives 0, 1, 2 ..
    if (!c->host_only) {
        c->sms = sm_count();
        if (c->sms <= 0 || pointer_device(dev_mem, &c->device)) return fail(KVARN_ECUDA, "no CUDA device");
    }
    *out = c.release();
    return KVARN_OK;
}

void kvarn_block_destroy(kvarn_block_cache* cache) { delete cache; }

kvarn_status kvarn_block_append(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                const int32_t* n_tokens, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, true);
    if (st) return st;
    st = check_append(c, layer, n_seqs, seq_ids, n_tokens, k, v, k_stride, v_stride);
    if (st) return st;
    return append(c, layer, n_seqs, seq_ids, n_tokens, k, v, k_stride, v_stride, stream);
}

kvarn_status kvarn_block_read(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                              const int32_t* starts, const int32_t* counts, void* k, void* v, int32_t out_fp32,
                              void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, false);
    if (st) return st;
    if (n_seqs > 0 && !counts) return fail(KVARN_EINVAL, "no token counts");
    static thread_local BlockReadParams p;
    p.c = c->view;
    p.c.layer = layer;
    p.k = k;
    p.v = v;
    p.f32 = out_fp32 != 0;
    p.n_seqs = 0;
    int64_t row = 0, items = 0;
    for (int i = 0; i < n_seqs; ++i) {
        const int64_t n = c->L(seq_ids[i], layer), s = starts ? starts[i] : 0, m = counts[i];
        if (s < 0 || m < 0 || s + m > n) return fail(KVARN_EINVAL, "a range is outside its sequence");
        if (m > 0) {
            BlockReadSeq& e = p.seqs[p.n_seqs++];
            e.seq = seq_ids[i];
            e.n = (int32_t)n;
            e.start = (int32_t)s;
            e.count = (int32_t)m;
            e.out_row = (int32_t)row;
            e.item_begin = (int32_t)items;
            items += ((s + m - 1) / kTileTokens - s / kTileTokens + 1) * c->cfg.num_kv_heads * 2;
        }
        row += m;
        if (row >= 1ll << 31 || items >= 1ll << 31) return fail(KVARN_ECAPACITY, "too many tokens in a call");
    }
    if (p.n_seqs == 0) return KVARN_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v)) return fail(KVARN_EINVAL, "k and v must be 16-byte aligned");
    p.items = (int32_t)items;
    if (c->host_only) return KVARN_OK;
    const int rc = launch_block_read(p, stream);
    return rc ? cuda_fail(rc, "read launch") : KVARN_OK;
}

kvarn_status kvarn_block_decode_attention(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                          const void* q, void* out, float softmax_scale, void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, false);
    if (st) return st;
    st = check_attention(c, layer, n_seqs, seq_ids, nullptr, nullptr, q, out, softmax_scale);
    if (st || n_seqs == 0) return st;
    return run_decode(c, layer, n_seqs, seq_ids, q, out, softmax_scale, stream);
}

kvarn_status kvarn_block_decode_step(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                     const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                                     void* out, float softmax_scale, void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, true);
    if (st) return st;
    int32_t ones[kBlockMaxSeqs];
    for (int i = 0; i < n_seqs; ++i) ones[i] = 1;
    st = check_append(c, layer, n_seqs, seq_ids, ones, k, v, k_stride, v_stride);
    if (st) return st;
    st = check_attention(c, layer, n_seqs, seq_ids, nullptr, ones, q, out, softmax_scale);
    if (st || n_seqs == 0) return st;
    st = append(c, layer, n_seqs, seq_ids, ones, k, v, k_stride, v_stride, stream);
    if (st) return st;
    return run_decode(c, layer, n_seqs, seq_ids, q, out, softmax_scale, stream);
}

kvarn_status kvarn_block_prefill_attention(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                           const int32_t* q_lens, const void* q, void* out, float softmax_scale,
                                           void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, false);
    if (st) return st;
    if (n_seqs > 0 && !q_lens) return fail(KVARN_EINVAL, "no query counts");
    st = check_attention(c, layer, n_seqs, seq_ids, q_lens, nullptr, q, out, softmax_scale);
    if (st || n_seqs == 0) return st;
    return run_prefill(c, layer, n_seqs, seq_ids, q_lens, q, out, softmax_scale, stream);
}

kvarn_status kvarn_block_prefill(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                 const int32_t* n_tokens, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, const void* q, void* out, float softmax_scale, void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, true);
    if (st) return st;
    st = check_append(c, layer, n_seqs, seq_ids, n_tokens, k, v, k_stride, v_stride);
    if (st) return st;
    st = check_attention(c, layer, n_seqs, seq_ids, n_tokens, n_tokens, q, out, softmax_scale);
    if (st || n_seqs == 0) return st;
    st = append(c, layer, n_seqs, seq_ids, n_tokens, k, v, k_stride, v_stride, stream);
    if (st) return st;
    return run_prefill(c, layer, n_seqs, seq_ids, n_tokens, q, out, softmax_scale, stream);
}

kvarn_status kvarn_block_attend_workspace(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                          const int32_t* prefix_ids, const int32_t* counts, int32_t appended, int32_t weights,
                                          size_t* bytes) {
    if (!c || !bytes) return fail(KVARN_EINVAL, "no cache, or no place for the size");
    if (layer < 0 || layer >= c->cfg.num_layers) return fail(KVARN_EINVAL, "no such layer");
    if (n_seqs < 0 || (n_seqs > 0 && !seq_ids)) return fail(KVARN_EINVAL, "bad sequence list");
    if (n_seqs > kBlockMaxSeqs) return fail(KVARN_ECAPACITY, "more than 256 sequences in a call");
    if (appended && n_seqs > 0 && !counts) return fail(KVARN_EINVAL, "no token counts");
    for (int i = 0; i < n_seqs; ++i) {
        if (seq_ids[i] < 0 || seq_ids[i] >= c->cfg.max_seqs || (prefix_ids && (prefix_ids[i] < -1 || prefix_ids[i] >= c->cfg.max_seqs)))
            return fail(KVARN_EINVAL, "a sequence id is out of range");
        if (counts && counts[i] < 0) return fail(KVARN_EINVAL, "a count is negative");
    }
    Workspace w;
    if (!make_workspace(c, layer, n_seqs, seq_ids, prefix_ids, counts, appended ? counts : nullptr, weights != 0, &w))
        return fail(KVARN_ECAPACITY, "the workspace is too large");
    *bytes = w.total;
    return KVARN_OK;
}

kvarn_status kvarn_block_attend(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                const int32_t* prefix_ids, const int32_t* q_lens, const void* q, void* out,
                                float softmax_scale, float* weights, void* workspace, size_t workspace_bytes, void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, false);
    if (st) return st;
    st = check_attention(c, layer, n_seqs, seq_ids, q_lens, nullptr, q, out, softmax_scale);
    if (st) return st;
    Workspace w;
    st = check_attend(c, layer, n_seqs, seq_ids, prefix_ids, q_lens, nullptr, q, out, weights, workspace, workspace_bytes, &w);
    if (st || n_seqs == 0) return st;
    return run_attend(c, layer, n_seqs, seq_ids, prefix_ids, q_lens, q, out, softmax_scale, weights, workspace, w, stream);
}

kvarn_status kvarn_block_append_attend(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                       const int32_t* prefix_ids, const int32_t* n_tokens, const void* k, int64_t k_stride,
                                       const void* v, int64_t v_stride, const void* q, void* out, float softmax_scale,
                                       float* weights, void* workspace, size_t workspace_bytes, void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, true);
    if (st) return st;
    st = check_append(c, layer, n_seqs, seq_ids, n_tokens, k, v, k_stride, v_stride);
    if (st) return st;
    st = check_attention(c, layer, n_seqs, seq_ids, n_tokens, n_tokens, q, out, softmax_scale);
    if (st) return st;
    Workspace w;
    st = check_attend(c, layer, n_seqs, seq_ids, prefix_ids, n_tokens, n_tokens, q, out, weights, workspace, workspace_bytes, &w);
    if (st || n_seqs == 0) return st;
    st = append(c, layer, n_seqs, seq_ids, n_tokens, k, v, k_stride, v_stride, stream);
    if (st) return st;
    return run_attend(c, layer, n_seqs, seq_ids, prefix_ids, n_tokens, q, out, softmax_scale, weights, workspace, w, stream);
}

kvarn_status kvarn_block_window_workspace(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                          const int32_t* q_lens, size_t* bytes) {
    return kvarn_block_window_workspace_prefixes(c, layer, n_seqs, seq_ids, nullptr, q_lens, bytes);
}

kvarn_status kvarn_block_window_workspace_prefixes(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                                   const int32_t* prefix_ids, const int32_t* q_lens, size_t* bytes) {
    if (!c || !bytes) return fail(KVARN_EINVAL, "no cache, or no place for the size");
    if (layer < 0 || layer >= c->cfg.num_layers) return fail(KVARN_EINVAL, "no such layer");
    if (n_seqs < 0 || (n_seqs > 0 && (!seq_ids || !q_lens))) return fail(KVARN_EINVAL, "bad sequence list");
    if (n_seqs > kBlockMaxSeqs) return fail(KVARN_ECAPACITY, "more than 256 sequences in a call");
    for (int i = 0; i < n_seqs; ++i)
        if (seq_ids[i] < 0 || seq_ids[i] >= c->cfg.max_seqs || (prefix_ids && (prefix_ids[i] < -1 || prefix_ids[i] >= c->cfg.max_seqs)))
            return fail(KVARN_EINVAL, "a sequence id is out of range");
    static thread_local BlockWindowParams p;
    Workspace w;
    const kvarn_status st = plan_window(c, layer, n_seqs, seq_ids, prefix_ids, q_lens, p, &w);
    if (st == KVARN_OK) *bytes = w.total;
    return st;
}

kvarn_status kvarn_block_window_weights(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                        const int32_t* q_lens, const void* q, float softmax_scale, float* weights,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    return kvarn_block_window_weights_prefixes(c, layer, n_seqs, seq_ids, nullptr, q_lens, q, softmax_scale, weights, workspace,
                                               workspace_bytes, stream);
}

kvarn_status kvarn_block_window_weights_prefixes(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids,
                                                 const int32_t* prefix_ids, const int32_t* q_lens, const void* q,
                                                 float softmax_scale, float* weights, void* workspace, size_t workspace_bytes,
                                                 void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, false);
    if (st) return st;
    if (!std::isfinite(softmax_scale * kLog2e)) return fail(KVARN_EINVAL, "softmax_scale must be finite, below 2^127");
    if (n_seqs > 0 && !q_lens) return fail(KVARN_EINVAL, "no query counts");
    static thread_local BlockWindowParams p;
    static thread_local BlockWeighParams wp;
    Workspace w;
    st = check_prefix_ids(c, n_seqs, seq_ids, prefix_ids);
    if (st) return st;
    st = plan_window(c, layer, n_seqs, seq_ids, prefix_ids, q_lens, p, &w);
    if (st || p.n_seqs == 0) return st;
    if (!q || !aligned16(q)) return fail(KVARN_EINVAL, "q must be 16-byte aligned");
    if (!weights) return fail(KVARN_EINVAL, "no weights");
    const BlockRowsSeq& end = p.seqs[p.n_seqs - 1];
    st = check_beside(c, (int64_t)end.q_row + end.q_len, q, nullptr, weights, workspace, workspace_bytes, w);
    if (st || c->host_only) return st;
    p.c = c->view;
    p.c.layer = layer;
    p.q = (const uint16_t*)q;
    p.sums = (float2*)((uint8_t*)workspace + w.sums);
    p.totals = (float2*)((uint8_t*)workspace + w.totals);
    p.hq = c->cfg.num_q_heads;
    p.r = c->r;
    p.scale_log2 = softmax_scale * kLog2e;
    const int rc = launch_block_window(p, stream);
    if (rc) return cuda_fail(rc, "window launch");
    wp.sums = p.sums;
    wp.totals = p.totals;
    wp.weights = weights;
    wp.units = p.units;
    wp.grid = p.grid;
    wp.n_seqs = p.n_seqs;
    for (int i = 0; i < p.n_seqs; ++i) {
        const BlockRowsSeq& e = p.seqs[i];
        wp.seqs[i] = BlockWeighSeq{e.seq, e.rows, e.pad, 0, tiles_of(e.n), tiles_of(e.n), 0, e.unit_begin, e.pair_begin, e.steps, e.sum_begin};
    }
    return run_weigh(c, wp, stream);
}

kvarn_status kvarn_block_evict(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* seq_ids, int32_t keep,
                               int32_t first, int32_t last, float* weights, int32_t* kept, void* stream) {
    kvarn_status st = check_call(c, layer, n_seqs, seq_ids, stream, true);
    if (st) return st;
    if (first < 0 || last < 0 || keep < 0 || (int64_t)first + last > keep)
        return fail(KVARN_EINVAL, "keep must be at least first + last, none of them negative");
    if (n_seqs == 0) return KVARN_OK;
    if (!weights || ((uintptr_t)weights & 3) || (keep > 0 && (!kept || ((uintptr_t)kept & 3))))
        return fail(KVARN_EINVAL, "weights and kept must be 4-byte aligned");
    if (meet(weights, (size_t)c->cfg.max_seqs * c->cfg.num_kv_heads * columns(c) * 4, kept,
             (size_t)n_seqs * c->cfg.num_kv_heads * keep * 4))
        return fail(KVARN_EINVAL, "weights and kept overlap");
    static thread_local BlockEvictParams p;
    const int bt = c->cfg.block_tokens;
    p.n_seqs = 0;
    for (int cut = 1; cut >= 0; --cut)  // those to cut come first
        for (int i = 0, n = cut ? 0 : p.n_seqs; i < n_seqs; ++i) {
            const int32_t full = c->L(seq_ids[i], layer) / bt;
            if ((full > keep) != (cut == 1)) continue;
            p.seqs[n++] = BlockEvictSeq{seq_ids[i], full, i};
            if (cut) p.n_seqs = n;
        }
    p.n_all = n_seqs;
    st = ensure_init(c, stream);
    if (st) return st;
    if (!c->host_only) {
        p.c = c->view;
        p.c.layer = layer;
        p.weights = weights;
        p.kept = kept;
        p.keep = keep;
        p.first = first;
        p.last = last;
        p.cols = (int32_t)columns(c);
        const int rc = launch_block_evict(p, stream);
        if (rc) return cuda_fail(rc, "evict launch");
    }
    for (int i = 0; i < p.n_seqs; ++i) {
        int32_t* t = c->T(p.seqs[i].seq, layer);
        for (int b = p.seqs[i].full - 1; b >= keep; --b) {
            c->free_slots.push_back(t[b]);
            t[b] = -1;
        }
        c->L(p.seqs[i].seq, layer) -= (p.seqs[i].full - keep) * bt;
    }
    return KVARN_OK;
}

kvarn_status kvarn_block_release(kvarn_block_cache* c, int32_t n_seqs, const int32_t* seq_ids) {
    if (!c || n_seqs < 0 || (n_seqs > 0 && !seq_ids)) return fail(KVARN_EINVAL, "bad sequence list");
    for (int i = 0; i < n_seqs; ++i)
        if (seq_ids[i] < 0 || seq_ids[i] >= c->cfg.max_seqs) return fail(KVARN_EINVAL, "no such sequence");
    for (int i = 0; i < n_seqs; ++i)
        for (int l = c->cfg.num_layers - 1; l >= 0; --l) {
            int32_t* t = c->T(seq_ids[i], l);
            // free_slots never holds more than pool_blocks entries: it was sized to that once
            for (int b = c->L(seq_ids[i], l) / c->cfg.block_tokens - 1; b >= 0; --b) {
                c->free_slots.push_back(t[b]);
                t[b] = -1;
            }
            c->L(seq_ids[i], l) = 0;
        }
    return KVARN_OK;
}

kvarn_status kvarn_block_length(const kvarn_block_cache* c, int32_t layer, int32_t seq_id, int64_t* len) {
    if (!c || !len || layer < 0 || layer >= c->cfg.num_layers || seq_id < 0 || seq_id >= c->cfg.max_seqs)
        return fail(KVARN_EINVAL, "no such layer or sequence");
    *len = c->len[(size_t)seq_id * c->cfg.num_layers + layer];
    return KVARN_OK;
}

kvarn_status kvarn_block_check_device_error(kvarn_block_cache* c, void* stream) {
    if (!c) return fail(KVARN_EINVAL, "no cache");
    if (c->host_only || !c->initialized) return KVARN_OK;
    int32_t err[4] = {0, 0, 0, 0};
    int rc = memcpy_d2h_sync(err, c->view.base + c->view.lay.err, sizeof(err), stream);
    if (rc) return cuda_fail(rc, "error word read");
    if (err[0] == 0) return KVARN_OK;
    // (not by a copy from here: that may read this frame after the return) and the counters, which a
    // launch in which a wait gave up may have left standing
    rc = launch_block_clear_errors(c->view, stream);
    if (rc) return cuda_fail(rc, "error word clear");
    return err[0] & kErrTimeout ? KVARN_ETIMEOUT : KVARN_ESTATE;
}

kvarn_status kvarn_qk_norm_rope(const kvarn_qk_config* cfg, int64_t n_tokens, const void* q, int64_t q_stride, const void* k,
                                int64_t k_stride, const float* q_weight, const float* k_weight, const int32_t* positions,
                                const double* freqs, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                void* stream) {
    return kvarn_qk_norm_rope_axes(cfg, n_tokens, q, q_stride, k, k_stride, q_weight, k_weight, positions, 0, 1, nullptr,
                                   freqs, q_out, q_out_stride, k_out, k_out_stride, stream);
}

kvarn_status kvarn_qk_norm_rope_axes(const kvarn_qk_config* cfg, int64_t n_tokens, const void* q, int64_t q_stride,
                                     const void* k, int64_t k_stride, const float* q_weight, const float* k_weight,
                                     const int32_t* positions, int64_t axis_stride, int32_t n_axes, const uint8_t* axes,
                                     const double* freqs, void* q_out, int64_t q_out_stride, void* k_out,
                                     int64_t k_out_stride, void* stream) {
    if (!cfg) return fail(KVARN_EINVAL, "no configuration");
    const int64_t hq = cfg->num_q_heads, hk = cfg->num_kv_heads, d = cfg->head_dim;
    if (hq < 0 || hk < 0 || hq + hk < 1 || hq + hk > (1 << 16)) return fail(KVARN_EINVAL, "bad head counts");
    if (d < 8 || d > 256 || d % 8) return fail(KVARN_EINVAL, "head_dim must be a multiple of 8 up to 256");
    if (cfg->rot_dim < 0 || cfg->rot_dim > d || cfg->rot_dim % 8)
        return fail(KVARN_EINVAL, "rot_dim must be a multiple of 8 up to head_dim");
    if ((cfg->in_type != KVARN_TYPE_F16 && cfg->in_type != KVARN_TYPE_BF16) ||
        (cfg->out_type != KVARN_TYPE_F16 && cfg->out_type != KVARN_TYPE_BF16))
        return fail(KVARN_EINVAL, "unknown type");
    if (!(cfg->eps >= 0.f) || !std::isfinite(cfg->eps)) return fail(KVARN_EINVAL, "eps must be finite and not negative");
    // the kernel counts items in 32 bits, a CTA's beyond the last one among them
    if (n_tokens < 0 || n_tokens > ((1ll << 31) - 1024) / (hq + hk)) return fail(KVARN_EINVAL, "bad token count");
    if (n_tokens == 0) return KVARN_OK;
    struct Side { const void* in; const void* out; int64_t heads, in_stride, out_stride; };
    for (const Side& s : {Side{q, q_out, hq, q_stride, q_out_stride}, Side{k, k_out, hk, k_stride, k_out_stride}}) {
        if (s.heads == 0) continue;
        if (!s.in || !s.out || !aligned16(s.in) || !aligned16(s.out))
            return fail(KVARN_EINVAL, "q, k and their outputs must be 16-byte aligned");
        if (s.in_stride < s.heads * d || s.out_stride < s.heads * d || s.in_stride % 8 || s.out_stride % 8)
            return fail(KVARN_EINVAL, "token strides must hold a token's heads and be multiples of 8 elements");
    }
    const Rows in[2] = {{q, hq * d, q_stride}, {k, hk * d, k_stride}};
    const Rows out[2] = {{q_out, hq * d, q_out_stride}, {k_out, hk * d, k_out_stride}};
    for (int i = 0; i < 2; ++i)  // an output on its own input is turned row by row
        for (int j = 0; j < 2; ++j) {
            if (in[i].len == 0 || out[j].len == 0) continue;
            if (i == j && in[i].at == out[i].at && (n_tokens == 1 || in[i].stride == out[i].stride)) continue;
            if (rows_meet(in[i], out[j], n_tokens))
                return fail(KVARN_EINVAL, "an output overlaps an input other than its own");
        }
    if (hq > 0 && hk > 0 && rows_meet(out[0], out[1], n_tokens)) return fail(KVARN_EINVAL, "the outputs overlap");
    if (cfg->rot_dim > 0 && (!positions || !freqs)) return fail(KVARN_EINVAL, "no positions or frequencies");
    if (!aligned16(q_weight) || !aligned16(k_weight)) return fail(KVARN_EINVAL, "weights must be 16-byte aligned");
    if (n_axes < 1 || n_axes > 255) return fail(KVARN_EINVAL, "1 to 255 axes of positions");
    if (axis_stride < 0 || axis_stride > (1ll << 48)) return fail(KVARN_EINVAL, "bad stride between axes");
    if (n_axes > 1 && cfg->rot_dim > 0 && !axes) return fail(KVARN_EINVAL, "several axes, but no axis for each pair");
    QkParams p;
    p.several = axes && n_axes > 1;
    p.axis_stride = axis_stride;
    std::memset(p.axes, 0, sizeof(p.axes));
    for (int i = 0; axes && i < cfg->rot_dim / 2; ++i) {
        if (axes[i] >= n_axes) return fail(KVARN_EINVAL, "a pair's axis is out of range");
        p.axes[i / 4] |= (uint32_t)axes[i] << 8 * (i % 4);
    }
    p.q = (const uint16_t*)q;
    p.k = (const uint16_t*)k;
    p.q_out = (uint16_t*)q_out;
    p.k_out = (uint16_t*)k_out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.positions = positions;
    p.freqs = freqs;
    p.n_tokens = n_tokens;
    p.hq = (int32_t)hq;
    p.hkv = (int32_t)hk;
    p.d = (int32_t)d;
    p.rot = cfg->rot_dim;
    p.interleaved = cfg->interleaved != 0;
    p.in_bf16 = cfg->in_type == KVARN_TYPE_BF16;
    p.out_bf16 = cfg->out_type == KVARN_TYPE_BF16;
    p.eps = cfg->eps;
    // Heads an item, a group's work in turn. Where the rows are not many times the resident groups (97,280
    // lanes): four, to have groups enough, or 16 of few tokens. Else all of a token's, so that its angles are
    // made once a side; 32 where a token's rows of very many heads would lie far apart.
    // (Measured, bf16 with weights, us: 1,000 tokens of 40 heads 8.2 by four, 10.3 by all; 4,000 of 72 43.3 by
    // four, 30.5 by all; 1,200 of 72 14.4 by four, 12.3 by 16, 16.4 by all; 2,000 of 128 26.7 by 32, 36.5 by all.)
    const int64_t heads = hq + hk, resident = 97280 / (d <= 64 ? 8 : d <= 128 ? 16 : 32);
    p.heads_per_item = n_tokens * heads <= 8 * resident ? 4 : n_tokens < resident / 4 ? 16 : heads <= 80 ? (int32_t)heads : 32;
    p.items_per_token = (int32_t)((heads + p.heads_per_item - 1) / p.heads_per_item);
    p.inv_d = 1.f / (float)d;
    const int rc = launch_qk_norm_rope(p, stream);
    return rc ? cuda_fail(rc, "norm and rotation launch") : KVARN_OK;
}

}  // extern "C"
