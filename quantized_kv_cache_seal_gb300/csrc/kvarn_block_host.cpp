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
int32_t head_tiles(int64_t n) { return (int32_t)std::max<int64_t>(1, (n + kTileTokens - 1) / kTileTokens); }
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

kvarn_status run_decode(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const void* q, void* out,
                        float scale, void* stream) {
    static thread_local BlockDecodeParams p;
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
        units += (int64_t)e.units * c->cfg.num_kv_heads;
    }
    p.units = units;
    // One CTA a SM, each of its eight warps a unit at least. Equal short sequences: whole (sequence, KV
    // head) pairs, so that nothing is joined across CTAs (which takes about as long as four rounds).
    const int64_t pairs = (int64_t)n_seqs * c->cfg.num_kv_heads, most = std::min(c->sms, kBlockMaxGrid);
    const bool equal = std::all_of(p.seqs, p.seqs + n_seqs, [](const BlockDecodeSeq& e) { return e.units == p.seqs[0].units; });
    p.grid = (int32_t)(equal && p.seqs[0].units <= 32 && pairs <= most ? pairs : std::min((units + 7) / 8, most));
    if (c->host_only) return KVARN_OK;
    const kvarn_status st = ensure_init(c, stream);
    if (st) return st;
    const int rc = launch_block_decode(p, stream);
    return rc ? cuda_fail(rc, "decode launch") : KVARN_OK;
}

kvarn_status run_prefill(kvarn_block_cache* c, int32_t layer, int32_t n_seqs, const int32_t* ids, const int32_t* q_lens,
                         const void* q, void* out, float scale, void* stream) {
    if (single_queries(n_seqs, q_lens)) {
        int32_t one[kBlockMaxSeqs];
        int32_t n = 0;
        for (int i = 0; i < n_seqs; ++i)
            if (q_lens[i] == 1) one[n++] = ids[i];
        return n ? run_decode(c, layer, n, one, q, out, scale, stream) : KVARN_OK;
    }
    static thread_local BlockPrefillParams p;
    p.c = c->view;
    p.c.layer = layer;
    p.q = (const uint16_t*)q;
    p.out = (uint16_t*)out;
    p.hq = c->cfg.num_q_heads;
    p.r = c->r;
    p.scale_log2 = scale * kLog2e;
    p.n_seqs = 0;
    const int hkv = c->cfg.num_kv_heads;
    int64_t row = 0;
    for (int i = 0; i < n_seqs; ++i) {
        if (q_lens[i] > 0) {
            BlockPrefillSeq& e = p.seqs[p.n_seqs++];
            e.seq = ids[i];
            e.n = c->L(ids[i], layer);
            e.q_len = q_lens[i];
            e.q_row = (int32_t)row;
        }
        row += q_lens[i];
    }
    if (p.n_seqs == 0) return KVARN_OK;
    // the longest sequences first: their segments are the longest
    std::sort(p.seqs, p.seqs + p.n_seqs, [](const BlockPrefillSeq& a, const BlockPrefillSeq& b) { return a.n > b.n; });
    int64_t segs = 0, steps = 0, longest = 0;
    for (int i = 0; i < p.n_seqs; ++i) {
        BlockPrefillSeq& e = p.seqs[i];
        e.pairs = (int32_t)head_pairs(c, e.q_len);
        e.seg_begin = (int32_t)segs;
        e.step_begin = (int32_t)steps;
        e.head_steps = (int32_t)head_steps(c, e.n, e.q_len);
        longest = std::max<int64_t>(longest, (e.n - 1) / 128 + 1);
        segs += (int64_t)e.pairs * hkv;
        steps += (int64_t)e.head_steps * hkv;
    }
    // Whole segments, the longest first, end when the longest does or the SMs have shared out all;
    // the line of all steps cut evenly ends a share of the steps later, and then costs about four more
    // for the partial results and the kernel that adds them (6 us where a step takes 1.5).
    const int64_t sms = std::min(c->sms, kBlockPrefillGrid);
    const int64_t share = (steps + sms - 1) / sms;
    const int64_t whole = segs >= 2 * sms ? share : std::max(share, longest * ((segs + sms - 1) / sms));
    p.line = whole > share + 4;
    p.steps = (int32_t)steps;
    p.segs = (int32_t)segs;
    p.grid = (int32_t)std::min<int64_t>(sms, p.line ? steps : segs);
    if (c->host_only) return KVARN_OK;
    const kvarn_status st = ensure_init(c, stream);
    if (st) return st;
    const int rc = launch_block_prefill(p, stream);
    return rc ? cuda_fail(rc, "prefill launch") : KVARN_OK;
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
    QkParams p;
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
