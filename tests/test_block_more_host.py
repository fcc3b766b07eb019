"""CPU tests of attention over shared prefixes, of the blocks' weights and of eviction (include/kvarn.h): refusals,
workspaces, lengths and pool. No kernel is launched: caches here use KVARN_FLAG_HOST_ONLY."""
import ctypes

import pytest
import torch

from quantized_kv_cache_seal_gb300 import kvarn as K
from quantized_kv_cache_seal_gb300.block_cache import BlockCache
from tests.test_block_host import FAKE, FAR, cache, refused

SPACE, W, KEPT = FAR, 2 * FAR, 3 * FAR


def filled(**kw):
    c = cache(**dict(dict(max_seqs=6), **kw))
    K.kvarn_block_append(c, 0, [0, 1, 5], [100, 70, 300], FAKE, 256, FAKE, 256)
    return c


def attend(c, ids, pre, m, q=FAKE, out=FAKE, scale=1.0, weights=None, space=SPACE, n=1 << 40, layer=0):
    K.kvarn_block_attend(c, layer, ids, pre, m, q, out, scale, weights, space, n)


def test_attend_refusals():
    c = filled()
    attend(c, [0, 1, 2], [5, 5, -1], [3, 70, 0])
    attend(c, [0, 1, 2], [5, 4, 3], None)
    attend(c, [], [], None, None, None)
    attend(c, [0], None, None, weights=W)
    for pre in ([6], [-2], [0], [2 ** 31 - 1]):
        refused(1, attend, c, [0], pre, None)
    refused(1, attend, c, [0, 1], [1, -1], None)  # a prefix in the call
    refused(1, attend, c, [0], [5], [101])
    refused(1, attend, c, [0, 0], [5, 5], None)
    refused(1, attend, c, [0], [5], None, out=None)
    refused(1, attend, c, [0], [5], None, q=FAKE + 2)
    refused(1, attend, c, [0], [5], None, scale=float("nan"))
    refused(1, attend, c, [0], [5], None, space=None)
    refused(1, attend, c, [0], [5], None, space=SPACE + 8)
    refused(1, attend, c, [0], [5], None, layer=2)
    refused(1, attend, c, [0], None, [2], weights=W)  # weights are of single queries
    refused(1, attend, c, [0], None, None, weights=W + 2)
    need = K.kvarn_block_attend_workspace(c, 0, [0], [5], None, False, True)
    attend(c, [0], [5], None, weights=W, n=need)
    refused(1, attend, c, [0], [5], None, weights=W, n=need - 1)
    # weights or workspace over queries, output or one another
    refused(1, attend, c, [0], [5], None, weights=FAKE)
    refused(1, attend, c, [0], [5], None, space=FAKE)
    refused(1, attend, c, [0], [5], None, weights=SPACE)
    refused(3, attend, cache(max_seqs=300), list(range(257)), [299] * 257, None)
    # ids refused once are free for the next call
    attend(c, [0, 1], [5, 5], None)
    K.kvarn_block_destroy(c)


def test_a_refused_append_changes_nothing():
    c = filled()
    call = lambda pre, out=FAKE, n=1 << 40, w=None, m=(1, 1): K.kvarn_block_append_attend(
        c, 0, [0, 1], pre, list(m), FAKE, 256, FAKE, 256, FAKE, out, 1.0, w, SPACE, n)
    refused(1, call, [5, 1])
    refused(1, call, [5, 6])
    refused(1, call, [5, 5], None)
    refused(1, call, [5, 5], FAKE, 0)
    refused(1, call, [5, 5], FAKE, 1 << 40, W, (2, 1))
    refused(3, call, [5, 5], FAKE, 1 << 40, None, (1000, 1))
    assert [K.kvarn_block_length(c, 0, s) for s in (0, 1, 5)] == [100, 70, 300]
    call([5, 5], FAKE, 1 << 40, W)
    call([5, -1], FAKE, 1 << 40, None, (3, 0))
    assert [K.kvarn_block_length(c, 0, s) for s in (0, 1, 5)] == [104, 71, 300]
    K.kvarn_block_destroy(c)


def test_workspace_sizes():
    c = filled()
    size = lambda *a: K.kvarn_block_attend_workspace(c, 0, *a)
    up = lambda n: -(-n // 256) * 256
    assert size([0, 1], None, None) == 0 and size([0, 1], [-1, -1], None) == 0
    rows = 2 * 8
    assert size([0, 1], [5, -1], None) == up(rows * 128 * 4) + up(rows * 4)
    assert size([0, 1], [5, 5], [100, 3]) == up(103 * 8 * 128 * 4) + up(103 * 8 * 4)
    # tiles of 32 tokens and eight more a sequence, heads, 8 bytes
    # and a row's totals
    assert size([0, 1], None, None, False, True) == up((4 + 3 + 2 * 8) * 8 * 8) + up(2 * 8 * 8)
    assert size([2], None, None, False, True) == up((1 + 8) * 8 * 8) + up(8 * 8)  # an empty sequence has one
    assert size([0], None, [29], True, True) == up((5 + 8) * 8 * 8) + up(29 * 8 * 8)
    assert size([0], [5], None, False, True) == up(8 * 128 * 4) + up(8 * 4) + up((4 + 10 + 8) * 8 * 8) + up(8 * 8)
    for bad in (([6], None, None), ([0], [6], None), ([0], None, [-1])):
        refused(1, size, *bad)
    refused(1, K.kvarn_block_attend_workspace, c, 2, [0], None, None)
    refused(1, K.kvarn_block_attend_workspace, c, 0, [0], None, None, True)
    K.kvarn_block_destroy(c)


def test_window_refusals():
    c = filled()
    call = lambda ids, m, q=FAKE, w=W, space=SPACE, n=1 << 40, scale=1.0: K.kvarn_block_window_weights(
        c, 0, ids, m, q, scale, w, space, n)
    call([0, 1, 2], [100, 1, 0])
    call([5], [128])
    call([2], [0], None, None, None, 0)
    refused(1, call, [5], [129])
    refused(1, call, [0], [101])
    refused(1, call, [0], [-1])
    refused(1, call, [0], [1], None)
    refused(1, call, [0], [1], FAKE + 2)
    refused(1, call, [0], [1], FAKE, None)
    refused(1, call, [0], [1], FAKE, W + 1)
    refused(1, call, [0], [1], FAKE, FAKE)
    refused(1, call, [0], [1], FAKE, W, None)
    refused(1, call, [0], [1], FAKE, W, SPACE + 8)
    refused(1, call, [0], [1], scale=float("inf"))
    size = lambda *a: K.kvarn_block_window_workspace(c, 0, *a)
    # sums of 2 heads, 4 tiles, 3 x 4 rows up to 16; rows of 2 (pairs) + 2 (thread blocks), in three parts
    need = 8 * 2 * 4 * 16 + (2 + 2) * 3 * 128 * 8
    assert size([0], [3]) == need and size([2], [0]) == 0
    for bad in (([6], [1]), ([0], [101]), ([0], [-1]), ([5], [129])):
        refused(1, size, *bad)
    call([0], [3], n=need)
    refused(1, call, [0], [3], n=need - 1)
    refused(1, call, [0, 0], [1, 1])
    with pytest.raises(ValueError):
        call([0, 1], [1])
    K.kvarn_block_destroy(c)


def test_evict_refusals_lengths_and_pool():
    c = filled(pool_blocks=9)  # 1 + 1 + 4 blocks of 64 are taken
    call = lambda ids, keep, first=0, last=0, w=W, kept=KEPT: K.kvarn_block_evict(c, 0, ids, keep, first, last, w, kept)
    for keep, first, last in ((-1, 0, 0), (2, 2, 1), (1, -1, 0), (1, 0, -1), (2 ** 31 - 1, 2 ** 31 - 1, 1)):
        refused(1, call, [5], keep, first, last)
    refused(1, call, [5], 2, 0, 0, None)
    refused(1, call, [5], 2, 0, 0, W + 2)
    refused(1, call, [5], 2, 0, 0, W, None)
    refused(1, call, [5], 2, 0, 0, W, KEPT + 2)
    refused(1, call, [5], 2, 0, 0, W, W + 8)
    refused(1, call, [6], 2)
    refused(1, call, [5, 5], 2)
    lengths = lambda: [K.kvarn_block_length(c, 0, s) for s in (0, 1, 2, 5)]
    assert lengths() == [100, 70, 0, 300]
    refused(3, K.kvarn_block_append, c, 0, [2], [256], FAKE, 256, FAKE, 256)  # 3 free
    call([0, 5, 2], 4, 2, 2)
    assert lengths() == [100, 70, 0, 300]
    call([5, 0], 2, 1, 1)
    assert lengths() == [100, 70, 0, 172]
    K.kvarn_block_append(c, 0, [2], [320], FAKE, 256, FAKE, 256)  # 5 free
    refused(3, K.kvarn_block_append, c, 0, [2], [64], FAKE, 256, FAKE, 256)
    call([0, 1, 2, 5], 0, 0, 0, W, None)
    assert lengths() == [36, 6, 0, 44]
    K.kvarn_block_append(c, 0, [2], [9 * 64], FAKE, 256, FAKE, 256)
    K.kvarn_block_release(c, [0, 1, 2, 5])
    assert lengths() == [0, 0, 0, 0]
    K.kvarn_block_append(c, 0, [3], [9 * 64], FAKE, 256, FAKE, 256)
    K.kvarn_block_destroy(c)


def test_work_that_32_bits_cannot_count():
    """Steps and tiles of long prefixes under many queries are refused before anything moves."""
    c = cache(max_seqs=200, num_q_heads=64, num_kv_heads=64, head_dim=64, block_tokens=128, max_seq_len=2 ** 30,
              pool_blocks=0, num_layers=1)
    # the cache is too large to be filled: lengths stay 0, and then there is nothing to refuse
    attend(c, list(range(199)), [199] * 199, None)
    K.kvarn_block_destroy(c)
    c = cache(max_seqs=3, num_q_heads=8192, num_kv_heads=8192, head_dim=64, block_tokens=32, max_seq_len=2 ** 25,
              pool_blocks=2 ** 20, num_layers=1)
    K.kvarn_block_append(c, 0, [2], [2 ** 25 - 31], FAKE, 8192 * 64, FAKE, 8192 * 64)
    refused(3, attend, c, [0, 1], [2, 2], None)
    K.kvarn_block_destroy(c)


def test_wrapper_checks_tensors():
    c = BlockCache(max_seqs=4, num_q_heads=8, num_kv_heads=2, max_seq_len=1000, block_tokens=64, device="cpu",
                   flags=K.KVARN_FLAG_HOST_ONLY)
    w = c.new_weights()
    assert w.shape == (1, 4, 2, 1000 // 64 + 1) and w.dtype is torch.float32 and not w.any()
    kv = torch.zeros(100, 2, 128, dtype=torch.float16)
    c.append(0, [0, 3], [40, 60], kv, kv)
    q = torch.zeros(4, 8, 128, dtype=torch.float16)
    c.decode_attention(0, [0, 1], q[:2], prefix_ids=[3, None], weights=w[0])
    c.decode_step(0, [0, 1], kv[:2], kv[:2], q[:2], prefix_ids=[3, None], weights=w[0])
    c.prefill_attention(0, [0, 1], [2, 1], q[:3], prefix_ids=[3, 3])
    c.prefill(0, [0, 1], [2, 1], kv[:3], kv[:3], q[:3], prefix_ids=[3, -1])
    c.window_weights(0, [0, 1], [3, 1], q, w[0])
    assert c.evict(0, [0, 1], w[0], 2).shape == (2, 2, 2)
    assert [c.length(0, s) for s in range(4)] == [43, 2, 0, 60]
    for bad in (w, w[0].double(), w[0][..., 1:], w[0].transpose(0, 1), w[0][:3]):
        for call in (lambda: c.decode_attention(0, [0, 1], q[:2], weights=bad),
                     lambda: c.window_weights(0, [0, 1], [3, 1], q, bad), lambda: c.evict(0, [0], bad, 2),
                     lambda: c.decode_step(0, [0, 1], kv[:2], kv[:2], q[:2], weights=bad)):
            with pytest.raises(ValueError):
                call()
    for call in (lambda: c.decode_attention(0, [0, 1], q[:2], prefix_ids=[3]),
                 lambda: c.prefill_attention(0, [0, 1], [1], q[:1], prefix_ids=[3, 3]),
                 lambda: c.window_weights(0, [0, 1], [3], q[:3], w[0]), lambda: c.window_weights(0, [0], [3], q, w[0]),
                 lambda: c.evict(0, [0], w[0], -1), lambda: c.evict(0, [0], w[0], 2 ** 31)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(K.KVarNError):
        c.decode_attention(0, [0, 1], q[:2], prefix_ids=[3, 0])
    assert [c.length(0, s) for s in range(4)] == [43, 2, 0, 60]


def test_norm_rope_axes_refusals():
    cfg = K.kvarn_qk_config(8, 2, 128, 64, 0, 0, 0, 1e-6)

    def call(axes=bytes(i % 3 for i in range(32)), count=3, stride=10, tokens=10, cfg=cfg):
        K.kvarn_qk_norm_rope_axes(cfg, tokens, FAKE, 1024, FAR, 256, None, None, FAKE, stride, count, axes, FAKE, 2 * FAR,
                                  1024, 3 * FAR, 256)

    call(tokens=0)
    for kw in (dict(count=0), dict(count=256), dict(stride=-1), dict(axes=None), dict(count=2), dict(axes=bytes([255] * 32)),
               dict(stride=2 ** 60)):
        refused(1, call, **kw)
    with pytest.raises(ValueError):
        call(axes=bytes(31))


def test_null_arguments():
    L = K.load()
    n = ctypes.c_size_t()
    assert L.kvarn_block_attend_workspace(None, 0, 0, None, None, None, 0, 0, ctypes.byref(n)) == 1
    assert L.kvarn_block_attend(None, 0, 0, None, None, None, None, None, 1.0, None, None, 0, None) == 1
    assert L.kvarn_block_append_attend(None, 0, 0, None, None, None, None, 0, None, 0, None, None, 1.0, None, None, 0, None) == 1
    assert L.kvarn_block_window_workspace(None, 0, 0, None, None, ctypes.byref(n)) == 1
    assert L.kvarn_block_window_weights(None, 0, 0, None, None, None, 1.0, None, None, 0, None) == 1
    assert L.kvarn_block_evict(None, 0, 0, None, 0, 0, 0, None, None, None) == 1
    c = cache()
    assert L.kvarn_block_attend_workspace(c, 0, 0, None, None, None, 0, 0, None) == 1
    assert L.kvarn_block_window_weights(c, 0, 1, K._i32([0]), None, FAKE, 1.0, W, SPACE, 1 << 30, None) == 1
    assert L.kvarn_block_append_attend(c, 0, 1, K._i32([0]), None, None, FAKE, 256, FAKE, 256, FAKE, FAKE, 1.0, None, None, 0, None) == 1
    K.kvarn_block_destroy(c)


def test_weights_of_too_many_heads():
    c = cache(num_q_heads=65536, num_kv_heads=65536, head_dim=64, block_tokens=32, max_seqs=2, pool_blocks=0, num_layers=1)
    refused(3, attend, c, [0], None, None, weights=W)
    attend(c, [0], [1], None)
    K.kvarn_block_destroy(c)
