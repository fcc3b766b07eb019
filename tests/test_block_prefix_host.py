"""CPU tests of calls behind shared prefixes (include/kvarn.h): refusals and workspaces. No kernel is launched: caches here use
KVARN_FLAG_HOST_ONLY."""
import ctypes

import pytest
import torch

from quantized_kv_cache_seal_gb300 import kvarn as K
from quantized_kv_cache_seal_gb300.block_cache import BlockCache
from tests.test_block_host import FAKE, cache, refused
from tests.test_block_more_host import SPACE, W, filled


def test_window_behind_prefixes_refusals():
    c = filled()
    call = lambda ids, pre, m, q=FAKE, w=W, space=SPACE, n=1 << 40: K.kvarn_block_window_weights_prefixes(
        c, 0, ids, pre, m, q, 1.0, w, space, n)
    call([0, 1, 2], [5, -1, 5], [100, 1, 0])
    call([0], [4], [3])  # an empty prefix
    call([0], None, [3])
    for pre in ([6], [-2], [0], [2 ** 31 - 1]):
        refused(1, call, [0], pre, [1])
    refused(1, call, [0, 1], [1, -1], [1, 1])  # a prefix in the call
    refused(1, call, [0], [5], [101])
    refused(1, call, [5], [0], [129])
    refused(1, call, [0], [5], [1], FAKE, FAKE)
    refused(1, call, [0], [5], [1], FAKE, W, SPACE + 8)
    size = lambda *a: K.kvarn_block_window_workspace_prefixes(c, 0, *a)
    # sums of 2 heads, 4 tiles, 3 x 4 rows up to 16; rows of 2 (pairs) and a thread block a step, in three parts: a step of each
    # pair's own, three of the prefix
    need = lambda steps: 8 * 2 * 4 * 16 + (2 + 2 * steps) * 3 * 128 * 8
    assert size([0], [5], [3]) == need(1 + 3) and size([0], [-1], [3]) == size([0], None, [3]) == need(1)
    assert size([0], [4], [3]) == need(1) and size([2], [5], [0]) == 0
    for bad in (([6], [5], [1]), ([0], [6], [1]), ([0], [-2], [1]), ([0], [5], [101])):
        refused(1, size, *bad)
    call([0], [5], [3], n=need(4))
    refused(1, call, [0], [5], [3], n=need(4) - 1)
    # ids refused once are free for the next call
    call([0, 1], [5, 5], [1, 1])
    for wrong in ([5], [5, 5, 5]):
        with pytest.raises(ValueError):
            call([0, 1], wrong, [1, 1])
    L, n = K.load(), ctypes.c_size_t()
    assert L.kvarn_block_window_workspace_prefixes(None, 0, 0, None, None, None, ctypes.byref(n)) == 1
    assert L.kvarn_block_window_weights_prefixes(None, 0, 0, None, None, None, None, 1.0, None, None, 0, None) == 1
    K.kvarn_block_destroy(c)


def test_window_behind_prefixes_through_the_wrapper():
    c = BlockCache(max_seqs=4, num_q_heads=8, num_kv_heads=2, max_seq_len=1000, block_tokens=64, device="cpu",
                   flags=K.KVARN_FLAG_HOST_ONLY)
    w, kv = c.new_weights()[0], torch.zeros(100, 2, 128, dtype=torch.float16)
    c.append(0, [0, 3], [40, 60], kv, kv)
    q = torch.zeros(4, 8, 128, dtype=torch.float16)
    c.window_weights(0, [0, 1], [4, 0], q, w, prefix_ids=[3, None])
    with pytest.raises(K.KVarNError):
        c.window_weights(0, [0, 1], [4, 0], q, w, prefix_ids=[1, None])
    with pytest.raises(ValueError):
        c.window_weights(0, [0, 1], [4, 0], q, w, prefix_ids=[3])


def test_no_workspace_for_rows_that_no_launch_writes():
    """Prompts of many queries that walk their prefix themselves want no fp32 rows; questions whose rows stand together do."""
    up = lambda n: -(-n // 256) * 256
    c = cache(max_seqs=202, num_q_heads=32, num_kv_heads=8, max_seq_len=1 << 17, pool_blocks=1 << 14, num_layers=1)
    K.kvarn_block_append(c, 0, [0, 1, 201] + list(range(2, 201)), [65536, 70000, 16384] + [50] * 199, FAKE, 1024, FAKE, 1024)
    size = lambda *a: K.kvarn_block_attend_workspace(c, 0, *a)
    call = lambda ids, pre, m, space, n: K.kvarn_block_attend(c, 0, ids, pre, m, FAKE, FAKE, 1.0, None, space, n)
    for ids, pre, m in (([0], [201], [65536]), ([0, 1], [201, 201], [60000, 70000]), ([0, 1, 2], [201, -1, 200], [4096, 1, 50])):
        assert size(ids, pre, m) == 0
        call(ids, pre, m, None, 0)
    assert size([0], [201], [65000], True) == 0
    K.kvarn_block_append_attend(c, 0, [0], [201], [65000], FAKE, 1024, FAKE, 1024, FAKE, FAKE, 1.0, None, None, 0)
    # 199 questions of 40 tokens over 16,384: walked once
    ids, rows = list(range(2, 201)), 199 * 40 * 32
    need = up(rows * 128 * 4) + up(rows * 4)
    assert size(ids, [201] * 199, [40] * 199) == need
    call(ids, [201] * 199, [40] * 199, SPACE, need)
    refused(1, call, ids, [201] * 199, [40] * 199, SPACE, need - 1)
    refused(1, call, ids, [201] * 199, [40] * 199, None, need)
    # rows that no call could have: 2^32 of 2^14 bytes, more than a workspace may take
    refused(3, size, [0, 1], [201, 201], [2 ** 31 - 1] * 2)
    K.kvarn_block_destroy(c)


def test_a_long_prompt_leaves_the_wrappers_workspace():
    c = BlockCache(max_seqs=2, num_q_heads=8, num_kv_heads=2, max_seq_len=30000, block_tokens=64, device="cpu",
                   flags=K.KVARN_FLAG_HOST_ONLY)
    kv, q = torch.zeros(20300, 2, 128, dtype=torch.float16), torch.zeros(20000, 8, 128, dtype=torch.float16)
    c.append(0, [1], [300], kv[:300], kv[:300])
    c.prefill(0, [0], [20000], kv[300:], kv[300:], q, prefix_ids=[1])
    c.prefill_attention(0, [0], [20000], q, prefix_ids=[1])
    assert len(c._spaces) == 1


def test_steps_of_long_prompts_are_counted_exactly():
    """A prompt of 2^20 tokens has half of the 2^31 steps that its pairs would have if all were as long as the last: no more of a
    refusal with prefixes than without. Behind a prefix of as many tokens it has 2^31 more, and its second half 2^30."""
    n = 1 << 20
    c = cache(max_seqs=4, num_q_heads=64, num_kv_heads=64, max_seq_len=n, pool_blocks=1 << 16, num_layers=1)
    K.kvarn_block_append(c, 0, [0, 2], [n, 128], FAKE, 64 * 128, FAKE, 64 * 128)
    call = lambda pre, m: K.kvarn_block_attend(c, 0, [0], pre, [m], FAKE, 1 << 40, 1.0, None, SPACE, 1 << 40)
    K.kvarn_block_prefill_attention(c, 0, [0], [n], FAKE, 1 << 40, 1.0)
    for pre in (None, [-1], [3], [2]):
        call(pre, n)
    K.kvarn_block_append(c, 0, [1], [n], FAKE, 64 * 128, FAKE, 64 * 128)
    refused(3, call, [1], n)
    call([1], n // 2)
    K.kvarn_block_destroy(c)
