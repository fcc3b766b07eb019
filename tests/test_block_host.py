"""CPU tests of the block cache and of the query/key norm + rotation (include/kvarn.h): refusals, pool and length
bookkeeping. No kernel is launched: caches here use KVARN_FLAG_HOST_ONLY."""
import ctypes

import pytest
import torch

from quantized_kv_cache_seal_gb300 import kvarn as K
from quantized_kv_cache_seal_gb300.block_cache import BlockCache
from quantized_kv_cache_seal_gb300.qk import qk_norm_rope

FAKE = 1 << 30  # a device address that is never dereferenced in host-only mode
FAR = 1 << 45  # another, beyond any tensor at FAKE


def config(**kw):
    args = dict(num_layers=2, max_seqs=4, num_q_heads=8, num_kv_heads=2, head_dim=128, block_tokens=64, code=0, type=0,
                max_seq_len=1000, pool_blocks=20, flags=K.KVARN_FLAG_HOST_ONLY)
    args.update(kw)
    return K.kvarn_block_config(*[args[n] for n, _ in K.kvarn_block_config._fields_])


def cache(**kw):
    cfg = config(**kw)
    return K.kvarn_block_create(cfg, FAKE, K.kvarn_block_required_bytes(cfg))


def refused(status, call, *args, **kw):
    with pytest.raises(K.KVarNError) as e:
        call(*args, **kw)
    assert e.value.status == status
    assert "(" in str(e.value)  # the reason is told
    return str(e.value)


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(head_dim=0), dict(block_tokens=16), dict(block_tokens=256), dict(code=2), dict(type=2),
    dict(num_q_heads=7), dict(num_q_heads=18), dict(num_kv_heads=0), dict(num_layers=0), dict(max_seqs=-1),
    dict(max_seq_len=0), dict(max_seq_len=2 ** 30 + 1), dict(pool_blocks=-1), dict(flags=2), dict(num_layers=2 ** 31 - 1, max_seqs=2 ** 31 - 1),
    dict(num_layers=2 ** 30, max_seqs=1, max_seq_len=2 ** 31 - 1)])
def test_bad_configurations(bad):
    refused(1, K.kvarn_block_required_bytes, config(**bad))
    refused(1, K.kvarn_block_create, config(**bad), FAKE, 1 << 60)


def test_create_refusals():
    cfg = config()
    n = K.kvarn_block_required_bytes(cfg)
    refused(2, K.kvarn_block_create, cfg, FAKE, n - 1)
    refused(1, K.kvarn_block_create, cfg, FAKE + 16, n)
    refused(1, K.kvarn_block_create, cfg, None, n)


def test_required_bytes_counts_the_pool():
    a, b = (K.kvarn_block_required_bytes(config(pool_blocks=n)) for n in (0, 64))
    # a slot: per KV head, 2 tiles of 32 tokens, K and V at 128 bytes a token, 16 bytes of scales a tile
    assert b - a == 64 * 2 * 2 * (16 + 2 * 32 * 128)
    assert K.kvarn_block_required_bytes(config(head_dim=64)) < a + 64 * 2 * 2 * (16 + 2 * 32 * 128)


def test_lengths_and_pool():
    c = cache()
    row = 2 * 128
    K.kvarn_block_append(c, 0, [1, 3], [130, 63], FAKE, row, FAKE, row)
    assert [K.kvarn_block_length(c, 0, s) for s in range(4)] == [0, 130, 0, 63]
    assert K.kvarn_block_length(c, 1, 1) == 0
    K.kvarn_block_append(c, 0, [3], [1], FAKE, 3 * row, FAKE, 4 * row)  # strided; the block fills
    K.kvarn_block_append(c, 1, [0], [1000], FAKE, row, FAKE, row)  # 15 blocks: 18 of 20 in use
    refused(3, K.kvarn_block_append, c, 0, [0], [3 * 64], FAKE, row, FAKE, row)
    assert K.kvarn_block_length(c, 0, 0) == 0
    refused(3, K.kvarn_block_append, c, 1, [0], [1], FAKE, row, FAKE, row)  # max_seq_len
    K.kvarn_block_append(c, 0, [0], [2 * 64 + 63], FAKE, row, FAKE, row)  # exactly the pool
    refused(3, K.kvarn_block_append, c, 0, [0], [1], FAKE, row, FAKE, row)
    K.kvarn_block_release(c, [0, 0])
    assert K.kvarn_block_length(c, 1, 0) == 0
    K.kvarn_block_append(c, 0, [0], [17 * 64 - 88], FAKE, row, FAKE, row)
    assert K.kvarn_block_length(c, 0, 0) == 1000
    K.kvarn_block_append(c, 0, [], [], None, 0, None, 0)
    K.kvarn_block_destroy(c)


def test_slots_are_handed_out_once():
    """Appends and releases in a random order never need more blocks than the live tokens fill."""
    import random
    rng = random.Random(5)
    c = cache(max_seqs=6, max_seq_len=2000, pool_blocks=40)
    length, row = [0] * 6, 256
    for _ in range(2000):
        s = rng.randrange(6)
        if rng.random() < 0.2:
            K.kvarn_block_release(c, [s])
            length[s] = 0
            continue
        n = rng.choice([1, 5, 63, 64, 65, 300])
        used = sum(x // 64 for x in length)
        fits = length[s] + n <= 2000 and used + (length[s] + n) // 64 - length[s] // 64 <= 40
        if fits:
            K.kvarn_block_append(c, 0, [s], [n], FAKE, row, FAKE, row)
            length[s] += n
        else:
            refused(3, K.kvarn_block_append, c, 0, [s], [n], FAKE, row, FAKE, row)
        assert K.kvarn_block_length(c, 0, s) == length[s]
    K.kvarn_block_destroy(c)


def test_large_appends_are_cut():
    """More blocks than one launch's parameters hold."""
    c = cache(max_seqs=3, max_seq_len=400000, pool_blocks=15000, block_tokens=32)
    K.kvarn_block_append(c, 0, [0, 1, 2], [170001, 31, 300000], FAKE, 256, FAKE, 256)
    assert [K.kvarn_block_length(c, 0, s) for s in range(3)] == [170001, 31, 300000]
    refused(3, K.kvarn_block_append, c, 0, [1], [32 * (15000 - 5312 - 9375) + 1], FAKE, 256, FAKE, 256)
    K.kvarn_block_append(c, 0, [1], [32 * (15000 - 5312 - 9375)], FAKE, 256, FAKE, 256)
    K.kvarn_block_destroy(c)


def test_append_refusals():
    c = cache()
    ok = (FAKE, 256, FAKE, 256)
    for layer in (-1, 2):
        refused(1, K.kvarn_block_append, c, layer, [0], [1], *ok)
    for ids in ([-1], [4], [1, 1]):
        refused(1, K.kvarn_block_append, c, 0, ids, [1] * len(ids), *ok)
    refused(1, K.kvarn_block_append, c, 0, [0], [-1], *ok)
    refused(1, K.kvarn_block_append, c, 0, [0], [1], None, 256, FAKE, 256)
    refused(1, K.kvarn_block_append, c, 0, [0], [1], FAKE, 256, FAKE + 8, 256)
    refused(1, K.kvarn_block_append, c, 0, [0], [1], FAKE, 255, FAKE, 256)
    refused(1, K.kvarn_block_append, c, 0, [0], [1], FAKE, 256, FAKE, 260)
    refused(3, K.kvarn_block_append, cache(max_seqs=300), 0, list(range(257)), [1] * 257, *ok)
    # an id refused once is free for the next call
    K.kvarn_block_append(c, 0, [1], [1], *ok)
    K.kvarn_block_destroy(c)


def test_read_and_attention_refusals():
    c = cache()
    K.kvarn_block_append(c, 0, [0], [100], FAKE, 256, FAKE, 256)
    for start, count in ((-1, 1), (0, 101), (100, 1), (2 ** 31 - 1, 1)):
        refused(1, K.kvarn_block_read, c, 0, [0], [start], [count], FAKE, FAKE)
    refused(1, K.kvarn_block_read, c, 0, [0], [0], [-1], FAKE, FAKE)
    refused(1, K.kvarn_block_read, c, 0, [0], None, [1], FAKE, None)
    K.kvarn_block_read(c, 0, [0, 1], [100, 0], [0, 0], None, None)
    K.kvarn_block_read(c, 0, [0], None, [100], FAKE, FAKE)
    for scale in (float("nan"), float("inf")):
        refused(1, K.kvarn_block_decode_attention, c, 0, [0], FAKE, FAKE, scale)
    refused(1, K.kvarn_block_decode_attention, c, 0, [0], FAKE + 2, FAKE, 1.0)
    refused(1, K.kvarn_block_decode_attention, c, 0, [0], FAKE, None, 1.0)
    refused(1, K.kvarn_block_prefill_attention, c, 0, [0], [101], FAKE, FAKE, 1.0)
    refused(1, K.kvarn_block_prefill_attention, c, 0, [0], [-1], FAKE, FAKE, 1.0)
    K.kvarn_block_prefill_attention(c, 0, [0, 1], [100, 0], FAKE, FAKE, 1.0)
    K.kvarn_block_decode_attention(c, 0, [], None, None, 1.0)
    # a refused step or prefill appends nothing
    refused(1, K.kvarn_block_decode_step, c, 0, [0], FAKE, 256, FAKE, 256, FAKE, None, 1.0)
    refused(1, K.kvarn_block_prefill, c, 0, [0], [5], FAKE, 256, FAKE, 256, None, FAKE, 1.0)
    assert K.kvarn_block_length(c, 0, 0) == 100
    K.kvarn_block_decode_step(c, 0, [0], FAKE, 256, FAKE, 256, FAKE, FAKE, 1.0)
    K.kvarn_block_prefill(c, 0, [0, 2], [5, 7], FAKE, 256, FAKE, 256, FAKE, FAKE, 1.0)
    assert [K.kvarn_block_length(c, 0, s) for s in range(4)] == [106, 0, 7, 0]
    refused(1, K.kvarn_block_length, c, 0, 4)
    refused(1, K.kvarn_block_release, c, [4])
    assert K.kvarn_block_check_device_error(c) == 0
    K.kvarn_block_destroy(c)


def test_ids_that_do_not_fit():
    """Numbers beyond 32 bits are refused, not cut."""
    c = cache()
    for bad in ([2 ** 32], [2 ** 31], [-2 ** 31 - 1]):
        with pytest.raises(OverflowError):
            K.kvarn_block_append(c, 0, bad, [1], FAKE, 256, FAKE, 256)
        with pytest.raises(OverflowError):
            K.kvarn_block_append(c, 0, [0], bad, FAKE, 256, FAKE, 256)
        with pytest.raises(OverflowError):
            K.kvarn_block_release(c, bad)
    with pytest.raises(TypeError):
        K.kvarn_block_append(c, 0, [0.5], [1], FAKE, 256, FAKE, 256)
    K.kvarn_block_destroy(c)


def test_null_cache():
    L = K.load()
    one = (ctypes.c_int32 * 1)(0)
    assert L.kvarn_block_append(None, 0, 1, one, one, FAKE, 256, FAKE, 256, None) == 1
    assert L.kvarn_block_decode_attention(None, 0, 1, one, FAKE, FAKE, 1.0, None) == 1
    assert L.kvarn_block_release(None, 0, None) == 1
    L.kvarn_block_destroy(None)


def test_wrapper_checks_tensors():
    c = BlockCache(max_seqs=2, num_q_heads=8, num_kv_heads=2, max_seq_len=256, device="cpu",
                   flags=K.KVARN_FLAG_HOST_ONLY)
    k = torch.zeros(5, 2, 128, dtype=torch.float16)
    c.append(0, [0], [5], k, k)
    packed = torch.zeros(5, 12, 128, dtype=torch.float16)
    c.append(0, [0], [5], packed[:, 8:10], packed[:, 10:])
    assert c.length(0, 0) == 10
    for bad in (k.float(), k[:4], k.transpose(0, 1), torch.zeros(5, 2, 256, dtype=torch.float16)[..., ::2]):
        with pytest.raises(ValueError):
            c.append(0, [0], [5], bad, k)
    with pytest.raises(ValueError):
        c.append(0, [0, 1], [5], k, k)
    q = torch.zeros(1, 8, 128, dtype=torch.float16)
    assert c.decode_attention(0, [0], q).shape == q.shape
    for bad in (q[:, :4], q.bfloat16(), torch.zeros(1, 128, 8, dtype=torch.float16).transpose(1, 2)):
        with pytest.raises(ValueError):
            c.decode_attention(0, [0], bad)
        with pytest.raises(ValueError):
            c.decode_attention(0, [0], q, out=bad)
    with pytest.raises(ValueError):
        c.prefill_attention(0, [0], [1, 1], q)
    with pytest.raises(ValueError):
        c.read(0, [0], None, [5], dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        c.read(0, [0], [0], [-5])
    with pytest.raises(ValueError):
        BlockCache(code="fp4", device="cpu")
    assert c.read(0, [0], None, [5], dtype=torch.float32)[0].shape == (5, 2, 128)


def qk(**kw):
    args = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, rot_dim=128, interleaved=0, in_type=0, out_type=0, eps=1e-6)
    args.update(kw)
    return K.kvarn_qk_config(*[args[n] for n, _ in K.kvarn_qk_config._fields_])


def test_norm_rope_refusals():
    good = [4, FAKE, 1024, FAKE, 256, None, None, FAKE, FAKE, FAKE, 1024, FAKE, 256]

    def call(cfg, **at):
        a = list(good)
        for i, v in at.items():
            a[int(i[1:])] = v
        refused(1, K.kvarn_qk_norm_rope, cfg, *a)

    for bad in (dict(head_dim=12), dict(head_dim=264), dict(rot_dim=136), dict(rot_dim=4), dict(rot_dim=-8), dict(in_type=2),
                dict(out_type=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(num_q_heads=0, num_kv_heads=0),
                dict(num_q_heads=-1)):
        call(qk(**bad))
    call(qk(), a0=-1)
    call(qk(), a0=1 << 40)
    for i in (1, 3, 7, 8, 9, 11):
        call(qk(), **{f"a{i}": None})
    call(qk(), a1=FAKE + 2)
    for i, v in ((2, 1023), (2, 1028), (4, 255), (10, 8), (12, 260)):
        call(qk(), **{f"a{i}": v})
    K.kvarn_qk_norm_rope(qk(), 0, None, 0, None, 0, None, None, None, None, None, 0, None, 0)  # no tokens


def test_norm_rope_token_counts_that_do_not_fit():
    """Products of tokens and heads that leave 64 bits, or 32 bits together with a CTA's share behind the last token."""
    big = 1 << 60  # times 16 heads: 0 modulo 2^64
    refused(1, K.kvarn_qk_norm_rope, qk(num_q_heads=8, num_kv_heads=8), big, FAKE, 1024, FAKE, 1024, None, None, FAKE, FAKE,
            FAKE, 1024, FAKE, 1024)
    one = qk(num_q_heads=1, num_kv_heads=0, head_dim=8, rot_dim=8)
    refused(1, K.kvarn_qk_norm_rope, one, (1 << 31) - 1, FAKE, 8, None, 0, None, None, FAKE, FAKE, FAKE, 8, None, 0)


def test_scale_that_leaves_fp32():
    c = cache()
    refused(1, K.kvarn_block_decode_attention, c, 0, [0], FAKE, FAKE, 3e38)  # times log2 e
    refused(1, K.kvarn_block_prefill_attention, c, 0, [0], [0], FAKE, FAKE, -3e38)
    K.kvarn_block_destroy(c)


def test_norm_rope_wrapper_wants_cuda_tensors():
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        qk_norm_rope(q, None, torch.zeros(3, dtype=torch.int32), torch.ones(32, dtype=torch.float64))


def test_calls_of_too_much_work_change_nothing():
    """A prefill of 2^31 steps, a decode step of 2^31 tiles: refused before anything is appended."""
    n = (1 << 20) + 128  # 16 heads, 32 queries a pair of tiles: n / 32 pairs of n / 128 / 2 steps each, on average
    c = cache(num_layers=1, num_q_heads=128, num_kv_heads=16, max_seq_len=n + 1, block_tokens=128, pool_blocks=n // 128)
    refused(3, K.kvarn_block_prefill, c, 0, [2], [n], FAKE, 2048, FAKE, 2048, FAKE, FAR, 1.0)
    assert K.kvarn_block_length(c, 0, 2) == 0
    K.kvarn_block_append(c, 0, [2], [n], FAKE, 2048, FAKE, 2048)  # every block of the pool was still free
    refused(3, K.kvarn_block_prefill_attention, c, 0, [2], [n], FAKE, FAR, 1.0)
    K.kvarn_block_prefill_attention(c, 0, [2], [n // 2], FAKE, FAR, 1.0)
    K.kvarn_block_destroy(c)
    n = 1 << 24  # 128 heads of 32 sequences of n tokens: 2^31 tiles of 32 tokens
    c = cache(num_layers=1, max_seqs=32, num_q_heads=128, num_kv_heads=128, head_dim=64, max_seq_len=n + 1, block_tokens=128,
              pool_blocks=32 * n // 128)
    ids, kv = list(range(32)), (FAKE, 8192, FAKE, 8192)
    K.kvarn_block_append(c, 0, ids, [n - 33] * 32, *kv)
    K.kvarn_block_decode_step(c, 0, ids, *kv, FAKE, FAR, 1.0)
    for step in (K.kvarn_block_decode_step, K.kvarn_block_prefill):
        counts = ([1] * 32,) if step is K.kvarn_block_prefill else ()
        refused(3, step, c, 0, ids, *counts, *kv, FAKE, FAR, 1.0)  # each at a new tile
        assert [K.kvarn_block_length(c, 0, s) for s in ids] == [n - 32] * 32
    K.kvarn_block_append(c, 0, ids, [1] * 32, *kv)
    refused(3, K.kvarn_block_decode_attention, c, 0, ids, FAKE, FAR, 1.0)
    refused(3, K.kvarn_block_prefill_attention, c, 0, ids, [1] * 32, FAKE, FAR, 1.0)
    K.kvarn_block_prefill_attention(c, 0, ids, [1] * 31 + [0], FAKE, FAR, 1.0)
    K.kvarn_block_decode_attention(c, 0, ids[:31], FAKE, FAR, 1.0)
    K.kvarn_block_destroy(c)


def test_outputs_that_overlap_the_queries():
    """out is q itself or lies apart from it."""
    c = cache()
    K.kvarn_block_append(c, 0, [0], [100], FAKE, 256, FAKE, 256)
    q, row = FAKE + (1 << 20), 8 * 128 * 2  # bytes of a row
    for out in (q - row + 16, q - 16, q + 16, q + row - 16):
        refused(1, K.kvarn_block_decode_attention, c, 0, [0], q, out, 1.0)
        refused(1, K.kvarn_block_prefill_attention, c, 0, [0], [100], q, out, 1.0)
        refused(1, K.kvarn_block_decode_step, c, 0, [0], FAKE, 256, FAKE, 256, q, out, 1.0)
        refused(1, K.kvarn_block_prefill, c, 0, [0], [2], FAKE, 256, FAKE, 256, q, out, 1.0)
    refused(1, K.kvarn_block_prefill_attention, c, 0, [0], [100], q, q + 99 * row, 1.0)
    refused(1, K.kvarn_block_prefill_attention, c, 0, [0], [100], q, q - 99 * row, 1.0)
    assert K.kvarn_block_length(c, 0, 0) == 100
    for out in (q, q - row, q + row):
        K.kvarn_block_decode_attention(c, 0, [0], q, out, 1.0)
    for out in (q, q - 100 * row, q + 100 * row):
        K.kvarn_block_prefill_attention(c, 0, [0], [100], q, out, 1.0)
    K.kvarn_block_destroy(c)


def test_norm_rope_outputs_that_overlap():
    """An output is its own input or touches no other tensor: packed rows with and without gaps, different strides."""
    b = 2  # bytes of a value

    def call(n, q, qs, k, ks, qo, qos, ko, kos):
        refused(1, K.kvarn_qk_norm_rope, qk(head_dim=64, rot_dim=64), n, q, qs, k, ks, None, None, FAR, FAR, qo, qos, ko, kos)

    q, k, qo, ko = (FAKE + i * (1 << 24) for i in range(4))  # rows of 512 and 128 values
    call(9, q, 512, k, 128, q + 16, 512, ko, 128)            # beside its input, not on it
    call(9, q, 512, k, 128, q, 520, ko, 128)                 # on it with another stride
    call(9, q, 512, k, 128, q + 8 * 512 * b, 512, ko, 128)   # on its last row
    call(1, q, 512, k, 128, q - 511 * b + 14, 512, ko, 128)  # one row, eight values
    call(9, q, 512, k, 128, k, 512, ko, 128)
    call(9, q, 512, k, 128, qo, 512, q + 511 * b - 14, 512)
    call(9, q, 512, k, 128, qo, 512, qo, 512)
    call(9, q, 512, k, 128, qo, 1024, qo + 1016 * b, 1024)   # the end of a row in the next one's beginning
    call(9, q, 512, k, 128, qo, 1024, qo + 504 * b, 1024)
    call(9, q, 4096, k, 4096, qo, 512, q + 512 * b, 2040)    # strides that meet two rows on
    call(1 << 27, q, 512, k, 128, FAR << 1, 512, q + (1 << 20), 128)


def test_streams_that_hold_memory():
    """A Stream object is noted with each tensor of the GPU, an address with none."""
    class Stream:
        cuda_stream = 7

    class Tensor:
        def __init__(self, is_cuda):
            self.is_cuda, self.noted = is_cuda, []

        def record_stream(self, s):
            self.noted.append(s)

    a, b, s = Tensor(True), Tensor(False), Stream()
    K.hold(s, a, None, b)
    K.hold(7, a)
    K.hold(None, a)
    assert a.noted == [s] and b.noted == []


def test_lists_of_different_lengths():
    """The library reads one count a sequence: a shorter list never reaches it."""
    c = cache()
    kv = (FAKE, 256, FAKE, 256)
    for counts in ([5], [5, 5, 5], []):
        for call, args in ((K.kvarn_block_append, (counts, *kv)), (K.kvarn_block_read, (None, counts, FAKE, FAR)),
                           (K.kvarn_block_read, (counts, [0, 0], FAKE, FAR)),
                           (K.kvarn_block_prefill_attention, (counts, FAKE, FAR, 1.0)),
                           (K.kvarn_block_prefill, (counts, *kv, FAKE, FAR, 1.0))):
            with pytest.raises(ValueError):
                call(c, 0, [0, 1], *args)
    assert K.kvarn_block_length(c, 0, 0) == 0
    K.kvarn_block_destroy(c)
