"""GPU tests of attention over prefixes that sequences share (include/kvarn.h, kvarn_block_attend) against the softmax
over prefix and sequence in 64 bits. block_ref.attend's bound holds for the two parts joined: weights are rounded
against their own part's largest, which enters the sum at most with that share, and the join adds a few fp32
roundings of a logarithm no larger than the largest logit's and 2^5, which its 2^-16 covers."""
import pytest
import torch

from tests import block_ref
from tests.test_gpu_block import TYPES, check, fill, make, tokens

pytestmark = pytest.mark.gpu


def want_of(q, at, k, v, pre, own, n, m, block, code, dim, scale=None):
    """o and tol of m queries from row `at` of sequence `own` (n tokens) behind sequence `pre` (None: none)."""
    sides = []
    for x in (k, v):
        parts = [block_ref.hold(x[own], block, code)]
        if pre is not None:
            parts.insert(0, block_ref.hold(x[pre], block, code))
        sides.append(torch.cat(parts))
    before = 0 if pre is None else k[pre].shape[0]
    return block_ref.attend(q[at:at + m].cpu(), sides[0], sides[1], dim ** -0.5 if scale is None else scale,
                            [before + n - m + t for t in range(m)])


SHAPES = [(32, 64, 2, 1), (64, 128, 2, 4), (128, 128, 1, 8), (32, 128, 3, 5), (64, 64, 1, 7), (128, 64, 2, 2), (64, 128, 1, 3)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block,dim,hkv,r", SHAPES)
def test_decode(dtype, code, block, dim, hkv, r):
    """Short prefixes, which each sequence walks by itself: of every kind of length, for one sequence or several, with
    sequences that have none, or no tokens of their own, in between."""
    dt = TYPES[dtype]
    lens = [1, 31, 0, 33, block, 5 * block - 1, 777, 40, 0, 1, 33, block, 300]  # 0 .. 8: own; 9 .. 12: prefixes
    c = make(max_seqs=14, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt)
    k, v = fill(c, lens, dt, 320)
    ids = [7, 8, 0, 3, 1, 6, 2, 5, 4]
    pre = [9, 9, 10, None, 11, 11, 12, 12, 13]  # 13 is empty; 8 and 2 have no tokens of their own
    q = tokens(9, hkv * r, dim, dt, 330, 0.3)
    q[2] *= 4
    out = c.decode_attention(0, ids, q, prefix_ids=pre)
    for row, (s, p) in enumerate(zip(ids, pre)):
        want, tol = want_of(q, row, k, v, None if p == 13 else p, s, lens[s], 1, block, code, dim)
        check(out[row:row + 1], want, tol, (s, p))
    assert torch.equal(out, c.decode_attention(0, ids, q, prefix_ids=pre))
    none = c.decode_attention(0, ids, q, prefix_ids=[-1] * 9)
    assert torch.equal(none, c.decode_attention(0, ids, q))
    assert not c.decode_attention(0, [8], q[:1], prefix_ids=[13]).any()
    assert c.check_device_error() == 0


@pytest.mark.parametrize("dtype,code", [("fp16", "e4m3"), ("bf16", "int8"), ("fp16", "int8"), ("bf16", "e4m3")])
@pytest.mark.parametrize("block,dim,hkv,r,seqs,n", [(32, 64, 2, 1, 120, 3001), (64, 128, 2, 4, 80, 4000), (128, 128, 1, 8, 160, 4096),
                                                    (64, 64, 1, 7, 250, 2500), (64, 128, 8, 4, 39, 2049), (32, 128, 3, 5, 200, 1025)])
def test_decode_walked_once(dtype, code, block, dim, hkv, r, seqs, n):
    """A long prefix of many sequences, walked once as tiles of rows, one walked by its only sequence, and none."""
    dt = TYPES[dtype]
    lens = [(37 * i) % 90 for i in range(seqs)] + [n, 500, 45, 64]  # own; the prefixes; two more sequences
    c = make(max_seqs=seqs + 4, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt,
             max_seq_len=4096, pool_blocks=(sum(lens) // block))
    k, v = fill(c, lens, dt, 340)
    ids = list(range(seqs)) + [seqs + 2, seqs + 3]
    pre = [seqs] * seqs + [seqs + 1, None]
    q = tokens(seqs + 2, hkv * r, dim, dt, 350, 0.3)
    q[1] *= 4
    out = c.decode_attention(0, ids, q, prefix_ids=pre)
    for row in sorted({0, 1, 2, seqs // 2, seqs - 1, seqs, seqs + 1}):
        want, tol = want_of(q, row, k, v, pre[row], ids[row], lens[ids[row]], 1, block, code, dim)
        check(out[row:row + 1], want, tol, row)
    assert torch.equal(out, c.decode_attention(0, ids, q, prefix_ids=pre))
    assert c.check_device_error() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block,dim,hkv,r", SHAPES)
def test_prefill(dtype, code, block, dim, hkv, r):
    dt = TYPES[dtype]
    lens = [1, 45, 128, 129, 300, 60, 260, 1, 129, 400]
    qlens = [1, 45, 0, 129, 37, 2, 200]
    c = make(max_seqs=11, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt)
    k, v = fill(c, lens, dt, 360)
    ids = [4, 0, 2, 6, 1, 3, 5]
    pre = [7, 8, 8, 8, None, 9, 10]  # 10 is empty
    m = [qlens[s] for s in ids]
    q = tokens(sum(m), hkv * r, dim, dt, 370, 0.3)
    out = c.prefill_attention(0, ids, m, q, prefix_ids=pre)
    at = 0
    for s, p in zip(ids, pre):
        want, tol = want_of(q, at, k, v, None if p == 10 else p, s, lens[s], qlens[s], block, code, dim)
        check(out[at:at + qlens[s]], want, tol, (s, p))
        at += qlens[s]
    assert torch.equal(out, c.prefill_attention(0, ids, m, q, prefix_ids=pre))
    assert c.check_device_error() == 0


@pytest.mark.parametrize("lens,qlens,n", [([700, 300], [700, 300], 3000), ([20] * 30, [20] * 30, 1500), ([5, 2000], [3, 2000], 130)])
def test_prefill_long(lens, qlens, n):
    """Many steps and many segments, cut and whole, of the prefix and of the sequences' own tokens."""
    c = make(max_seqs=len(lens) + 1, num_q_heads=32, num_kv_heads=8, block_tokens=64)
    k, v = fill(c, lens + [n], torch.float16, 380)
    ids, p = list(range(len(lens))), len(lens)
    q = tokens(sum(qlens), 32, 128, torch.float16, 381, 0.3)
    out = c.prefill_attention(0, ids, qlens, q, prefix_ids=[p] * len(lens))
    at = 0
    for s, m in enumerate(qlens):
        if s in (0, 1, len(lens) - 1):
            rows = sorted({0, 1, m // 2, m - 1})
            kk, vv = (torch.cat([block_ref.hold(x[p], 64, "e4m3"), block_ref.hold(x[s], 64, "e4m3")]) for x in (k, v))
            want, tol = block_ref.attend(q[[at + t for t in rows]].cpu(), kk, vv, 128 ** -0.5, [n + lens[s] - m + t for t in rows])
            check(out[[at + t for t in rows]], want, tol, s)
        at += m
    assert c.check_device_error() == 0


@pytest.mark.parametrize("scale", [-0.05, 0.0, 0.5])
def test_other_scales(scale):
    c = make(max_seqs=41, block_tokens=32, num_q_heads=8, num_kv_heads=8)
    lens = [33 + i for i in range(40)] + [2000]
    k, v = fill(c, lens, torch.float16, 390)
    q = tokens(80, 8, 128, torch.float16, 391, 0.3)
    one = c.decode_attention(0, list(range(40)), q[:40], scale=scale, prefix_ids=[40] * 40)  # walked once
    few = c.decode_attention(0, [0, 1], q[:2], scale=scale, prefix_ids=[40] * 2)             # by each sequence
    two = c.prefill_attention(0, list(range(40)), [2] * 40, q, scale=scale, prefix_ids=[40] * 40)
    for s in (0, 1, 39):
        want, tol = want_of(q, s, k, v, 40, s, lens[s], 1, 32, "e4m3", 128, scale)
        check(one[s:s + 1], want, tol, s)
        if s < 2:
            check(few[s:s + 1], want, tol, s)
        want, tol = want_of(q, 2 * s, k, v, 40, s, lens[s], 2, 32, "e4m3", 128, scale)
        check(two[2 * s:2 * s + 2], want, tol, s)


@pytest.mark.parametrize("heavy", ["prefix", "own"])
def test_parts_of_very_different_weight(heavy):
    """All the weight on one side, the other's values a thousand times as large: nothing of it is left or comes through."""
    n, own = 2000, 50
    c = make(max_seqs=41, num_q_heads=8, num_kv_heads=8, block_tokens=64, max_seq_len=2048)
    k, v = (tokens(n + 40 * own, 8, 128, torch.float16, s, 0.2) for s in (401, 402))
    q = tokens(40, 8, 128, torch.float16, 403, 0.2)
    q[:, :] = q[:1]
    part = slice(0, n) if heavy == "prefix" else slice(n, None)
    other = slice(n, None) if heavy == "prefix" else slice(0, n)
    k[part] = (q[:1].float() * 3).half() + k[part] * 0.1
    k[other] = (q[:1].float() * -3).half()
    v[other] *= 200
    c.append(0, [40] + list(range(40)), [n] + [own] * 40, k, v)
    out = c.decode_attention(0, list(range(40)), q, prefix_ids=[40] * 40)
    kk, vv = ([x[n + i * own:n + (i + 1) * own] for i in range(40)] + [x[:n]] for x in (k, v))
    for s in (0, 39):
        want, tol = want_of(q, s, kk, vv, 40, s, own, 1, 64, "e4m3", 128)
        check(out[s:s + 1], want, tol, s)


@pytest.mark.parametrize("many", [False, True])
def test_non_finite_values_of_a_prefix(many):
    """An infinity in V of a prefix's exact token: its channel of every sequence behind it, and nothing else."""
    seqs = 40 if many else 2
    c = make(max_seqs=seqs + 2, num_q_heads=8, num_kv_heads=8, block_tokens=64)
    lens = [40] * seqs + [2010, 40]
    k, v = (tokens(sum(lens), 8, 128, torch.float16, s, 0.3) for s in (411, 412))
    at = 40 * seqs + 2000
    v[at, 3, 17] = float("inf")
    c.append(0, list(range(seqs + 2)), lens, k, v)
    q = tokens(2 * seqs + 1, 8, 128, torch.float16, 413, 0.3)
    pre = [seqs] * seqs + [None]
    ids = list(range(seqs)) + [seqs + 1]
    for out in (c.decode_attention(0, ids, q[:seqs + 1], prefix_ids=pre),
                c.prefill_attention(0, ids, [2] * seqs + [1], q, prefix_ids=pre)):
        bad = ~torch.isfinite(out)
        want = torch.zeros_like(bad)
        want[:-1, 3, 17] = True
        assert torch.equal(bad, want)


def test_every_logit_minus_infinity():
    c = make(max_seqs=41, num_q_heads=8, num_kv_heads=8, block_tokens=64)
    q = torch.ones(80, 8, 128, dtype=torch.float16, device="cuda")
    k, v = (tokens(40 * 5 + 2010, 8, 128, torch.float16, s, 0.3) for s in (421, 422))
    k[:, 2] = float("-inf")
    # exact tokens keep their infinities
    c.append(0, list(range(40)), [5] * 40, k[:200], v[:200])
    c.append(0, [40], [40], k[200:240], v[200:240])
    for out in (c.decode_attention(0, list(range(40)), q[:40], prefix_ids=[40] * 40),
                c.prefill_attention(0, list(range(40)), [2] * 40, q, prefix_ids=[40] * 40)):
        assert not out[:, 2].any() and torch.isfinite(out).all() and out[:, 3].any()


def test_steps_equal_their_parts():
    a, b = make(block_tokens=32, max_seqs=5), make(block_tokens=32, max_seqs=5)
    k, v = (tokens(400, 2, 128, torch.float16, s) for s in (430, 431))
    q = tokens(400, 8, 128, torch.float16, 432)
    for c in (a, b):
        c.append(0, [4], [200], k[:200], v[:200])
    got = a.prefill(0, [0, 1], [60, 95], k[200:355], v[200:355], q[200:355], prefix_ids=[4, 4])
    b.append(0, [0, 1], [60, 95], k[200:355], v[200:355])
    assert torch.equal(got, b.prefill_attention(0, [0, 1], [60, 95], q[200:355], prefix_ids=[4, 4]))
    for t in range(355, 395, 2):
        got = a.decode_step(0, [1, 0], k[t:t + 2], v[t:t + 2], q[t:t + 2], prefix_ids=[4, None])
        b.append(0, [1, 0], [1, 1], k[t:t + 2], v[t:t + 2])
        assert torch.equal(got, b.decode_attention(0, [1, 0], q[t:t + 2], prefix_ids=[4, None]))
    assert [a.length(0, s) for s in range(5)] == [80, 115, 0, 0, 200]


def test_output_over_the_queries_and_layers():
    """out = q, and a prefix of another layer that has other tokens."""
    c = make(max_seqs=41, num_layers=2, num_q_heads=32, num_kv_heads=8, block_tokens=64, max_seq_len=2048)
    sides = []
    for layer in (0, 1):
        k, v = (tokens(40 * 30 + 2000, 8, 128, torch.float16, 440 + 2 * layer + s) for s in (0, 1))
        c.append(layer, list(range(41)), [30] * 40 + [2000 - layer], k[:3200 - layer], v[:3200 - layer])
        sides.append([[x[30 * i:30 * i + 30] for i in range(40)] + [x[1200:3200 - layer]] for x in (k, v)])
    for layer in (0, 1):
        q = tokens(80, 32, 128, torch.float16, 446 + layer, 0.3)
        for qlens in (None, [2] * 40):
            x = q[:40].clone() if qlens is None else q.clone()
            call = (lambda y, out: c.decode_attention(layer, list(range(40)), y, out=out, prefix_ids=[40] * 40)) if qlens is None else (
                lambda y, out: c.prefill_attention(layer, list(range(40)), qlens, y, out=out, prefix_ids=[40] * 40))
            want = call(x, None)
            assert call(x, x) is x and torch.equal(x, want)
            m = 1 if qlens is None else 2
            ref, tol = want_of(q, 5 * m, *sides[layer], 40, 5, 30, m, 64, "e4m3", 128)
            check(want[5 * m:5 * m + m], ref, tol, (layer, m))


def test_captured_and_replayed():
    c = make(max_seqs=41, num_q_heads=32, num_kv_heads=8, block_tokens=32, max_seq_len=3000)
    fill(c, [33] * 40 + [2100], torch.float16, 450)
    ids, pre = list(range(40)), [40] * 40
    qs = [tokens(80, 32, 128, torch.float16, s, 0.3) for s in (452, 453)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = [(c.decode_attention(0, ids, q[:40], prefix_ids=pre), c.prefill_attention(0, ids, [2] * 40, q, prefix_ids=pre))
                for q in qs]
        static = qs[0].clone()
        graphs = []
        for call in (lambda: c.decode_attention(0, ids, static[:40], prefix_ids=pre),
                     lambda: c.prefill_attention(0, ids, [2] * 40, static, prefix_ids=pre)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = call()
            graphs.append((g, out))
        for q, w in list(zip(qs, want)) * 2:
            static.copy_(q)
            for (g, out), x in zip(graphs, w):
                g.replay()
                assert torch.equal(out, x)
    s.synchronize()
    a = c.decode_attention(0, ids, qs[0][:40], prefix_ids=pre, stream=s)
    s.synchronize()
    assert torch.equal(a, want[0][0])


def test_nothing_around_the_workspace_is_written():
    from quantized_kv_cache_seal_gb300 import kvarn as K
    c = make(max_seqs=41, num_q_heads=24, num_kv_heads=8, block_tokens=32, max_seq_len=3000)
    fill(c, [33] * 40 + [2100], torch.float16, 460)
    w = c.new_weights()[0]
    q = tokens(120, 24, 128, torch.float16, 462, 0.3)
    ids, stream = list(range(40)), torch.cuda.current_stream().cuda_stream
    for qlens, pre, weights in ((None, [40] * 40, w), ([3] * 40, [40] * 40, None), (None, None, w)):
        n = K.kvarn_block_attend_workspace(c.handle, 0, ids, pre, qlens, False, weights is not None)
        assert n > 0 and n % 256 == 0
        space = torch.full((n + 1024,), 0xa5, dtype=torch.uint8, device="cuda")
        base = (space.data_ptr() + 255) // 256 * 256 + 256
        rows = 40 if qlens is None else 120
        out = torch.full((rows + 2, 24, 128), 7.0, dtype=torch.float16, device="cuda")
        K.kvarn_block_attend(c.handle, 0, ids, pre, qlens, q, out[1:], 0.1, weights, base, n, stream)
        at = base - space.data_ptr()
        assert bool((space[:at] == 0xa5).all()) and bool((space[at + n:] == 0xa5).all())
        assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all()) and not bool((out[1:-1] == 7).all())


def test_after_a_wait_has_given_up():
    """With the timeout bit set, as by a wait of a launch before, calls end at once and say so; then all is right again."""
    from tests.test_gpu_block_edges import _words
    c = make(max_seqs=41, num_q_heads=32, num_kv_heads=8, block_tokens=32, max_seq_len=3000)
    fill(c, [33] * 40 + [2100], torch.float16, 470)
    q = tokens(80, 32, 128, torch.float16, 472, 0.3)
    ids, pre = list(range(40)), [40] * 40
    calls = (lambda: c.decode_attention(0, ids, q[:40], prefix_ids=pre),
             lambda: c.prefill_attention(0, ids, [2] * 40, q, prefix_ids=pre))
    want = [f() for f in calls]
    for _ in range(5):
        _words(c, 0, 1).fill_(1)
        for f in calls:
            f()
        assert c.check_device_error() == 6
        assert all(torch.equal(f(), w) for f, w in zip(calls, want))
        assert c.check_device_error() == 0


@pytest.mark.parametrize("dtype,code,dim,block", [("fp16", "e4m3", 128, 64), ("bf16", "int8", 64, 32)])
@pytest.mark.parametrize("hkv,r", [(8, 4), (10, 1), (7, 5), (8, 8)])
def test_many_short_sequences(dtype, code, dim, block, hkv, r):
    """Short pairs whose line is cut over warps: with a long prefix, walked once, and with weights."""
    from tests.test_gpu_block_evict import near, received, some_weights
    dt, seqs, n = TYPES[dtype], 200, 1500
    lens = [(131 * i) % 700 for i in range(seqs)] + [n]
    c = make(max_seqs=seqs + 1, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt,
             max_seq_len=1600, pool_blocks=sum(x // block for x in lens))
    k, v = fill(c, lens, dt, 480)
    q = tokens(seqs, hkv * r, dim, dt, 482, 0.3)
    ids = list(range(seqs))
    for pre in ([seqs] * seqs, None):
        w = some_weights(c, 483)
        before = w.clone()
        out = c.decode_attention(0, ids, q, prefix_ids=pre, weights=w)
        again = before.clone()
        assert torch.equal(out, c.decode_attention(0, ids, q, prefix_ids=pre, weights=again)) and torch.equal(w, again)
        for s in (0, 1, 2, 77, seqs - 1):  # 0 has no tokens of its own
            if pre is None and s == 0:
                assert not out[s].any()
                continue
            want, tol = want_of(q, s, k, v, None if pre is None else seqs, s, lens[s], 1, block, code, dim)
            check(out[s:s + 1], want, tol, s)
            first = 0 if pre is None else n
            parts = ([block_ref.hold(k[seqs], block, code)] if pre else []) + [block_ref.hold(k[s], block, code)]
            want, tol = received(q[s:s + 1], torch.cat(parts), dim ** -0.5, [first + lens[s] - 1], block, first)
            near(w[s], before[s], want, tol, s)
    assert c.check_device_error() == 0


def test_streams_that_hold_a_workspace_that_grows(monkeypatch):
    """A stream given by its address holds nothing, also where a call lets the workspace grow; the next Stream object that
    a call names holds the cache's memory and every workspace."""
    held = []
    record = torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda x, s: (held.append(x.data_ptr()), record(x, s))[1])
    hq, hkv, dim, m = 32, 8, 128, 200
    c = make(max_seqs=2, num_q_heads=hq, num_kv_heads=hkv)
    k, v = fill(c, [m, 65], torch.float16, 900)
    q = tokens(m, hq, dim, torch.float16, 910, 0.3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    del held[:]
    out = c.prefill_attention(0, [0], [m], q, stream=s.cuda_stream, prefix_ids=[1])
    assert len(c._spaces) == 2 and not held
    s.synchronize()
    again = c.prefill_attention(0, [0], [m], q, stream=s, prefix_ids=[1])
    assert {c.mem.data_ptr(), *(x.data_ptr() for x in c._spaces)} <= set(held)
    s.synchronize()
    assert torch.equal(out, again)
    for t in (0, 64, m - 1):
        want, tol = want_of(q, 0, k, v, 1, 0, m, m, 64, "e4m3", dim)
        check(out[t:t + 1], want[t:t + 1], tol[t:t + 1], t)
    assert c.check_device_error() == 0


@pytest.mark.parametrize("dtype,code", [("fp16", "e4m3"), ("bf16", "int8")])
@pytest.mark.parametrize("block,dim,hkv,r,seqs,n", [(64, 128, 4, 4, 60, 4001), (32, 64, 2, 1, 90, 4090), (64, 128, 8, 4, 150, 700),
                                                    (128, 128, 8, 7, 120, 1024), (64, 64, 5, 8, 130, 1300)])
def test_prefill_walked_once(dtype, code, block, dim, hkv, r, seqs, n):
    """Many sequences of few queries, whose rows stand together over the prefix: of tiles by themselves, and of so many that they
    go in pairs; with a second prefix and sequences without one."""
    dt = TYPES[dtype]
    lens = [9 + (37 * i) % 90 for i in range(seqs)] + [n, 333, 45]
    qlens = [2 + i % 7 for i in range(seqs)] + [1]
    c = make(max_seqs=seqs + 3, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt,
             max_seq_len=4096, pool_blocks=(sum(lens) // block))
    k, v = fill(c, lens, dt, 920)
    ids = list(range(seqs)) + [seqs + 2]
    pre = [seqs] * (seqs - 2) + [seqs + 1] * 2 + [None]
    q = tokens(sum(qlens), hkv * r, dim, dt, 930, 0.3)
    out = c.prefill_attention(0, ids, qlens, q, prefix_ids=pre)
    at = [sum(qlens[:i]) for i in range(len(ids))]
    for i in (0, 1, seqs // 2, seqs - 3, seqs - 2, seqs - 1, seqs):
        want, tol = want_of(q, at[i], k, v, pre[i], ids[i], lens[ids[i]], qlens[i], block, code, dim)
        check(out[at[i]:at[i] + qlens[i]], want, tol, i)
    assert torch.equal(out, c.prefill_attention(0, ids, qlens, q, prefix_ids=pre))
    assert c.check_device_error() == 0


@pytest.mark.parametrize("dtype,code", [("fp16", "e4m3"), ("bf16", "int8"), ("fp16", "int8"), ("bf16", "e4m3")])
@pytest.mark.parametrize("block,dim,hkv,r,n", [(64, 128, 2, 4, 3001), (128, 128, 1, 8, 1024), (32, 64, 3, 5, 515), (64, 64, 40, 1, 129),
                                               (64, 128, 40, 2, 127), (128, 128, 2, 3, 1)])
def test_prefill_with_the_prefix_in_front(dtype, code, block, dim, hkv, r, n):
    """Prefixes in front of the sequences' own tokens, steps of both cut over thread blocks and segments taken whole, beside
    sequences without one, for prompts whose last tokens only ask as well."""
    dt = TYPES[dtype]
    lens = [150, 61, 200, 33, 300, n, 95]
    qlens = [150, 45, 7, 33, 129]
    pre = [5, 5, None, 6, 5]
    c = make(max_seqs=7, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt)
    k, v = fill(c, lens, dt, 940)
    q = tokens(sum(qlens), hkv * r, dim, dt, 950, 0.3)
    out = c.prefill_attention(0, range(5), qlens, q, prefix_ids=pre)
    at = 0
    for s in range(5):
        rows = sorted({0, 1, qlens[s] // 2, qlens[s] - 2, qlens[s] - 1})
        want, tol = want_of(q, at, k, v, pre[s], s, lens[s], qlens[s], block, code, dim)
        check(out[at:at + qlens[s]][rows], want[rows], tol[rows], s)
        at += qlens[s]
    assert torch.equal(out, c.prefill_attention(0, range(5), qlens, q, prefix_ids=pre))
    assert c.check_device_error() == 0


@pytest.mark.parametrize("hkv", [2, 80])
def test_non_finite_values_on_both_sides(hkv):
    """Infinities in V of the prefix's last exact token, of an own token that only later queries see, and of another sequence's:
    each in its channel of the rows that see it. Few segments, cut over thread blocks, and many, taken whole."""
    c = make(max_seqs=3, num_q_heads=hkv, num_kv_heads=hkv, block_tokens=64)
    lens = [150, 40, 700]  # two sequences, their prefix
    k, v = (tokens(sum(lens), hkv, 128, torch.float16, s, 0.3) for s in (961, 962))
    v[140, 1, 5] = float("inf")   # own position 140
    v[155, 0, 9] = float("-inf")  # the other's own position 5
    v[-1, 1, 77] = float("inf")
    c.append(0, [0, 1, 2], lens, k, v)
    q = tokens(160, hkv, 128, torch.float16, 963, 0.3)
    out = c.prefill_attention(0, [0, 1], [150, 10], q, prefix_ids=[2, 2])
    want = torch.zeros_like(out, dtype=torch.bool)
    want[:, 1, 77] = True
    want[140:150, 1, 5] = True
    want[150:, 0, 9] = True
    assert torch.equal(~torch.isfinite(out), want)
    assert c.check_device_error() == 0


@pytest.mark.parametrize("first", ["nothing", "copy", "other stream", "both"])
def test_captured_behind_other_work(first):
    """A graph whose first kernel is an attention call's, or that has a copy, another stream's work or both right before it."""
    c = make(max_seqs=10, num_q_heads=8, num_kv_heads=2)
    fill(c, [40 + 30 * i for i in range(9)] + [700], torch.float16, 970)
    ids, pre = list(range(9)), [9] * 4 + [None] + [9] * 4
    given = tokens(45, 8, 128, torch.float16, 980, 0.3)
    q, w, more = torch.empty_like(given), c.new_weights()[0], torch.zeros(1 << 22, device="cuda")

    def calls():
        return (c.decode_attention(0, ids, q[:9], prefix_ids=pre, weights=w), c.prefill_attention(0, ids, [5] * 9, q, prefix_ids=pre))

    q.copy_(given)
    want = [x.clone() for x in calls()] + [w.clone()]
    torch.cuda.synchronize()
    s, t, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        if first in ("other stream", "both"):
            t.wait_stream(s)
            with torch.cuda.stream(t):
                for _ in range(4):
                    more.add_(1)
                q.copy_(given)
            if first == "both":
                w.zero_()
            s.wait_stream(t)
        elif first == "copy":
            q.copy_(given)
        got = calls()
    for _ in range(3):
        w.zero_()
        if first != "nothing":
            q.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, w), want))
    assert c.check_device_error() == 0
