"""GPU tests of the weights that blocks receive and of eviction by them (include/kvarn.h) against 64 bits."""
import random

import pytest
import torch

from tests import block_ref
from tests.test_gpu_block import TYPES, as_type, check, fill, make, same, tokens

pytestmark = pytest.mark.gpu


def received(q, k, scale, last, block, first=0):
    """What the blocks of k[first:] receive of q's softmax weights, [hkv][blocks] in 64 bits, and a bound on an fp32
    kernel's error. q [rows][hq][dim] in the inputs' type, row i sees positions <= last[i]; k [n][hkv][dim] in 64 bits.

    The bound: logits are off by (dim + 8) roundings of 2^-24 of sum |q k| scale, and by as many of the size of
    log2 of V's scale, under 2^5 here, that decode adds to and takes off them (8 * 2^5 * 2^-24 = 2^-16 of a weight); numerator and
    denominator each change a weight by that share. Exponentials, sums over at most 2^12 tokens (32 at a time, then in turn),
    the division and the sum over rows: under 2^7 + 2^6 roundings of 2^-24, 2^-16. Weights under 2^-100 may be lost."""
    q = block_ref.f64(q)
    rows, hq, dim = q.shape
    n, hkv, _ = k.shape
    r = hq // hkv
    got, tol = (torch.zeros(hkv, -(-(n - first) // block), dtype=torch.float64) for _ in (0, 1))
    seen = torch.arange(n)[None] <= torch.as_tensor(last)[:, None]
    for h in range(hq):
        s = (q[:, h] @ k[:, h // r].T) * scale
        s = torch.where(seen, s, torch.tensor(float("-inf"), dtype=torch.float64))
        p = torch.softmax(s, -1)
        off = (q[:, h].abs() @ k[:, h // r].abs().T) * abs(scale) * (dim + 8) * 2.0 ** -24
        off = torch.where(seen, off, torch.zeros_like(off)).amax(-1, keepdim=True)
        for x, to in ((p, got), (p * (2 * off + 2.0 ** -15), tol)):
            x = x[:, first:].sum(0)
            to[h // r] += torch.cat([x, torch.zeros(-len(x) % block, dtype=torch.float64)]).view(-1, block).sum(-1)
    return got, tol + 2.0 ** -100


def near(w, before, want, tol, what):
    """w = before + want but for tol and the sum's rounding; places behind the blocks stay as they were."""
    w, before = w.cpu().double(), before.cpu().double()
    n = want.shape[1]
    total = before[:, :n] + want
    far = ((w[:, :n] - total).abs() / (tol + total.abs() * 2.0 ** -23)).max() if n else 0
    assert far <= 1, (what, float(far))
    assert torch.equal(w[:, n:], before[:, n:]), what


def some_weights(c, seed):
    return torch.rand(c.weights_shape, generator=torch.Generator().manual_seed(seed)).cuda()


SHAPES = [(32, 64, 2, 1), (64, 128, 2, 4), (128, 128, 1, 8), (32, 128, 3, 5), (64, 64, 1, 7), (128, 64, 2, 2), (64, 128, 1, 3)]


# ------------------------------------------------------------------------------------------------ weights of decode
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block,dim,hkv,r", SHAPES)
def test_decode_weights(dtype, code, block, dim, hkv, r):
    dt = TYPES[dtype]
    lens = [1, 31, 32, 33, block, block + 1, 5 * block - 1, 1777]
    c = make(max_seqs=10, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt)
    k, _ = fill(c, lens, dt, 520)
    ids = [7, 8, 0, 3, 1, 6, 2, 5, 4]  # 8 is empty
    q = tokens(9, hkv * r, dim, dt, 530, 0.3)
    q[2] *= 4
    w = some_weights(c, 531)
    before = w.clone()
    out = c.decode_attention(0, ids, q, weights=w)
    assert torch.equal(out, c.decode_attention(0, ids, q))
    for row, s in enumerate(ids):
        if s == 8:
            continue
        want, tol = received(q[row:row + 1], block_ref.hold(k[s], block, code), dim ** -0.5, [lens[s] - 1], block)
        near(w[s], before[s], want, tol, s)
    assert torch.equal(w[8:], before[8:])
    again = before.clone()
    c.decode_attention(0, ids, q, weights=again)
    assert torch.equal(w, again)
    assert c.check_device_error() == 0


@pytest.mark.parametrize("lens", [[4000], [3000, 40, 2000], [700] * 40])
def test_decode_weights_split(lens):
    c = make(max_seqs=len(lens), num_q_heads=8, num_kv_heads=2, block_tokens=32, pool_blocks=sum(n // 32 for n in lens))
    k, _ = fill(c, lens, torch.float16, 540)
    q = tokens(len(lens), 8, 128, torch.float16, 541, 0.3)
    w = some_weights(c, 542)
    before = w.clone()
    c.decode_attention(0, list(range(len(lens))), q, weights=w)
    for s in sorted({0, 1, 2, len(lens) - 1} & set(range(len(lens)))):
        want, tol = received(q[s:s + 1], block_ref.hold(k[s], 32, "e4m3"), 128 ** -0.5, [lens[s] - 1], 32)
        near(w[s], before[s], want, tol, s)


@pytest.mark.parametrize("seqs,n", [(3, 300), (40, 2000)])
def test_decode_weights_behind_a_prefix(seqs, n):
    """Shares of the softmax over prefix and sequence; of the prefix itself nothing is noted."""
    c = make(max_seqs=seqs + 2, num_q_heads=32, num_kv_heads=8, block_tokens=32)
    lens = [(37 * i) % 200 for i in range(seqs)] + [n, 99]
    k, _ = fill(c, lens, torch.float16, 550)
    q = tokens(seqs + 1, 32, 128, torch.float16, 551, 0.3)
    w = some_weights(c, 552)
    before = w.clone()
    ids, pre = list(range(seqs)) + [seqs + 1], [seqs] * seqs + [None]
    out = c.decode_attention(0, ids, q, prefix_ids=pre, weights=w)
    assert torch.equal(out, c.decode_attention(0, ids, q, prefix_ids=pre))
    for row in sorted({0, 1, 2, seqs - 1, seqs}):
        s, parts = ids[row], [block_ref.hold(k[ids[row]], 32, "e4m3")]
        if pre[row] is not None:
            parts.insert(0, block_ref.hold(k[pre[row]], 32, "e4m3"))
        first = 0 if pre[row] is None else n
        want, tol = received(q[row:row + 1], torch.cat(parts), 128 ** -0.5, [first + lens[s] - 1], 32, first)
        near(w[s], before[s], want, tol, s)
    assert torch.equal(w[seqs], before[seqs])


def test_rows_that_add_nothing():
    """NaN and infinite logits: their rows' heads add nothing, the other KV heads theirs."""
    c = make(max_seqs=2, block_tokens=32)
    k, v = (tokens(210, 2, 128, torch.float16, s, 0.3) for s in (560, 561))
    k[207, 0, 3] = float("nan")   # exact, head 0 of sequence 0
    k[105, 0, 3] = float("-inf")  # exact, of sequence 1
    c.append(0, [1, 0], [110, 100], k, v)
    q = tokens(2, 8, 128, torch.float16, 562, 0.3).abs()
    w = torch.zeros(c.weights_shape, device="cuda")
    c.decode_attention(0, [1, 0], q, weights=w)
    for call in (lambda: None, lambda: c.window_weights(0, [1, 0], [1, 1], q, w)):
        call()
        assert torch.isfinite(w).all()
        assert not w[0, 0].any()
        for s, h in ((0, 1), (1, 0), (1, 1)):  # a key of -inf has no weight, the row its others
            assert abs(float(w[s, h].sum()) / 4 - round(float(w[s, h].sum()) / 4)) < 2.0 ** -15 and w[s, h].any()


# ------------------------------------------------------------------------------------------------ window
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block,dim,hkv,r", SHAPES)
def test_window(dtype, code, block, dim, hkv, r):
    dt = TYPES[dtype]
    lens = [1, 31, 32, 60, block, 129, 5 * block - 1, 1777]
    qlens = [1, 31, 1, 60, 5, 128, 0, 70]
    c = make(max_seqs=9, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt)
    k, _ = fill(c, lens, dt, 570)
    ids = [7, 0, 3, 1, 6, 2, 5, 4]
    m = [qlens[s] for s in ids]
    q = tokens(sum(m), hkv * r, dim, dt, 580, 0.3)
    w = some_weights(c, 581)
    before = w.clone()
    c.window_weights(0, ids, m, q, w)
    at = 0
    for s in ids:
        n = qlens[s]
        if n:
            want, tol = received(q[at:at + n], block_ref.hold(k[s], block, code), dim ** -0.5,
                                 list(range(lens[s] - n, lens[s])), block)
            near(w[s], before[s], want, tol, s)
        else:
            assert torch.equal(w[s], before[s])
        at += n
    assert torch.equal(w[8], before[8])
    again = before.clone()
    c.window_weights(0, ids, m, q, again)
    assert torch.equal(w, again)
    assert c.check_device_error() == 0


@pytest.mark.parametrize("scale", [-0.05, 0.0, 0.5])
def test_window_and_decode_agree(scale):
    """One query of a sequence either way, at other scales, against the definition."""
    c = make(max_seqs=3, block_tokens=64, num_q_heads=10, num_kv_heads=2, dtype=torch.bfloat16)
    lens = [200, 63, 1]
    k, _ = fill(c, lens, torch.bfloat16, 590)
    q = tokens(3, 10, 128, torch.bfloat16, 591, 0.3)
    a, b = (torch.zeros(c.weights_shape, device="cuda") for _ in (0, 1))
    c.decode_attention(0, [0, 1, 2], q, scale=scale, weights=a)
    c.window_weights(0, [0, 1, 2], [1, 1, 1], q, b, scale=scale)
    for s in range(3):
        want, tol = received(q[s:s + 1], block_ref.hold(k[s], 64, "e4m3"), scale, [lens[s] - 1], 64)
        for w in (a, b):
            near(w[s], torch.zeros_like(w[s]), want, tol, s)


def test_window_leaves_the_rest_of_its_workspace():
    from quantized_kv_cache_seal_gb300 import kvarn as K
    c = make(max_seqs=2, num_q_heads=10, num_kv_heads=2, block_tokens=32)
    fill(c, [300, 33], torch.float16, 600)
    q = tokens(10, 10, 128, torch.float16, 601, 0.3)
    w = torch.zeros(c.weights_shape, device="cuda")
    n = K.kvarn_block_window_workspace(c.handle, 0, [0, 1], [7, 3])
    assert n > 0
    space = torch.full((n + 1024,), 0xa5, dtype=torch.uint8, device="cuda")
    base = (space.data_ptr() + 255) // 256 * 256 + 256
    K.kvarn_block_window_weights(c.handle, 0, [0, 1], [7, 3], q, 0.1, w, base, n, torch.cuda.current_stream().cuda_stream)
    at = base - space.data_ptr()
    assert bool((space[:at] == 0xa5).all()) and bool((space[at + n:] == 0xa5).all())
    assert w[0].any() and w[1].any()


# ------------------------------------------------------------------------------------------------ eviction
def cut(full, keep, first, last, w):
    """Blocks that stay, by the rule, of one KV head with weights w."""
    if full <= keep:
        return list(range(full))
    always = set(range(first)) | set(range(full - last, full))
    value = [float("-inf") if x != x else x for x in w]  # NaN stands below all: behind -inf
    rest = sorted((i for i in range(full) if i not in always), key=lambda i: (-value[i], w[i] != w[i], i))
    return sorted(list(always) + rest[:keep - len(always)])


def evicted(c, ids, lens, k, v, w, keep, first, last, block, code, layer=0):
    """Evicts and checks all that a user sees of it: numbers, weights, values, lengths."""
    before = w.clone()
    kept = c.evict(layer, ids, w, keep, first=first, last=last)
    hkv = before.shape[1]
    assert kept.shape == (len(ids), hkv, keep) and kept.dtype is torch.int32
    now = [min(lens[s], keep * block + lens[s] % block) for s in ids]
    assert [c.length(layer, s) for s in ids] == now
    got = [x.cpu() for x in c.read(layer, ids, None, now, dtype=torch.float32)]
    at = 0
    for row, s in enumerate(ids):
        full, tail = lens[s] // block, lens[s] % block
        whole = [block_ref.hold(x[s], block, code) for x in (k, v)]
        for h in range(hkv):
            old = before[s, h].cpu().tolist()
            blocks = cut(full, keep, first, last, old)
            assert kept[row, h].tolist() == blocks + [-1] * (keep - len(blocks)), (s, h)
            new = list(old)
            if full > keep:
                new = [old[b] for b in blocks] + [old[full]] + [0.0] * (full - keep) + old[full + 1:]
            assert same(w[s, h], torch.tensor(new)), (s, h)
            pick = [b * block + t for b in blocks for t in range(block)] + list(range(full * block, full * block + tail))
            for x, g in zip(whole, got):
                assert same(g[at:at + now[row], h], x[pick, h].float()), (s, h)
        at += now[row]
    others = [s for s in range(before.shape[0]) if s not in ids]
    assert same(w[others], before[others])
    return kept


@pytest.mark.parametrize("dtype,code", [("fp16", "e4m3"), ("bf16", "int8"), ("fp16", "int8")])
@pytest.mark.parametrize("block,dim,hkv", [(32, 64, 2), (64, 128, 3), (128, 128, 1), (32, 128, 5), (128, 64, 2)])
@pytest.mark.parametrize("keep,first,last", [(3, 1, 1), (5, 0, 0), (4, 2, 2), (1, 0, 1), (9, 1, 3)])
def test_evict(dtype, code, block, dim, hkv, keep, first, last):
    dt = TYPES[dtype]
    lens = [10 * block + 7, 5 * block, 0, 3 * block - 1, 17 * block + 31, 4 * block + 1, 20]
    c = make(max_seqs=8, num_q_heads=hkv, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt)
    k, v = fill(c, lens, dt, 610)
    w = some_weights(c, 611)
    evicted(c, [4, 0, 2, 3, 1, 6], lens, k, v, w, keep, first, last, block, code)
    assert same(c.read(0, [5], None, [lens[5]], dtype=torch.float32)[0], block_ref.hold(k[5], block, code).float())
    assert c.check_device_error() == 0


@pytest.mark.parametrize("kind", ["equal", "two values", "zeros", "signs", "nan", "infinite", "tiny"])
def test_evict_by_hard_weights(kind):
    block, n = 32, 40 * 32 + 5
    c = make(max_seqs=1, num_q_heads=4, num_kv_heads=4, block_tokens=block)
    k, v = fill(c, [n], torch.float16, 620)
    w = some_weights(c, 621)
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "two values":
        w = (w > 0.5).float()
    elif kind == "zeros":
        w = torch.where(w > 0.5, -0.0, 0.0)
    elif kind == "signs":
        w = (w - 0.5) * 1e3
    elif kind == "nan":
        w = torch.where(w > 0.6, float("nan"), w - 0.3)
        w[0, 1, ::2] = float("-inf")
        w[0, 2] = float("nan")
    elif kind == "infinite":
        w = torch.where(w > 0.6, float("inf"), torch.where(w < 0.3, float("-inf"), w))
    else:
        w = w * 2.0 ** -149 * 5
    evicted(c, [0], [n], k, v, w.contiguous(), 11, 1, 2, block, "e4m3")


@pytest.mark.parametrize("blocks,keep", [(1030, 1025), (1500, 400), (2100, 2000), (1024, 1023)])
def test_evict_of_many_blocks(blocks, keep):
    """More blocks than the selection takes at a time."""
    n = 32 * blocks + 3
    c = make(max_seqs=1, num_q_heads=2, num_kv_heads=2, head_dim=64, block_tokens=32, max_seq_len=n)
    k, v = fill(c, [n], torch.float16, 630)
    w = torch.round(some_weights(c, 631) * 300) / 300  # with ties
    evicted(c, [0], [n], k, v, w, keep, 3, 7, 32, "e4m3")


def test_pool_and_later_appends():
    """Freed blocks are used again, the sequences go on, in two layers of their own."""
    block, n = 32, 20 * 32 + 9
    c = make(num_layers=2, max_seqs=2, block_tokens=block, pool_blocks=40 + 5, max_seq_len=n + 400)
    sides = [fill(c, [n], torch.float16, 640 + 10 * layer, layer) if layer else fill(c, [n], torch.float16, 640) for layer in (0, 1)]
    w = [some_weights(c, 660), some_weights(c, 661)]
    more = [tokens(300, 2, 128, torch.float16, s) for s in (662, 663)]
    from quantized_kv_cache_seal_gb300.kvarn import KVarNError
    with pytest.raises(KVarNError):
        c.append(0, [1], [300], *more)  # 9 blocks, 5 free
    kept = evicted(c, [0], [n], *sides[0], w[0], 6, 1, 1, block, "e4m3", 0)
    assert same(c.read(1, [0], None, [n], dtype=torch.float32)[0], block_ref.hold(sides[1][0][0], block, "e4m3").float())
    c.append(0, [1], [300], *more)
    now = c.length(0, 0)
    c.append(0, [0], [100], more[0][:100], more[1][:100])
    got = c.read(0, [0], None, [now + 100], dtype=torch.float32)
    for x, y, g in zip(sides[0], more, got):
        held = block_ref.hold(x[0], block, "e4m3")
        for h in range(2):
            pick = [b * block + t for b in kept[0, h].tolist() for t in range(block)]
            tail = block_ref.hold(torch.cat([x[0][n // block * block:].cpu(), y[:100].cpu()]), block, "e4m3")
            assert same(g[:, h], torch.cat([held[pick, h], tail[:, h]]).float())
    assert same(c.read(0, [1], None, [300], dtype=torch.float32)[1], block_ref.hold(more[1], block, "e4m3").float())
    evicted(c, [0], [n], *sides[1], w[1], 0, 0, 0, block, "e4m3", 1)
    assert c.length(1, 0) == 9


def test_chain_as_a_server_uses_it():
    """Prompts behind a shared one, what their ends need, cut to a budget, steps that note weights, cut again: outputs against
    64 bits over what the numbers say is left."""
    block, n, hq, hkv = 32, 700, 8, 2
    c = make(max_seqs=4, num_q_heads=hq, num_kv_heads=hkv, block_tokens=block, code="int8")
    w = c.new_weights()[0]
    k, v = (tokens(200 + 3 * n, hkv, 128, torch.float16, s, 0.5) for s in (670, 671))
    q = tokens(3 * n, hq, 128, torch.float16, 672, 0.3)
    c.append(0, [3], [200], k[:200], v[:200])
    own = [[x[200 + i * n:200 + (i + 1) * n] for i in range(3)] for x in (k, v)]
    prompt = n - 60
    rows = torch.cat([torch.arange(i * n, i * n + prompt) for i in range(3)]).cuda()
    c.prefill(0, [0, 1, 2], [prompt] * 3, k[200:][rows], v[200:][rows], q[rows].contiguous(), prefix_ids=[3] * 3)
    ends = torch.cat([torch.arange(i * n + prompt - 16, i * n + prompt) for i in range(3)]).cuda()
    c.window_weights(0, [0, 1, 2], [16] * 3, q[ends].contiguous(), w)
    # of each sequence and head: positions held
    held = [[list(range(prompt)) for _ in range(hkv)] for _ in range(3)]

    def cut_to(keep):
        kept = c.evict(0, [0, 1, 2], w, keep, first=1, last=2).tolist()
        for s in range(3):
            for h in range(hkv):
                old = held[s][h]
                full = len(old) // block
                blocks = [b for b in kept[s][h] if b >= 0]
                assert len(blocks) == min(keep, full)
                held[s][h] = [p for b in blocks for p in old[b * block:(b + 1) * block]] + old[full * block:]

    cut_to(8)
    pre = [block_ref.hold(x[:200], block, "int8") for x in (k, v)]
    for t in range(prompt, n):
        at = [i * n + t for i in range(3)]
        before = w.clone()
        out = c.decode_step(0, [0, 1, 2], k[200:][at], v[200:][at], q[at].contiguous(), prefix_ids=[3] * 3, weights=w)
        for s in range(3):
            for h in range(hkv):
                held[s][h].append(t)
        if t % 13 == 0 or t == n - 1:
            for s in range(3):
                whole = [block_ref.hold(x[s][:t + 1], block, "int8") for x in own]
                sides = [torch.cat([p, torch.stack([x[held[s][h], h] for h in range(hkv)], 1)]) for p, x in zip(pre, whole)]
                m = sides[0].shape[0]
                want, tol = block_ref.attend(q[at[s]:at[s] + 1].cpu(), *sides, 128 ** -0.5, [m - 1])
                check(out[s:s + 1], want, tol, (t, s))
                share, off = received(q[at[s]:at[s] + 1], sides[0], 128 ** -0.5, [m - 1], block, 200)
                near(w[s], before[s], share, off, (t, s))
        if t == prompt + 40:
            cut_to(7)
    assert c.check_device_error() == 0


def test_weights_captured_and_replayed():
    from quantized_kv_cache_seal_gb300.kvarn import KVarNError
    c = make(max_seqs=2, block_tokens=32)
    fill(c, [300, 200], torch.float16, 680)
    qs = [tokens(8, 8, 128, torch.float16, s, 0.3) for s in (682, 683)]
    w, g = torch.zeros(c.weights_shape, device="cuda"), torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        static = qs[0].clone()
        want = torch.zeros_like(w)
        for q in qs * 2:
            c.decode_attention(0, [0, 1], q[:2].contiguous(), weights=want)
            c.window_weights(0, [0, 1], [4, 4], q, want)
        with torch.cuda.graph(g, stream=s):
            c.decode_attention(0, [0, 1], static[:2], weights=w)
            c.window_weights(0, [0, 1], [4, 4], static, w)
            with pytest.raises(KVarNError) as e:
                c.evict(0, [0], w, 2)
            assert e.value.status == 5
        for q in qs * 2:
            static.copy_(q)
            g.replay()
    s.synchronize()
    assert torch.equal(w, want)
    assert c.length(0, 0) == 300


def test_other_streams():
    """Calls that name a stream: the same results, in its order."""
    c = make(max_seqs=2, block_tokens=32)
    k, v = fill(c, [300, 200], torch.float16, 690)
    q = tokens(8, 8, 128, torch.float16, 692, 0.3)
    want = torch.zeros(c.weights_shape, device="cuda")
    out = c.decode_attention(0, [0, 1], q[:2], weights=want)
    c.window_weights(0, [0, 1], [4, 4], q, want)
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        w = torch.zeros_like(want)
        torch.cuda.synchronize()
        got = c.decode_attention(0, [0, 1], q[:2], weights=w, stream=s)
        c.window_weights(0, [0, 1], [4, 4], q, w, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(w, want)
    kept = c.evict(0, [0], want.clone(), 3, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert kept.shape == (1, 2, 3) and c.length(0, 0) == 3 * 32 + 12


def test_sequences_shorter_than_a_block():
    """One place of weights a (sequence, KV head) where no block can fill."""
    c = make(max_seqs=2, block_tokens=128, max_seq_len=100)
    k, _ = fill(c, [100, 33], torch.float16, 700)
    q = tokens(4, 8, 128, torch.float16, 702, 0.3)
    w = c.new_weights()[0]
    assert w.shape == (2, 2, 1)
    c.decode_attention(0, [0, 1], q[:2], weights=w)
    assert bool(((w - 4).abs() < 2.0 ** -15).all())
    c.window_weights(0, [0, 1], [2, 2], q, w)
    assert bool(((w - 12).abs() < 2.0 ** -14).all())
    before = w.clone()
    assert not c.evict(0, [0, 1], w, 0, 0, 0).numel() and bool((c.evict(0, [0, 1], w, 2) == -1).all())
    assert torch.equal(w, before) and c.length(0, 0) == 100


@pytest.mark.parametrize("dim", [64, 128])
def test_after_a_wait_has_given_up(dim):
    """With the timeout bit set, as by a wait of a launch before, calls end at once and say so; then all is right again."""
    from tests.test_gpu_block_edges import _words
    c = make(max_seqs=60, num_q_heads=16, head_dim=dim, block_tokens=32, dtype=torch.bfloat16, code="int8")
    fill(c, [33 + 9 * i for i in range(58)] + [4000, 700], torch.bfloat16, 710)
    ids = list(range(60))
    q = tokens(20 * 60, 16, dim, torch.bfloat16, 712, 0.3)

    def both():
        w = torch.zeros(c.weights_shape, device="cuda")
        out = c.decode_attention(0, ids, q[:60], weights=w)
        c.window_weights(0, ids, [20] * 60, q, w)
        return out, w

    want = both()
    for _ in range(5):
        _words(c, 0, 1).fill_(1)
        both()
        assert c.check_device_error() == 6
        got = both()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert c.check_device_error() == 0


def test_a_pool_of_more_than_4_gb():
    """Slots whose bytes 32 bits cannot count: eviction, prefixes and weights of what lies there."""
    c = make(max_seqs=4, num_q_heads=64, num_kv_heads=64, block_tokens=128, max_seq_len=1 << 20, pool_blocks=2400)
    filler = torch.zeros(1 << 16, 64, 128, dtype=torch.float16, device="cuda")
    for _ in range(4):
        c.append(0, [0], [1 << 16], filler, filler)
    del filler
    lens = [1500, 300]
    k, v = (tokens(sum(lens), 64, 128, torch.float16, s, 0.3) for s in (720, 721))
    c.append(0, [1, 2], lens, k, v)
    k, v = ([None] + list(torch.split(x, lens)) for x in (k, v))
    w = some_weights(c, 722)
    kept = c.evict(0, [1], w, 5)
    assert c.length(0, 1) == 5 * 128 + 1500 % 128
    got = c.read(0, [1], None, [c.length(0, 1)], dtype=torch.float32)
    sides = []
    for x, g in zip((k, v), got):
        held = block_ref.hold(x[1][:, :2], 128, "e4m3")
        pick = [[b * 128 + t for b in kept[0, h].tolist() for t in range(128)] + list(range(1500 // 128 * 128, 1500)) for h in (0, 1)]
        sides.append(torch.stack([held[pick[h], h] for h in (0, 1)], 1))
        assert same(g[:, :2], sides[-1].float())
    q = tokens(1, 64, 128, torch.float16, 723, 0.3)
    before = w.clone()
    out = c.decode_attention(0, [2], q, prefix_ids=[1], weights=w)
    parts = [torch.cat([a, block_ref.hold(x[2][:, :2], 128, "e4m3")]) for a, x in zip(sides, (k, v))]
    n = parts[0].shape[0]
    want, tol = block_ref.attend(q[:, :2].cpu(), *parts, 128 ** -0.5, [n - 1])
    check(out[:, :2], want, tol, "prefix")
    share, off = received(q[:, :2], parts[0], 128 ** -0.5, [n - 1], 128, n - 300)
    near(w[2, :2], before[2, :2], share, off, "weights")


def test_window_of_long_prompts_repeats():
    """Many steps a thread block, on every SM: the same bits each time, and right."""
    lens = [9000, 5762, 8000, 7531, 4464, 3220, 9001, 2356]
    c = make(max_seqs=8, num_q_heads=40, num_kv_heads=10, block_tokens=32, dtype=torch.bfloat16, max_seq_len=9001,
             pool_blocks=sum(n // 32 for n in lens))
    k, _ = fill(c, lens, torch.bfloat16, 730)
    ids = list(range(8))
    q = tokens(32 * 8, 40, 128, torch.bfloat16, 732, 0.3)
    first = torch.zeros(c.weights_shape, device="cuda")
    c.window_weights(0, ids, [32] * 8, q, first)
    for _ in range(40):
        w = torch.zeros_like(first)
        c.window_weights(0, ids, [32] * 8, q, w)
        assert torch.equal(w, first)
    # the mass that blocks receive: 32 queries of 4 heads
    assert bool(((first.double().sum(-1) - 128).abs() < 128 * 2.0 ** -12).all())
    for s in (0, 7):
        held = block_ref.hold(k[s][:, :1], 32, "e4m3")
        want, tol = received(q[32 * s:32 * s + 32, :4], held, 128 ** -0.5, list(range(lens[s] - 32, lens[s])), 32)
        # received()'s bound is for 2^12 tokens; sums of 2^14 in turn add as many roundings four times
        near(first[s, :1], torch.zeros_like(first[s, :1]), want, tol + want * 2.0 ** -14, s)
    assert c.check_device_error() == 0


def test_two_caches_at_once():
    """Two caches' calls on two streams, interleaved: each as alone."""
    caches, want, w, q = [], [], [], []
    for i in range(2):
        c = make(max_seqs=41, num_q_heads=32, num_kv_heads=8, block_tokens=32, max_seq_len=3000)
        fill(c, [50 + 3 * j for j in range(40)] + [2300], torch.float16, 740 + 10 * i)
        caches.append(c)
        q.append(tokens(160, 32, 128, torch.float16, 760 + i, 0.3))
    ids, pre = list(range(40)), [40] * 40

    def run(i, weights):
        c = caches[i]
        a = c.decode_attention(0, ids, q[i][:40], prefix_ids=pre, weights=weights)
        c.window_weights(0, ids, [4] * 40, q[i], weights)
        return a, c.prefill_attention(0, ids, [4] * 40, q[i], prefix_ids=pre), weights

    for i in range(2):
        want.append(run(i, torch.zeros(caches[i].weights_shape, device="cuda")))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(run(i, torch.zeros(caches[i].weights_shape, device="cuda")))
        torch.cuda.synchronize()
        for g, x in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, x))


def test_a_space_that_grows_under_a_graph():
    """A captured call keeps its workspace when later calls need a larger one, and one captured when it has to grow works too."""
    c = make(max_seqs=64, num_q_heads=64, num_kv_heads=64, block_tokens=32, max_seq_len=2000, pool_blocks=64 * 20)
    fill(c, [600] * 64, torch.float16, 780)
    q = tokens(64 * 8, 64, 128, torch.float16, 782, 0.3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        w, g, big = torch.zeros(c.weights_shape, device="cuda"), torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        c.decode_attention(0, [0], q[:1], weights=torch.zeros_like(w))
        size = c._spaces[-1].numel()
        with torch.cuda.graph(g, stream=s):
            c.decode_attention(0, [0, 1], q[:2], weights=w)
        with torch.cuda.graph(big, stream=s):
            c.window_weights(0, list(range(64)), [8] * 64, q, w)
        assert c._spaces[-1].numel() == size  # the graph's own
        want = torch.zeros_like(w)
        c.decode_attention(0, [0, 1], q[:2], weights=want)
        c.window_weights(0, list(range(64)), [8] * 64, q, want)
        assert c._spaces[-1].numel() > size
        junk = [torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(8)]
        for _ in range(2):
            w.zero_()
            g.replay()
            big.replay()
            s.synchronize()
            assert torch.equal(w, want)
    del junk
