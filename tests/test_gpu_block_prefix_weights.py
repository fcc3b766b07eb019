"""GPU tests of the weights that blocks receive behind a shared prefix (include/kvarn.h) where the prefix's part of a row's
denominator is nothing, far from 1, or walked by each sequence itself."""
import pytest
import torch

from tests import block_ref
from tests.test_gpu_block import TYPES, fill, make, tokens
from tests.test_gpu_block_evict import SHAPES, near, received, some_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("seqs,n", [(40, 2100), (3, 200)])
def test_a_prefix_without_weight(seqs, n, code, dtype):
    """Logits of the prefix that all leave fp32 downwards (-inf): rows are those over the sequence's own tokens, and where
    these are -inf as well the rows add nothing. Own keys are zero, so that their logits are 0 and their shares equal;
    sequence 1 has the prefix's keys instead. The prefix walked once and by each sequence."""
    dt, own = TYPES[dtype], 37
    c = make(max_seqs=seqs + 1, num_q_heads=32, num_kv_heads=8, block_tokens=32, max_seq_len=2200, code=code, dtype=dt)
    k = torch.zeros(n + seqs * own, 8, 128, dtype=dt, device="cuda")
    k[:n] = -8
    k[n + own:n + 2 * own] = -8
    v = tokens(n + seqs * own, 8, 128, dt, 1001, 0.3)
    c.append(0, [seqs] + list(range(seqs)), [n] + [own] * seqs, k, v)
    q = torch.full((seqs, 32, 128), 4, dtype=dt, device="cuda")
    w = some_weights(c, 1002)
    before = w.clone()
    out = c.decode_attention(0, list(range(seqs)), q, scale=1e36, prefix_ids=[seqs] * seqs, weights=w)
    share = torch.tensor([[4 * 32 / own, 4 * 5 / own]] * 8, dtype=torch.float64)
    nothing = torch.zeros_like(share)
    # a weight of 1 / 37: its sum's 37 roundings of 2^-24, exponentials and the division, four heads' sums: under 2^-17
    for s in range(seqs):
        near(w[s], before[s], nothing if s == 1 else share, share * 2.0 ** -17, s)
    assert torch.equal(w[1], before[1])
    assert not out[1].any() and torch.isfinite(out).all() and out[0].any()
    assert c.check_device_error() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("seqs,n,hkv", [(40, 2100, 8), (200, 1500, 40)])
def test_logits_far_from_zero(seqs, n, hkv, dtype):
    """Logits of 4,096 and a little, all exact, behind a prefix walked once (of single row tiles, and of so many that they go in
    pairs): a share is as exact as beside logits near 0. The log2 of a denominator would be rounded to 2^-12 there.

    The bound: sums over the tokens take fewer than 2^7 roundings of 2^-24 one after another, exponentials 2^-22 each, the
    division and the four heads a few more: under 2^-16 of a share."""
    dt, own, r, g = TYPES[dtype], 40, 4, torch.Generator().manual_seed(1010)
    scale = next(s for s in (0.6931471824645996, 0.6931471228599548, 0.693147242069244)
                 if float(torch.tensor(s, dtype=torch.float32) * torch.tensor(1.4426950408889634, dtype=torch.float32)) == 1)
    c = make(max_seqs=seqs + 1, num_q_heads=hkv * r, num_kv_heads=hkv, block_tokens=32, max_seq_len=2200, dtype=dt)
    total = n + seqs * own
    k = torch.zeros(total, hkv, 128)
    k[:, :, 0] = 64
    k[:, :, 1] = torch.randint(0, 4, (total, hkv), generator=g).float()
    q = torch.zeros(seqs, hkv * r, 128)
    q[:, :, 0] = 64
    q[:, :, 1] = torch.randint(-3, 4, (seqs, hkv * r), generator=g).float() / 2
    v = tokens(total, hkv, 128, dt, 1011, 0.3)
    held = block_ref.hold(k[:n + 32].to(dt), 32, "e4m3")
    assert torch.equal(held, k[:n + 32].double())
    c.append(0, [seqs] + list(range(seqs)), [n] + [own] * seqs, k.to(dt).cuda(), v)
    w = torch.zeros(c.weights_shape, device="cuda")
    c.decode_attention(0, list(range(seqs)), q.to(dt).cuda(), scale=scale, prefix_ids=[seqs] * seqs, weights=w)
    k, q = k.double(), q.double()
    for s in {0, 1, 2, 3, 5, seqs - 1}:
        mine = torch.cat([k[:n], k[n + s * own:n + (s + 1) * own]])
        x = torch.einsum("hrd,nhd->hrn", q[s].view(hkv, r, 128), mine)
        p = torch.exp2(x - x.amax(-1, keepdim=True))
        p = (p / p.sum(-1, keepdim=True)).sum(1)[:, n:]
        want = torch.stack([p[:, :32].sum(-1), p[:, 32:].sum(-1)], -1)
        near(w[s], torch.zeros_like(w[s]), want, want * 2.0 ** -16, s)
    assert c.check_device_error() == 0


# ------------------------------------------------------------------------------------------------ last queries of a prompt
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block,dim,hkv,r", SHAPES)
def test_window_behind_a_prefix(dtype, code, block, dim, hkv, r):
    """Prompts' last queries: shares of the softmax over prefix and sequence, of the prefix itself nothing. Prefixes of every
    kind of length, one for several sequences, none and an empty one."""
    dt = TYPES[dtype]
    lens = [1, 45, 128, 129, 300, 60, 260, 1, 129, 5 * block - 1, 777]
    m_of = [1, 45, 0, 128, 37, 2, 100]
    c = make(max_seqs=12, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt)
    k, _ = fill(c, lens, dt, 1020)
    ids = [4, 0, 2, 6, 1, 3, 5]
    pre = [7, 8, 8, 10, None, 9, 11]  # 11 is empty
    m = [m_of[s] for s in ids]
    q = tokens(sum(m), hkv * r, dim, dt, 1030, 0.3)
    w = some_weights(c, 1031)
    before = w.clone()
    c.window_weights(0, ids, m, q, w, prefix_ids=pre)
    at = 0
    for s, p, n in zip(ids, pre, m):
        parts, first = [block_ref.hold(k[s], block, code)], 0
        if p not in (None, 11):
            parts.insert(0, block_ref.hold(k[p], block, code))
            first = lens[p]
        if n:
            want, tol = received(q[at:at + n], torch.cat(parts), dim ** -0.5, [first + lens[s] - n + t for t in range(n)], block, first)
            near(w[s], before[s], want, tol, s)
        else:
            assert torch.equal(w[s], before[s])
        at += n
    assert torch.equal(w[7:], before[7:])
    again = before.clone()
    c.window_weights(0, ids, m, q, again, prefix_ids=pre)
    assert torch.equal(w, again)
    # without a prefix by either form
    a, b = before.clone(), before.clone()
    c.window_weights(0, ids, m, q, a)
    c.window_weights(0, ids, m, q, b, prefix_ids=[-1] * 7)
    assert torch.equal(a, b)
    assert c.check_device_error() == 0


@pytest.mark.parametrize("scale", [-0.05, 0.0, 0.5])
def test_window_and_decode_agree_behind_a_prefix(scale):
    """One query of a sequence either way, against the definition."""
    c = make(max_seqs=4, block_tokens=64, num_q_heads=10, num_kv_heads=2, dtype=torch.bfloat16)
    lens = [200, 63, 1, 333]
    k, _ = fill(c, lens, torch.bfloat16, 1040)
    q = tokens(3, 10, 128, torch.bfloat16, 1041, 0.3)
    a, b = (torch.zeros(c.weights_shape, device="cuda") for _ in (0, 1))
    c.decode_attention(0, [0, 1, 2], q, scale=scale, weights=a, prefix_ids=[3, 3, None])
    c.window_weights(0, [0, 1, 2], [1, 1, 1], q, b, scale=scale, prefix_ids=[3, 3, None])
    for s in range(3):
        first = 0 if s == 2 else 333
        held = [block_ref.hold(k[x], 64, "e4m3") for x in ([s] if s == 2 else [3, s])]
        want, tol = received(q[s:s + 1], torch.cat(held), scale, [first + lens[s] - 1], 64, first)
        for w in (a, b):
            near(w[s], torch.zeros_like(w[s]), want, tol, s)


def test_window_behind_a_long_prefix():
    """Steps of prefix and sequence cut over every SM: the same bits each time, and right; a prefix with a NaN key behind which rows
    of its head add nothing."""
    lens, n = [2500, 33, 700, 1, 1024, 300], 9001
    c = make(max_seqs=8, num_q_heads=40, num_kv_heads=10, block_tokens=32, dtype=torch.bfloat16, max_seq_len=9001,
             pool_blocks=sum(x // 32 for x in lens + [n]) + 2)
    k, _ = fill(c, lens + [n], torch.bfloat16, 1050)
    bad = tokens(40, 10, 128, torch.bfloat16, 1052)
    bad[35, 2, 7] = float("nan")
    c.append(0, [7], [40], bad, bad)
    ids, m = list(range(6)), [32, 33, 1, 1, 128, 7]
    q = tokens(sum(m), 40, 128, torch.bfloat16, 1053, 0.3)
    pre = [6, 6, None, 6, 6, 7]
    first = torch.zeros(c.weights_shape, device="cuda")
    c.window_weights(0, ids, m, q, first, prefix_ids=pre)
    for _ in range(20):
        w = torch.zeros_like(first)
        c.window_weights(0, ids, m, q, w, prefix_ids=pre)
        assert torch.equal(w, first)
    assert torch.isfinite(first).all() and not first[5, 2].any() and first[5, 3].any() and not first[6:].any()
    at = 0
    for s in range(6):
        if s < 5:
            held = [block_ref.hold(k[x][:, :1], 32, "e4m3") for x in ([6, s] if pre[s] == 6 else [s])]
            skip = n if pre[s] == 6 else 0
            want, tol = received(q[at:at + m[s], :4], torch.cat(held), 128 ** -0.5,
                                 [skip + lens[s] - m[s] + t for t in range(m[s])], 32, skip)
            # received()'s bound is for 2^12 tokens; sums of 2^14 in turn add as many roundings four times
            near(first[s, :1], torch.zeros_like(first[s, :1]), want, tol + want * 2.0 ** -14, s)
        at += m[s]
    assert c.check_device_error() == 0


def test_window_behind_a_prefix_captured_and_on_other_streams():
    c = make(max_seqs=3, block_tokens=32)
    fill(c, [300, 200, 150], torch.float16, 1060)
    qs = [tokens(8, 8, 128, torch.float16, s, 0.3) for s in (1062, 1063)]
    w, g, s = torch.zeros(c.weights_shape, device="cuda"), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        static, want = qs[0].clone(), torch.zeros_like(w)
        for q in qs * 2:
            c.window_weights(0, [0, 1], [4, 4], q, want, prefix_ids=[2, 2])
        with torch.cuda.graph(g, stream=s):
            c.window_weights(0, [0, 1], [4, 4], static, w, prefix_ids=[2, 2])
        for q in qs * 2:
            static.copy_(q)
            g.replay()
    s.synchronize()
    assert torch.equal(w, want) and w.any()
    for t in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        w = torch.zeros_like(want)
        torch.cuda.synchronize()
        for q in qs * 2:
            c.window_weights(0, [0, 1], [4, 4], q, w, prefix_ids=[2, 2], stream=t)
        torch.cuda.synchronize()
        assert torch.equal(w, want)


def test_window_behind_a_prefix_leaves_the_rest_of_its_workspace():
    from quantized_kv_cache_seal_gb300 import kvarn as K
    c = make(max_seqs=3, num_q_heads=10, num_kv_heads=2, block_tokens=32)
    fill(c, [300, 33, 1000], torch.float16, 1070)
    q = tokens(10, 10, 128, torch.float16, 1071, 0.3)
    w = torch.zeros(c.weights_shape, device="cuda")
    n = K.kvarn_block_window_workspace_prefixes(c.handle, 0, [0, 1], [2, 2], [7, 3])
    assert n > K.kvarn_block_window_workspace(c.handle, 0, [0, 1], [7, 3]) > 0
    space = torch.full((n + 1024,), 0xa5, dtype=torch.uint8, device="cuda")
    base = (space.data_ptr() + 255) // 256 * 256 + 256
    K.kvarn_block_window_weights_prefixes(c.handle, 0, [0, 1], [2, 2], [7, 3], q, 0.1, w, base, n,
                                          torch.cuda.current_stream().cuda_stream)
    at = base - space.data_ptr()
    assert bool((space[:at] == 0xa5).all()) and bool((space[at + n:] == 0xa5).all())
    assert w[0].any() and w[1].any() and not w[2].any()
