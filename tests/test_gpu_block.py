"""GPU tests of the block cache (include/kvarn.h) against its definition in 64 bits."""
import random

import pytest
import torch

from tests import block_ref

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def make(**kw):
    from quantized_kv_cache_seal_gb300.block_cache import BlockCache
    args = dict(max_seqs=4, num_q_heads=8, num_kv_heads=2, max_seq_len=4096)
    args.update(kw)
    return BlockCache(**args)


def tokens(n, heads, dim, dtype, seed, spread=1.0):
    """[n][heads][dim] on the GPU: channels and tokens of different sizes."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, dim, generator=g) * torch.exp(spread * torch.randn(1, heads, dim, generator=g))
    x *= torch.exp(0.7 * torch.randn(n, 1, 1, generator=g))
    return x.clamp(-6e4, 6e4).to(dtype).cuda()


def as_type(v, dtype):
    """64-bit values through fp32 to the type, beyond its range its largest (NaN stays)."""
    most = torch.finfo(dtype).max
    return v.float().clamp(-most, most).to(dtype)


def same(a, b):
    """Equal as numbers, NaN where NaN."""
    a, b = a.cpu().double(), b.cpu().double()
    return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


# ------------------------------------------------------------------------------------------------ write and read
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block,dim", [(32, 64), (32, 128), (64, 64), (64, 128), (128, 64), (128, 128)])
def test_write_and_read(dtype, code, block, dim):
    lens = [1, block - 1, block, block + 1, 3 * block + 17, 0, 33]
    heads, dt = 3, TYPES[dtype]
    c = make(max_seqs=8, num_q_heads=3, num_kv_heads=heads, head_dim=dim, block_tokens=block, code=code, dtype=dt,
             max_seq_len=1000)
    k, v = (tokens(sum(lens), heads, dim, dt, s) for s in (1, 2))
    c.append(0, list(range(7)), lens, k, v)
    at = 0
    got = [x.cpu() for x in c.read(0, list(range(7)), None, lens)]
    got32 = [x.cpu() for x in c.read(0, list(range(7)), None, lens, dtype=torch.float32)]
    for i, n in enumerate(lens):
        for x, g, g32 in ((k, got[0], got32[0]), (v, got[1], got32[1])):
            want = block_ref.hold(x[at:at + n], block, code)
            assert same(g32[at:at + n], want.float())
            assert same(g[at:at + n], as_type(want, dt))
        at += n
    assert c.check_device_error() == 0


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("code,dtype", [("e4m3", "fp16"), ("int8", "bf16")])
def test_content_does_not_depend_on_the_cuts(block, code, dtype):
    """One append, token by token, odd pieces, and two layers and strided inputs: the same content."""
    n, heads, dim, dt = 2 * block + 45, 2, 128, TYPES[dtype]
    k, v = (tokens(n, heads, dim, dt, s) for s in (3, 4))
    qkv = torch.zeros(n, 12, dim, dtype=dt, device="cuda")
    qkv[:, 8:10], qkv[:, 10:] = k, v
    c = make(num_layers=2, block_tokens=block, code=code, dtype=dt)
    c.append(1, [2], [n], k, v)
    rng = random.Random(block)
    for t in range(n):
        c.append(0, [0], [1], k[t:t + 1], v[t:t + 1])
    at = 0
    while at < n:
        m = min(n - at, rng.choice([1, 7, 31, 33, block, block + 1]))
        c.append(0, [1, 3], [m, 0], qkv[at:at + m, 8:10], qkv[at:at + m, 10:])
        at += m
    whole = c.read(1, [2], None, [n])
    for s in (0, 1):
        for a, b in zip(whole, c.read(0, [s], None, [n])):
            assert torch.equal(a, b)
    assert c.length(0, 3) == 0


def test_read_of_ranges():
    c = make(block_tokens=64, code="int8")
    lens = [300, 129]
    k, v = (tokens(sum(lens), 2, 128, torch.float16, s) for s in (5, 6))
    c.append(0, [3, 0], lens, k, v)
    full = dict(zip([3, 0], [[x[:300] for x in c.read(0, [3, 0], None, lens)],
                             [x[300:] for x in c.read(0, [3, 0], None, lens)]]))
    rng = random.Random(1)
    for _ in range(40):
        ids = rng.sample([3, 0], rng.choice([1, 2]))
        starts = [rng.randrange(0, len(full[i][0]) + 1) for i in ids]
        counts = [rng.randrange(0, len(full[i][0]) - s + 1) for i, s in zip(ids, starts)]
        for side, x in enumerate(c.read(0, ids, starts, counts)):
            want = torch.cat([full[i][side][s:s + m] for i, s, m in zip(ids, starts, counts)])
            assert torch.equal(x, want)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_hard_values(code, dtype):
    """Zero blocks, the type's largest and smallest values, ties of every code, infinities and NaN."""
    dt = TYPES[dtype]
    fi = torch.finfo(dt)
    rows = []
    zero = torch.zeros(32, 64)
    rows.append(zero)
    a = zero.clone()
    a[3, 5], a[0, 0] = fi.max, -fi.max
    rows.append(a)
    a = zero.clone()
    a[31, 63] = fi.smallest_normal
    a[0, 1] = fi.smallest_normal * fi.eps  # the smallest subnormal
    rows.append(a)
    # int8 ties: amax 127 makes s = 1 and halves are ties; e4m3: amax 448, middles of neighbouring codes
    a = (torch.arange(32 * 64).view(32, 64) % 256 - 128).clamp(-127, 127) + 0.5
    a[0, 0] = 127
    rows.append(a.clamp(-127, 127))
    near = torch.arange(1, 2049, dtype=torch.float32).view(32, 64) * 2.0 ** -4
    near[0, 0] = 448
    rows.append(near)
    # quotients next to a tie: (n + 1/2) amax / 127 rounded to the type
    a = ((torch.arange(32 * 64).view(32, 64) % 253 - 126.5) * (3.14159 / 127))
    a[5, 5] = 3.14159
    rows.append(a)
    for bad in (float("inf"), float("-inf"), float("nan")):
        a = torch.randn(32, 64, generator=torch.Generator().manual_seed(9))
        a[7, 9] = bad
        rows.append(a)
    x = torch.cat(rows)[:, None].to(dt).cuda()  # [9 * 32][1][64]
    n = x.shape[0]
    c = make(num_q_heads=1, num_kv_heads=1, head_dim=64, block_tokens=32, code=code, dtype=dt)
    c.append(0, [0], [n], x, x.flip(0))
    k, v = c.read(0, [0], None, [n], dtype=torch.float32)
    assert same(k, block_ref.hold(x, 32, code).float())
    assert same(v, block_ref.hold(x.flip(0), 32, code).float())
    k16, v16 = c.read(0, [0], None, [n])
    assert same(k16, as_type(k.cpu().double(), dt)) and same(v16, as_type(v.cpu().double(), dt))


def test_pool_reuse_and_other_sequences_untouched():
    c = make(block_tokens=32, max_seqs=3, max_seq_len=400, pool_blocks=20)
    k, v = (tokens(900, 2, 128, torch.float16, s) for s in (7, 8))
    c.append(0, [0, 1], [300, 250], k[:550], v[:550])
    keep = [x.clone() for x in c.read(0, [1], None, [250])]
    c.release(0)
    c.append(0, [2], [340], k[550:890], v[550:890])  # takes the released blocks
    for a, b in zip(keep, c.read(0, [1], None, [250])):
        assert torch.equal(a, b)
    for x, g in zip((k, v), c.read(0, [2], None, [340], dtype=torch.float32)):
        assert same(g, block_ref.hold(x[550:890], 32, "e4m3").float())


def test_many_blocks_in_one_call():
    """More blocks than one launch's parameters hold."""
    n = 32 * 5100 + 9
    c = make(num_q_heads=1, num_kv_heads=1, head_dim=64, block_tokens=32, max_seqs=2, max_seq_len=n, pool_blocks=5120)
    k, v = (tokens(n + 70, 1, 64, torch.float16, s) for s in (9, 10))
    c.append(0, [1, 0], [70, n], k, v)
    for x, g in zip((k, v), c.read(0, [1, 0], None, [70, n], dtype=torch.float32)):
        x = x.cpu()
        for at in (0, 70, 70 + 32 * 4990, 70 + 32 * 5000, 70 + 32 * 5098):
            m = min(64, n + 70 - at) if at else 70
            assert same(g[at:at + m], block_ref.hold(x[at:at + m], 32, "e4m3").float())


# ------------------------------------------------------------------------------------------------ attention
def fill(c, lens, dt, seed, layer=0):
    h, d = c.cfg.num_kv_heads, c.cfg.head_dim
    k, v = tokens(sum(lens), h, d, dt, seed), tokens(sum(lens), h, d, dt, seed + 1)
    c.append(layer, list(range(len(lens))), lens, k, v)
    return _split(k, lens), _split(v, lens)


def _split(x, lens):
    return list(torch.split(x, lens))


def check(out, want, tol, what):
    out = out.cpu().double()
    assert bool(torch.isfinite(out).all()), what
    far = ((out - want).abs() / tol).max() if out.numel() else 0.0
    assert far <= 1, (what, float(far))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block,dim,hkv,r", [(32, 64, 2, 1), (64, 128, 2, 4), (128, 128, 1, 8), (32, 128, 3, 5), (64, 64, 1, 7),
                                             (128, 64, 2, 2), (64, 128, 1, 3)])
def test_decode(dtype, code, block, dim, hkv, r):
    dt = TYPES[dtype]
    lens = [1, 31, 32, 33, block, block + 1, 5 * block - 1, 777]
    c = make(max_seqs=9, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt)
    k, v = fill(c, lens, dt, 20)
    ids = [7, 8, 0, 3, 1, 6, 2, 5, 4]  # 8 is empty
    q = tokens(9, hkv * r, dim, dt, 30, 0.3)
    q[2] *= 4  # peaked weights
    out = c.decode_attention(0, ids, q)
    for row, s in enumerate(ids):
        if s == 8:
            assert not out[row].any()
            continue
        want, tol = block_ref.attend(q[row:row + 1].cpu(), block_ref.hold(k[s], block, code),
                                     block_ref.hold(v[s], block, code), dim ** -0.5, [lens[s] - 1])
        check(out[row:row + 1], want, tol, (s, lens[s]))
    assert torch.equal(out, c.decode_attention(0, ids, q))  # the same bits again
    assert c.check_device_error() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("block,dim,hkv,r", [(32, 64, 2, 1), (64, 128, 2, 4), (128, 128, 1, 8), (32, 128, 1, 5), (64, 64, 1, 7),
                                             (128, 64, 2, 2), (64, 128, 1, 3)])
def test_prefill(dtype, code, block, dim, hkv, r):
    dt = TYPES[dtype]
    lens = [1, 45, 128, 129, 300, 513, 260]
    qlens = [1, 45, 0, 129, 37, 2, 260]
    c = make(max_seqs=8, num_q_heads=hkv * r, num_kv_heads=hkv, head_dim=dim, block_tokens=block, code=code, dtype=dt)
    k, v = fill(c, lens, dt, 40)
    ids = [4, 0, 2, 6, 1, 3, 5]
    m = [qlens[s] for s in ids]
    q = tokens(sum(m), hkv * r, dim, dt, 50, 0.3)
    out = c.prefill_attention(0, ids, m, q)
    at = 0
    for s in ids:
        n = qlens[s]
        want, tol = block_ref.attend(q[at:at + n].cpu(), block_ref.hold(k[s], block, code),
                                     block_ref.hold(v[s], block, code), dim ** -0.5, list(range(lens[s] - n, lens[s])))
        check(out[at:at + n], want, tol, (s, lens[s], n))
        at += n
    assert torch.equal(out, c.prefill_attention(0, ids, m, q))
    assert c.check_device_error() == 0


@pytest.mark.parametrize("n,m", [(3000, 700), (4000, 3), (2049, 2049)])
def test_prefill_long(n, m):
    """Many key tiles; the queries of a few rows checked."""
    c = make(max_seqs=1, num_q_heads=8, num_kv_heads=2, block_tokens=64)
    k, v = fill(c, [n], torch.float16, 60)
    q = tokens(m, 8, 128, torch.float16, 61, 0.3)
    out = c.prefill_attention(0, [0], [m], q)
    rows = sorted({0, 1, m // 3, m // 2, m - 2, m - 1} & set(range(m)))
    want, tol = block_ref.attend(q[rows].cpu(), block_ref.hold(k[0], 64, "e4m3"), block_ref.hold(v[0], 64, "e4m3"),
                                 128 ** -0.5, [n - m + t for t in rows])
    check(out[rows], want, tol, (n, m))


def test_prefill_many_segments():
    """More (sequence, KV head, query tile pair) segments than the SMs hold twice: one a thread block, no cuts."""
    lens, qlens = [1500, 2100, 40], [1500, 1300, 33]
    c = make(max_seqs=3, num_q_heads=32, num_kv_heads=4, block_tokens=128, code="int8", dtype=torch.bfloat16)
    k, v = fill(c, lens, torch.bfloat16, 62)
    q = tokens(sum(qlens), 32, 128, torch.bfloat16, 64, 0.3)
    out = c.prefill_attention(0, [0, 1, 2], qlens, q)
    at = 0
    for s, (n, m) in enumerate(zip(lens, qlens)):
        rows = sorted({0, 1, 31, 32, m // 2, m - 1} & set(range(m)))
        want, tol = block_ref.attend(q[[at + t for t in rows]].cpu(), block_ref.hold(k[s], 128, "int8"),
                                     block_ref.hold(v[s], 128, "int8"), 128 ** -0.5, [n - m + t for t in rows])
        check(out[[at + t for t in rows]], want, tol, s)
        at += m


@pytest.mark.parametrize("scale", [-0.05, 0.0, 0.5])
def test_other_scales(scale):
    c = make(max_seqs=2, block_tokens=32)
    lens = [150, 45]
    k, v = fill(c, lens, torch.float16, 66)
    q = tokens(50, 8, 128, torch.float16, 68, 0.3)
    out = c.prefill_attention(0, [0, 1], [20, 30], q, scale=scale)
    one = c.decode_attention(0, [0, 1], q[[19, 49]].contiguous(), scale=scale)
    at = 0
    for s, (n, m) in enumerate(zip(lens, [20, 30])):
        held = [block_ref.hold(x[s], 32, "e4m3") for x in (k, v)]
        want, tol = block_ref.attend(q[at:at + m].cpu(), *held, scale, list(range(n - m, n)))
        check(out[at:at + m], want, tol, s)
        check(one[s:s + 1], want[-1:], tol[-1:], s)
        at += m


@pytest.mark.parametrize("lens", [[20000], [9000, 40, 3000], [700] * 40])
def test_decode_split(lens):
    """Long sequences cut over many thread blocks, and many sequences in one."""
    c = make(max_seqs=len(lens), num_q_heads=8, num_kv_heads=2, block_tokens=128, code="int8", max_seq_len=20000,
             pool_blocks=sum(n // 128 for n in lens))
    k, v = fill(c, lens, torch.float16, 70)
    q = tokens(len(lens), 8, 128, torch.float16, 71, 0.3)
    out = c.decode_attention(0, list(range(len(lens))), q)
    for s in sorted({0, 1, 2, len(lens) - 1} & set(range(len(lens)))):
        want, tol = block_ref.attend(q[s:s + 1].cpu(), block_ref.hold(k[s], 128, "int8"), block_ref.hold(v[s], 128, "int8"),
                                     128 ** -0.5, [lens[s] - 1])
        check(out[s:s + 1], want, tol, s)


def test_step_and_prefill_equal_their_parts():
    a, b = make(block_tokens=32), make(block_tokens=32)
    k, v = (tokens(200, 2, 128, torch.float16, s) for s in (80, 81))
    q = tokens(200, 8, 128, torch.float16, 82)
    got = a.prefill(0, [0, 1], [60, 95], k[:155], v[:155], q[:155])
    b.append(0, [0, 1], [60, 95], k[:155], v[:155])
    assert torch.equal(got, b.prefill_attention(0, [0, 1], [60, 95], q[:155]))
    for t in range(155, 195, 2):
        got = a.decode_step(0, [1, 0], k[t:t + 2], v[t:t + 2], q[t:t + 2])
        b.append(0, [1, 0], [1, 1], k[t:t + 2], v[t:t + 2])
        assert torch.equal(got, b.decode_attention(0, [1, 0], q[t:t + 2]))


def test_scales_of_very_different_size():
    """V blocks whose scales differ by 2^20 and logits that favour the small one: its weights are not lost."""
    c = make(num_q_heads=2, num_kv_heads=1, block_tokens=32, max_seqs=1)
    g = torch.Generator().manual_seed(3)
    k = torch.randn(96, 1, 128, generator=g)
    v = torch.randn(96, 1, 128, generator=g)
    q = torch.randn(1, 2, 128, generator=g)
    k[32:64] = q[0, :1] * 2.0  # these tokens take all the weight
    v[:32] *= 1000.0
    v[32:64] *= 2.0 ** -10
    k, v, q = (x.half().cuda() for x in (k, v, q))
    c.append(0, [0], [96], k, v)
    for out in (c.decode_attention(0, [0], q), c.prefill_attention(0, [0], [1], q)):
        want, tol = block_ref.attend(q.cpu(), block_ref.hold(k, 32, "e4m3"), block_ref.hold(v, 32, "e4m3"), 128 ** -0.5, [95])
        check(out, want, tol, "scales")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("power", [-40, -18, 0, 40])
@pytest.mark.parametrize("where", ["sealed", "exact"])
def test_values_of_zero_beside_others(where, power, code):
    """Tokens whose V is zero (a whole block, the exact tokens) keep their weight, and the others their bits."""
    c = make(num_q_heads=4, num_kv_heads=1, block_tokens=32, dtype=torch.bfloat16, code=code, max_seqs=1)
    k, v, q = (tokens(n, h, 128, torch.bfloat16, s, 0.2) for n, h, s in ((106, 1, 31), (106, 1, 32), (106, 4, 33)))
    v = v * 2.0 ** power
    v[32:64 if where == "sealed" else 32] = 0
    v[106 if where == "sealed" else 96:] = 0
    c.append(0, [0], [106], k, v)
    held = [block_ref.hold(x, 32, code) for x in (k, v)]
    want, tol = block_ref.attend(q.cpu(), *held, 128 ** -0.5, list(range(106)))
    check(c.prefill_attention(0, [0], [106], q), want, tol, "prefill")
    check(c.decode_attention(0, [0], q[105:]), want[105:], tol[105:], "decode")


def test_bf16_of_large_range():
    """bf16 queries, keys and values beyond f16's range (their products are not)."""
    c = make(num_q_heads=4, num_kv_heads=1, block_tokens=32, dtype=torch.bfloat16, max_seqs=1)
    k, v, q = (tokens(n, h, 128, torch.bfloat16, s, 0.2) for n, h, s in ((75, 1, 1), (75, 1, 2), (75, 4, 3)))
    k, v, q = k * 2.0 ** -40, v * 2.0 ** 30, q * 2.0 ** 38
    c.append(0, [0], [75], k, v)
    held = [block_ref.hold(x, 32, "e4m3") for x in (k, v)]
    want, tol = block_ref.attend(q.cpu(), *held, 128 ** -0.5, list(range(75)))
    check(c.prefill_attention(0, [0], [75], q), want, tol, "prefill")
    check(c.decode_attention(0, [0], q[74:]), want[74:], tol[74:], "decode")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_nan_reaches_its_head_only(code):
    """A sealed block or a tail with a NaN makes its KV head's outputs NaN, and no other's; unwritten rows and
    channels never show."""
    c = make(block_tokens=32, code=code)
    c.mem.fill_(0xff)  # whatever was there before the cache
    k, v = (tokens(140, 2, 128, torch.float16, s) for s in (90, 91))
    q = tokens(3, 8, 128, torch.float16, 92)
    c.append(0, [0, 1, 2], [45, 45, 50], k, v)
    assert bool(torch.isfinite(c.decode_attention(0, [0, 1, 2], q)).all())
    assert bool(torch.isfinite(c.prefill_attention(0, [0, 1, 2], [1, 1, 1], q)).all())
    c.release([0, 1, 2])
    v[10, 1, 5] = float("nan")   # sequence 0, sealed block
    v[45 + 44, 0, 7] = float("nan")  # sequence 1, tail
    k[90 + 49, 1, 0] = float("nan")  # sequence 2, tail
    c.append(0, [0, 1, 2], [45, 45, 50], k, v)
    for out in (c.decode_attention(0, [0, 1, 2], q), c.prefill_attention(0, [0, 1, 2], [1, 1, 1], q)):
        assert bool(torch.isfinite(out[0, :4]).all()) and bool(out[0, 4:].isnan().all())
        assert bool(torch.isfinite(out[1, 4:]).all()) and bool(out[1, :4, 7].isnan().all())
        assert bool(torch.isfinite(out[2, :4]).all()) and bool(out[2, 4:].isnan().all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("at", [70, 190, 212])
@pytest.mark.parametrize("side", ["k", "v"])
def test_nan_of_a_later_token_stays_there(dtype, at, side):
    """A NaN or infinity at position `at` (sealed blocks up to 191, then the tail): queries before its block, or
    before the token itself where it is still exact, are as without it; later ones are NaN."""
    dt = TYPES[dtype]
    n, m = 220, 200
    k, v = (tokens(n, 1, 128, dt, s) for s in (100, 101))
    q = tokens(m, 4, 128, dt, 102, 0.3)
    outs = []
    for value in (None, float("nan"), float("inf")):
        x, y = k.clone(), v.clone()
        if value is not None:
            (x if side == "k" else y)[at, 0, 3] = value
        c = make(num_q_heads=4, num_kv_heads=1, block_tokens=64, dtype=dt, max_seqs=1)
        c.append(0, [0], [n], x, y)
        outs.append(c.prefill_attention(0, [0], [m], q))
    first = at if at >= 192 else at // 64 * 64  # the first token that is not finite in the cache
    rows = slice(0, first - (n - m))
    want, tol = block_ref.attend(q[rows].cpu(), block_ref.hold(k[:first], 64, "e4m3"), block_ref.hold(v[:first], 64, "e4m3"),
                                 128 ** -0.5, list(range(n - m, first)))
    for out in outs:
        check(out[rows], want, tol, (at, side))
    assert bool(torch.isfinite(outs[0]).all())
    channels = slice(0, 128) if side == "k" or at < 192 else slice(3, 4)
    assert bool(outs[1][first - (n - m):, :, channels].isnan().all())
    if at < 192:
        assert bool(outs[2][first - (n - m):].isnan().all())


def test_nothing_around_the_outputs_is_written():
    """Outputs inside larger buffers: what stands before and behind stays, for every call that writes one."""
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    for dim, hkv, r in ((128, 2, 3), (64, 1, 8)):
        hq = hkv * r
        c = make(num_q_heads=hq, num_kv_heads=hkv, head_dim=dim, block_tokens=32)
        lens = [100, 33, 7]
        fill(c, lens, torch.float16, 110)
        for ids, m in (([0, 1, 2], None), ([1, 0], [33, 50]), ([2], [1]), ([0, 2], [0, 7])):
            rows = len(ids) if m is None else sum(m)
            q = tokens(rows, hq, dim, torch.float16, 111)
            big = torch.full((rows + 20, hq, dim), 7.0, dtype=torch.float16, device="cuda")
            out = big[10:10 + rows]
            if m is None:
                c.decode_attention(0, ids, q, out=out)
            else:
                c.prefill_attention(0, ids, m, q, out=out)
            assert bool((big[:10] == 7).all()) and bool((big[10 + rows:] == 7).all())
            assert not bool((out == 7).all(dim=-1).any())
    qkv = tokens(37, 10, 80, torch.bfloat16, 112)
    big = torch.full((57, 10, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    pos, freqs = torch.arange(37, dtype=torch.int32, device="cuda"), torch.rand(20, dtype=torch.float64, device="cuda")
    qk_norm_rope(qkv[:, :6], qkv[:, 6:8], pos, freqs, q_out=big[10:47, :6], k_out=big[10:47, 6:8])
    assert bool((big[:10] == 7).all()) and bool((big[47:] == 7).all()) and bool((big[:, 8:] == 7).all())


def test_two_caches_on_two_streams():
    """Caches have workspaces of their own: calls on two of them may overlap."""
    a, b = (make(max_seqs=2, block_tokens=32, max_seq_len=4000) for _ in range(2))
    fill(a, [3000, 1000], torch.float16, 120)
    fill(b, [2000, 3500], torch.float16, 122)
    q = tokens(600, 8, 128, torch.float16, 124, 0.3)
    want = [(c.decode_attention(0, [0, 1], q[:2]), c.prefill_attention(0, [0, 1], [400, 200], q)) for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, c in enumerate((a, b)):
            got[i].append((c.decode_attention(0, [0, 1], q[:2], stream=streams[i]),
                           c.prefill_attention(0, [0, 1], [400, 200], q, stream=streams[i])))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for x in g:
            assert torch.equal(x[0], w[0]) and torch.equal(x[1], w[1])


def test_streams_and_graphs():
    """Calls on another stream; decode, prefill and read captured and replayed with new queries; calls that change
    the cache refused while capturing."""
    from quantized_kv_cache_seal_gb300.kvarn import KVarNError
    c = make(block_tokens=32)
    k, v = (tokens(150, 2, 128, torch.float16, s) for s in (95, 96))
    qs = [tokens(2, 8, 128, torch.float16, s) for s in (97, 98)]
    fresh = make(block_tokens=32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.append(0, [0, 1], [100, 50], k, v)
        want = [(c.decode_attention(0, [0, 1], q), c.prefill_attention(0, [0], [2], q)) for q in qs]
        other = c.decode_attention(0, [0, 1], qs[0], stream=s.cuda_stream)
        static = qs[0].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = c.decode_attention(0, [0, 1], static), c.prefill_attention(0, [0], [2], static)
            back = c.read(0, [0], [90], [10])
            for call in (lambda: c.append(0, [0], [1], k[:1], v[:1]), lambda: fresh.decode_attention(0, [0], qs[0][:1]),
                         lambda: c.decode_step(0, [0], k[:1], v[:1], qs[0][:1])):
                with pytest.raises(KVarNError) as e:
                    call()
                assert e.value.status == 5
    s.synchronize()
    assert torch.equal(other, want[0][0])
    assert c.length(0, 0) == 100
    for q, w in list(zip(qs, want)) * 2:
        with torch.cuda.stream(s):
            static.copy_(q)
            g.replay()
        s.synchronize()
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    assert torch.equal(back[0], c.read(0, [0], [90], [10])[0])


def test_replay_after_the_cache_has_moved_on():
    """A captured call sees the lengths of its capture while its partial block has not filled (or where it had none)."""
    c = make(block_tokens=32, max_seqs=2)
    k, v = (tokens(227, 2, 128, torch.float16, s) for s in (61, 62))
    q = tokens(2, 8, 128, torch.float16, 63)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.append(0, [0, 1], [64, 40], k[:104], v[:104])
        want = c.decode_attention(0, [0, 1], q), c.prefill_attention(0, [1], [2], q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = c.decode_attention(0, [0, 1], q), c.prefill_attention(0, [1], [2], q)
        c.append(0, [0, 1], [100, 23], k[104:], v[104:])
        g.replay()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_stream_that_a_call_names_owns_its_results():
    from quantized_kv_cache_seal_gb300 import kvarn as K
    device, side = torch.device("cuda", 0), torch.cuda.Stream()
    with torch.cuda.stream(side):
        with K.on_device(device, 0) as s:  # the default stream by its address
            assert s == 0 and torch.cuda.current_stream() == torch.cuda.default_stream()
        with K.on_device(device) as s:
            assert s == side.cuda_stream
    for name in (side, side.cuda_stream):
        with K.on_device(device, name) as s:
            assert s == side.cuda_stream and torch.cuda.current_stream().cuda_stream == s
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_chain_as_a_layer_uses_it():
    """Packed projection -> norm + rotation -> prefill, then decode steps, against the definitions in 64 bits."""
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    hq, hkv, d, dt = 8, 2, 128, torch.bfloat16
    c = make(num_q_heads=hq, num_kv_heads=hkv, block_tokens=32, dtype=dt, code="int8", max_seqs=1)
    qkv = tokens(120, hq + 2 * hkv, d, dt, 99, 0.3)
    wq, wk = (torch.rand(d, generator=torch.Generator().manual_seed(s)).cuda() + 0.5 for s in (1, 2))
    freqs = 1e6 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    pos = torch.arange(120, dtype=torch.int32, device="cuda")

    def rows(a, b):
        q, k = qk_norm_rope(qkv[a:b, :hq], qkv[a:b, hq:hq + hkv], pos[a:b], freqs, q_weight=wq, k_weight=wk)
        return q, k, qkv[a:b, hq + hkv:]

    q, k, v = rows(0, 100)
    outs, qs, ks = [c.prefill(0, [0], [100], k, v, q)], [q], [k]
    seen = [block_ref.attend(q.cpu(), block_ref.hold(k, 32, "int8"), block_ref.hold(v, 32, "int8"), d ** -0.5,
                             list(range(100)))]
    for t in range(100, 120):
        q, k, v = rows(t, t + 1)
        outs.append(c.decode_step(0, [0], k, v, q))
        ks.append(k)
        held = [block_ref.hold(x, 32, "int8") for x in (torch.cat(ks), qkv[:t + 1, hq + hkv:])]
        seen.append(block_ref.attend(q.cpu(), *held, d ** -0.5, [t]))
    for o, (want, tol) in zip(outs, seen):
        check(o, want, tol, "chain")


# ------------------------------------------------------------------------------------------------ norm + rotation
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (128, 64), (80, 80), (96, 48), (256, 256), (192, 96), (8, 8), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("types", [("fp16", "fp16"), ("bf16", "fp16"), ("bf16", "bf16"), ("fp16", "bf16")])
def test_norm_rope(dim, rot, interleaved, types):
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    src, dst = TYPES[types[0]], TYPES[types[1]]
    freqs = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    for t, hq, hkv in ((1, 1, 1), (7, 5, 2), (1000, 16, 3)):
        qkv = tokens(t, hq + 2 * hkv, dim, src, t, 0.3)
        g = torch.Generator().manual_seed(t)
        pos = torch.randint(-5, 2 ** 31 - 1 if t == 7 else 300000, (t,), generator=g, dtype=torch.int32).cuda()
        w = torch.rand(dim, generator=g).cuda() + 0.5
        for qw, kw in ((w, None), (None, w), (w, w)):
            q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
            got = qk_norm_rope(q, k, pos, freqs, qw, kw, eps=1e-5, interleaved=interleaved, dtype=dst)
            for x, wt, y in ((q, qw, got[0]), (k, kw, got[1])):
                want, tol = block_ref.norm_rope(x, wt, pos, freqs, interleaved, 1e-5)
                # a double angle of 2^31 turns is itself good to 2^-21 rad
                tol = tol + (want.abs().amax(-1, keepdim=True) * 2 * 2.0 ** -20 if t == 7 else 0)
                tol = tol + want.abs() * torch.finfo(dst).eps / 2 + float(torch.finfo(dst).smallest_normal)
                assert y.dtype == dst and y.is_contiguous()
                assert float(((y.cpu().double() - want).abs() / tol).max()) <= 1
        alone = qk_norm_rope(q, None, pos, freqs, w, interleaved=interleaved, dtype=dst)
        assert alone[1] is None


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_frequencies(interleaved):
    """Frequencies of any sign and size: none, tiny, whole turns and many turns a position."""
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    freqs = torch.tensor([0.0, -0.0, 1e-300, 2.0 ** -1040, 2.0 ** -40, -2.0 ** -13, 0.5, -1.0, 2.0, 3.141592653589793,
                          6.283185307179586, -6.283185307179587, 12.5, 1000.123, -123456.789, 1048577.0], dtype=torch.float64,
                         device="cuda")
    x = tokens(40, 3, 32, torch.float16, 5, 0.3)
    pos = torch.arange(-20, 20, dtype=torch.int32, device="cuda") * 51
    got, _ = qk_norm_rope(x, None, pos, freqs, interleaved=interleaved)
    # the angle, up to 2^30 in 64 bits, is good to 2^-23 there
    want, tol = block_ref.norm_rope(x, None, pos, freqs, interleaved, 0)
    tol = tol + want.abs().amax(-1, keepdim=True) * 2 * 2.0 ** -23 + want.abs() * 2.0 ** -11 + 2.0 ** -24
    assert float(((got.cpu().double() - want).abs() / tol).max()) <= 1


@pytest.mark.parametrize("tokens_, hq, hkv, dim", [(1000, 40, 8, 128), (2100, 20, 3, 64), (1530, 32, 9, 128), (900, 70, 20, 128),
                                                  (1600, 64, 30, 128),
                                                  (800, 17, 0, 256), (3, 0, 5, 256)])
def test_norm_rope_by_items(tokens_, hq, hkv, dim):
    """The ways in which heads are cut into items, with and without a side."""
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    x = tokens(tokens_, hq + hkv, dim, torch.bfloat16, 6, 0.3)
    pos = torch.arange(tokens_, dtype=torch.int32, device="cuda")
    freqs = 1e4 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    w = torch.rand(dim, generator=torch.Generator().manual_seed(7)).cuda() + 0.5
    q, k = (x[:, :hq], x[:, hq:]) if hkv else (x, None)
    got = qk_norm_rope(q, k, pos, freqs, w if hq else None, w if hkv else None)
    for part, y in zip((q, k), got):
        if part is not None and part.shape[1]:
            want, tol = block_ref.norm_rope(part, w, pos, freqs, False, 1e-6)
            tol = tol + want.abs() * 2.0 ** -8 + 2.0 ** -126
            assert float(((y.cpu().double() - want).abs() / tol).max()) <= 1


def test_norm_rope_in_place_and_captured():
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    qkv = tokens(300, 12, 128, torch.float16, 5, 0.3)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    freqs = 1e4 ** (-torch.arange(0, 128, 2, dtype=torch.float64, device="cuda") / 128)
    w = torch.rand(128, device="cuda") + 0.5
    want = qk_norm_rope(qkv[:, :8], qkv[:, 8:10], pos, freqs, w, w)
    keep = qkv[:, 10:].clone()
    work = qkv.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        qk_norm_rope(work[:, :8], work[:, 8:10], pos, freqs, w, w, q_out=work[:, :8], k_out=work[:, 8:10])
    torch.cuda.synchronize()
    for _ in range(2):
        work.copy_(qkv)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(work[:, :8], want[0]) and torch.equal(work[:, 8:10], want[1])
        assert torch.equal(work[:, 10:], keep)
    a = qk_norm_rope(qkv[:, :8], qkv[:, 8:10], pos, freqs, w, w, stream=s)
    s.synchronize()
    assert torch.equal(a[0], want[0])


def test_norm_rope_refusals():
    from quantized_kv_cache_seal_gb300.kvarn import KVarNError
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    q = tokens(4, 2, 64, torch.float16, 1)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    for args, kw in (((q.float(), None, pos, f), {}), ((q, None, pos.long(), f), {}), ((q, None, pos[:3], f), {}),
                     ((q, None, pos, f.float()), {}), ((q, None, pos, f, f.float()[:5]), {}),
                     ((q, q.bfloat16(), pos, f), {}), ((q.transpose(1, 2), None, pos, f), {}),
                     ((q, None, pos, f), dict(q_out=q[:, :1])), ((q, None, pos, f), dict(k_weight=f.float())),
                     ((q, None, pos.cpu(), f), {}), ((q, None, pos, f), dict(dtype=torch.float32))):
        with pytest.raises(ValueError):
            qk_norm_rope(*args, **kw)
    for bad in (torch.ones(40, dtype=torch.float64, device="cuda"), torch.ones(3, dtype=torch.float64, device="cuda")):
        with pytest.raises(KVarNError):
            qk_norm_rope(q, None, pos, bad)
    with pytest.raises(KVarNError):  # not 16-byte aligned
        x = torch.zeros(4 * 128 + 8, dtype=torch.float16, device="cuda")[4:4 + 512].view(4, 2, 64)
        qk_norm_rope(x, None, pos, f)
