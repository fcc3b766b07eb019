"""GPU tests of the block cache at the edges of its number range and of its calls (include/kvarn.h), against the
definition in 64 bits."""
import pytest
import torch

from tests import block_ref
from tests.test_gpu_block import TYPES, check, fill, make, tokens

pytestmark = pytest.mark.gpu


def held(x, block, code="e4m3"):
    return block_ref.hold(x, block, code)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("at", [70, 100])
def test_infinite_key_of_an_exact_token(dtype, dim, at):
    """A key with an infinity whose logit is -inf takes its token out and leaves the other tokens' logits alone; where
    the logit is +inf the output is NaN. Both attention kernels."""
    dt, n = TYPES[dtype], 110  # exact from 64 on
    k, v, q = (tokens(m, h, dim, dt, s, 0.3) for m, h, s in ((n, 1, 201), (n, 1, 202), (2, 4, 203)))
    k[at, 0, 5] = float("inf")
    q[:, :, 5] = torch.tensor([-1.0, -0.25, 1.0, 2.0], dtype=dt).cuda()  # by head
    c = make(num_q_heads=4, num_kv_heads=1, head_dim=dim, block_tokens=64, dtype=dt, max_seqs=1)
    c.append(0, [0], [n], k, v)
    rest = [i for i in range(n) if i != at]
    kk, vv = (held(x, 64)[rest] for x in (k, v))
    want, tol = block_ref.attend(q[:, :2].contiguous().cpu(), kk, vv, dim ** -0.5, [n - 3, n - 2])
    both = c.prefill_attention(0, [0], [2], q)
    check(both[:, :2], want, tol, "prefill")
    assert bool(both[:, 2:].isnan().all())
    one = c.decode_attention(0, [0], q[1:])
    check(one[:, :2], want[1:], tol[1:], "decode")
    assert bool(one[:, 2:].isnan().all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,r", [(64, 3), (128, 4)])
@pytest.mark.parametrize("n,m", [(110, 60), (110, 1), (4090, 45), (4090, 1)])
def test_non_finite_value_of_an_exact_token(dtype, dim, r, n, m):
    """An infinity or NaN in V of an exact token reaches its own channel, of the queries that see it, and nothing else,
    in both kernels and where work is cut between thread blocks (long sequences)."""
    dt = TYPES[dtype]
    k, v, q = (tokens(t, h, dim, dt, s, 0.3) for t, h, s in ((n, 1, 211), (n, 1, 212), (m, r, 213)))
    bad = {(n - 40, 3): float("inf"), (n - 30, 9): float("-inf"), (n - 25, 3): float("inf"), (n - 20, 12): float("nan")}
    first = {}  # channel: first position
    for (t, ch), x in bad.items():
        v[t, 0, ch] = x
        first[ch] = min(t, first.get(ch, n))
    block = 64
    assert n - 40 >= n // block * block
    c = make(num_q_heads=r, num_kv_heads=1, head_dim=dim, block_tokens=block, dtype=dt, max_seqs=1)
    c.append(0, [0], [n], k, v)
    out = c.prefill_attention(0, [0], [m], q).cpu()
    clean = v.clone()
    for t, ch in bad:
        clean[t, 0, ch] = 0
    want, tol = block_ref.attend(q.cpu(), held(k, block), held(clean, block), dim ** -0.5, list(range(n - m, n)))
    pos = torch.arange(n - m, n)
    for ch, t in first.items():
        sees = pos >= t
        assert bool((~torch.isfinite(out[sees][..., ch])).all()), ch
        out[..., ch][sees] = 0
        want[..., ch][sees] = 0
    check(out, want, tol, (n, m))


TINY, HUGE = 2.0 ** -100, 2.0 ** 126


def _one_size(n, dim, size, seed):
    """Values of random sign, size to 1.98 times it."""
    g = torch.Generator().manual_seed(seed)
    x = (1 + torch.randint(0, 126, (n, 1, dim), generator=g) / 128.0) * size
    return (x * (torch.randint(0, 2, (n, 1, dim), generator=g) * 2 - 1)).to(torch.bfloat16).cuda()


# (tokens, size) of stretches of V. A block's e4m3 scale is 2^-8 of its size, an int8 one 2^-6, and 2^-100 at least.
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("parts", [
    [(32, TINY)],                                 # 32 exact tokens of 2^-100
    [(64, 2.0 ** -10), (32, TINY)],               # beside larger sealed ones
    [(64, 2.0 ** -9), (63, 2.0 ** -92)],
    [(16384, 2.0 ** -92)],                        # many sealed ones of the smallest scale
    [(16384, 2.0 ** -92), (64, 1.0), (7, TINY)],
    [(300, HUGE)],                                # the other end
    [(64, HUGE), (64, 2.0 ** 40), (50, 2.0 ** 40)],
], ids=str)
def test_values_at_the_ends_of_bf16(parts, code):
    """V at the ends of bf16's range, all tokens weighted alike and not: the denominator stays in fp32's range."""
    dim, n = 64, sum(m for m, _ in parts)
    v = torch.cat([_one_size(m, dim, size, i) for i, (m, size) in enumerate(parts)])
    k = tokens(n, 1, dim, torch.bfloat16, 221, 0.3)
    m = min(n, 40)
    q = tokens(m, 2, dim, torch.bfloat16, 222, 0.3)
    q[:, 0] = 0  # all tokens alike
    c = make(num_q_heads=2, num_kv_heads=1, head_dim=dim, block_tokens=64, dtype=torch.bfloat16, max_seqs=1, code=code,
             max_seq_len=n)
    c.append(0, [0], [n], k, v)
    kk, vv = (held(x, 64, code) for x in (k, v))
    want, tol = block_ref.attend(q.cpu(), kk, vv, dim ** -0.5, list(range(n - m, n)))
    check(c.decode_attention(0, [0], q[m - 1:]), want[m - 1:], tol[m - 1:], "decode")
    check(c.prefill_attention(0, [0], [m], q), want, tol, "prefill")


def _words(c, at, n):
    """int32 words of the cache's device block from byte `at` on: the error word stands first, the counters behind
    the block table."""
    off = -c.mem.data_ptr() % 256 + at
    return c.mem[off:off + 4 * n].view(torch.int32)


def _round(n):
    return (n + 255) // 256 * 256


def _counters_at(c):
    g = c.cfg
    return 256 + _round(g.max_seqs * g.num_layers * max(1, g.max_seq_len // g.block_tokens) * 4)


def test_a_reported_error_is_cleared_with_the_counters():
    """What a launch in which a wait gave up leaves behind (error word, counters), written here by hand."""
    c = make(max_seqs=2, block_tokens=32)
    fill(c, [3000, 700], torch.float16, 231)
    q = tokens(600, 8, 128, torch.float16, 233, 0.3)
    want = c.decode_attention(0, [0, 1], q[:2]), c.prefill_attention(0, [0, 1], [400, 200], q)
    assert not _words(c, _counters_at(c), 256).any()  # zero between calls
    for word, status in ((1, 6), (2, 5)):
        _words(c, 0, 1).fill_(word)
        _words(c, _counters_at(c), 256).fill_(3)
        assert c.check_device_error() == status
        assert c.check_device_error() == 0
        assert not _words(c, 0, 4).any() and not _words(c, _counters_at(c), 256).any()
        got = c.decode_attention(0, [0, 1], q[:2]), c.prefill_attention(0, [0, 1], [400, 200], q)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert c.check_device_error() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype,code", [("fp16", "e4m3"), ("bf16", "int8")])
def test_decode_after_a_wait_has_given_up(dtype, code, dim):
    """With the timeout bit of the error word set, as by a wait of a launch before, every wait that would have to wait
    gives up: the call ends at once, says so, and the next one after the check is right."""
    dt = TYPES[dtype]
    c = make(max_seqs=3, num_q_heads=16, head_dim=dim, block_tokens=128, dtype=dt, code=code)
    fill(c, [4000, 127, 700], dt, 241)
    q = tokens(3, 16, dim, dt, 243, 0.3)
    want = c.decode_attention(0, [0, 1, 2], q)
    for _ in range(10):
        _words(c, 0, 1).fill_(1)
        c.decode_attention(0, [0, 1, 2], q)
        c.decode_attention(0, [0, 1, 2], q)
        assert c.check_device_error() == 6
        assert torch.equal(c.decode_attention(0, [0, 1, 2], q), want)
        assert c.check_device_error() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,qlens", [([4000, 300], [40, 300]), ([2000, 1500], [2000, 1500])])
def test_prefill_after_a_wait_has_given_up(lens, qlens, dim):
    """The same for prefill, with its work cut between thread blocks and in whole segments."""
    c = make(max_seqs=2, num_q_heads=32, num_kv_heads=8, head_dim=dim, block_tokens=32)
    fill(c, lens, torch.float16, 251)
    q = tokens(sum(qlens), 32, dim, torch.float16, 253, 0.3)
    want = c.prefill_attention(0, [0, 1], qlens, q)
    for _ in range(5):
        _words(c, 0, 1).fill_(1)
        c.prefill_attention(0, [0, 1], qlens, q)
        c.prefill_attention(0, [0, 1], qlens, q)
        assert c.check_device_error() == 6
        assert torch.equal(c.prefill_attention(0, [0, 1], qlens, q), want)
        assert c.check_device_error() == 0


@pytest.mark.parametrize("hkv,r", [(8, 1), (2, 8), (3, 5)])
@pytest.mark.parametrize("lens,qlens", [([4000, 300], [40, 300]), ([2500, 2400], [2500, 2400]), ([20, 0], [20, 0])])
def test_output_over_the_queries(lens, qlens, hkv, r):
    """out = q: the same bits as into a tensor of its own; an output that overlaps the queries otherwise is refused."""
    from quantized_kv_cache_seal_gb300.kvarn import KVarNError
    c = make(max_seqs=2, num_q_heads=hkv * r, num_kv_heads=hkv, block_tokens=32)
    fill(c, lens, torch.float16, 261)
    big = tokens(sum(qlens) + 4, hkv * r, 128, torch.float16, 263, 0.3)
    q, keep = big[:sum(qlens)], big.clone()
    want = c.prefill_attention(0, [0, 1], qlens, q), c.decode_attention(0, [0, 1], q[:2])
    for call in (lambda out: c.prefill_attention(0, [0, 1], qlens, q, out=out),
                 lambda out: c.prefill_attention(0, [0], [2], q[:2], out=out),
                 lambda out: c.decode_attention(0, [0, 1], q[:2], out=out)):
        rows = sum(qlens) if call(None).shape[0] > 2 else 2
        for at in (1, 3):
            if at < rows:
                with pytest.raises(KVarNError):
                    call(big[at:at + rows])
    assert torch.equal(big, keep)
    assert torch.equal(c.decode_attention(0, [0, 1], q[:2], out=q[:2]), want[1])
    big.copy_(keep)
    assert c.prefill_attention(0, [0, 1], qlens, q, out=q) is q
    assert torch.equal(q, want[0])
    assert torch.equal(big[sum(qlens):], keep[sum(qlens):])


def _two_pi(bits):
    """2 pi * 2^bits, by Machin's formula in integers."""
    def atan_inverse(x):
        t = (1 << bits + 32) // x
        total, k = t, 1
        while t:
            t //= -x * x
            k += 2
            total += t // k
        return total
    return 8 * (4 * atan_inverse(5) - atan_inverse(239)) >> 32


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [32, 64])
def test_norm_rope_large_frequencies_at_far_positions(interleaved, dim):
    """Angles of many turns, against whole-number arithmetic: the fraction of a turn is right at any position."""
    import math
    from fractions import Fraction
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    freqs = [1.0, -3.999999, 4.0, 4.000001, 6.283185307179586, 7.7, -12345.678, 1048577.0, 1e9, -987654321.125, 2.0 ** 33 + 0.25,
             1e13, 2.0 ** 53 - 1, -2.0 ** 60 * 1.1, 2.0 ** 63 * 1.7, 0.001]
    positions = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1234567891, -987654321, 131071, 2 ** 30]
    x = torch.zeros(len(positions), 2, dim, dtype=torch.float16, device="cuda")
    a, b = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    x[..., a] = 1  # (1, 0) turns to (cos, sin)
    y, _ = qk_norm_rope(x, None, torch.tensor(positions, dtype=torch.int32, device="cuda"),
                        torch.tensor(freqs, dtype=torch.float64, device="cuda"), interleaved=interleaved)
    y = y.cpu().double()
    circle = _two_pi(400)
    for t, p in enumerate(positions):
        for i, f in enumerate(freqs):
            turn = Fraction(f) * p * (1 << 400) / circle
            phi = float(turn - math.floor(turn)) * 2 * math.pi
            for got, want in zip((y[t, 1, a][i], y[t, 1, b][i]), (math.cos(phi), math.sin(phi))):
                # the angle to 2^-29 and fp32 (2^-22 with sincospi's 2 ulp), fp16's rounding
                assert abs(float(got) - want) <= 2.0 ** -22 + 2.0 ** -11 * abs(want) + 2.0 ** -25, (p, f)


def test_a_stream_that_a_call_names_holds_its_tensors():
    """What the caller drops after a call on another stream is not handed out again before that stream is through."""
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    c = make(max_seqs=1, block_tokens=32)
    c.append(0, [0], [100], *(tokens(100, 2, 128, torch.float16, s) for s in (271, 272)))
    base = [tokens(500, h, 128, torch.float16, s) for h, s in ((2, 273), (2, 274), (8, 275))]
    pos = torch.arange(500, dtype=torch.int32, device="cuda")
    freqs = torch.rand(64, dtype=torch.float64, device="cuda")
    other = make(max_seqs=1, block_tokens=32)
    other.append(0, [0], [100], *(tokens(100, 2, 128, torch.float16, s) for s in (271, 272)))
    want = other.prefill(0, [0], [500], *base), qk_norm_rope(base[2], base[0], pos, freqs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def dropped(call, tensors):
        at = {t.data_ptr(): t.nbytes for t in tensors}
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)  # some 50 ms
        got = call(*tensors)
        tensors.clear()
        again = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in at.values() for _ in range(3)]
        assert not {t.data_ptr() for t in again} & set(at)
        side.synchronize()
        return got

    got = dropped(lambda k, v, q: c.prefill(0, [0], [500], k, v, q, stream=side), [x.clone() for x in base])
    assert torch.equal(got, want[0])
    got = dropped(lambda q, k, p, f: qk_norm_rope(q, k, p, f, stream=side), [base[2].clone(), base[0].clone(), pos.clone(),
                                                                          freqs.clone()])
    assert torch.equal(got[0], want[1][0]) and torch.equal(got[1], want[1][1])


@pytest.mark.parametrize("named", [False, True])
def test_the_streams_of_its_calls_hold_the_cache(named):
    c = make(max_seqs=1, block_tokens=32)
    c.append(0, [0], [100], *(tokens(100, 2, 128, torch.float16, s) for s in (281, 282)))
    q = tokens(1, 8, 128, torch.float16, 283)
    want = c.decode_attention(0, [0], q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        got = c.decode_attention(0, [0], q) if not named else None
    if named:
        got = c.decode_attention(0, [0], q, stream=side)
    at, n = c.mem.data_ptr(), c.mem.nbytes
    del c
    again = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert at not in {t.data_ptr() for t in again}
    side.synchronize()
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------------- the many-query kernel by itself
def test_prefill_with_scales_of_very_different_size():
    """V blocks whose scales differ by 2^20 and logits that favour the small one, for several queries of a sequence."""
    c = make(num_q_heads=2, num_kv_heads=1, block_tokens=32, max_seqs=1)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(98, 1, 128, generator=g) for _ in range(2))
    q = torch.randn(1, 2, 128, generator=g).expand(3, 2, 128).contiguous()
    k[32:64] = q[0, :1] * 2.0  # these tokens take all the weight
    v[:32] *= 1000.0
    v[32:64] *= 2.0 ** -10
    k, v, q = (x.half().cuda() for x in (k, v, q))
    c.append(0, [0], [98], k, v)
    want, tol = block_ref.attend(q.cpu(), held(k, 32), held(v, 32), 128 ** -0.5, [95, 96, 97])
    check(c.prefill_attention(0, [0], [3], q), want, tol, "scales")


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prefill_keeps_heads_and_unwritten_memory_apart(code, dtype):
    """A NaN in one KV head shows in its query heads only; rows and channels never written show nowhere."""
    dt = TYPES[dtype]
    c = make(block_tokens=32, code=code, dtype=dt)
    c.mem.fill_(0xff)  # whatever was there before the cache
    lens, m = [45, 45, 50], [2, 3, 4]
    k, v = (tokens(140, 2, 128, dt, s, 0.3) for s in (290, 291))
    q = tokens(9, 8, 128, dt, 292, 0.3)
    c.append(0, [0, 1, 2], lens, k, v)
    out, at = c.prefill_attention(0, [0, 1, 2], m, q), 0
    for s, (x, y) in enumerate(zip(k.split(lens), v.split(lens))):
        want, tol = block_ref.attend(q[at:at + m[s]].cpu(), held(x, 32, code), held(y, 32, code), 128 ** -0.5,
                                     list(range(lens[s] - m[s], lens[s])))
        check(out[at:at + m[s]], want, tol, s)
        at += m[s]
    clean = out
    c.release([0, 1, 2])
    v[10, 1, 5] = float("nan")       # sequence 0, sealed block
    v[45 + 44, 0, 7] = float("nan")  # sequence 1, its last token
    k[90 + 48, 1, 0] = float("nan")  # sequence 2, its last but one
    c.append(0, [0, 1, 2], lens, k, v)
    out = c.prefill_attention(0, [0, 1, 2], m, q)
    assert torch.equal(out[:2, :4], clean[:2, :4]) and bool(out[:2, 4:].isnan().all())
    rest = [i for i in range(128) if i != 7]
    assert torch.equal(out[2:4], clean[2:4]) and torch.equal(out[4, 4:], clean[4, 4:])
    assert bool(out[4, :4, 7].isnan().all()) and torch.equal(out[4, :4][:, rest], clean[4, :4][:, rest])
    assert torch.equal(out[5:, :4], clean[5:, :4]) and torch.equal(out[5:7], clean[5:7]) and bool(out[7:, 4:].isnan().all())


@pytest.mark.parametrize("dtype,code,dim", [("fp16", "int8", 64), ("bf16", "e4m3", 128)])
def test_layers_and_scattered_blocks(dtype, code, dim):
    """Attention and read on other layers than the first, where appends to several sequences and layers in turn, with
    releases between, have scattered each sequence's blocks over the pool."""
    dt, layers, seqs = TYPES[dtype], 3, 3
    c = make(num_layers=layers, max_seqs=seqs, head_dim=dim, block_tokens=32, dtype=dt, code=code, max_seq_len=700,
             pool_blocks=130)
    g = torch.Generator().manual_seed(5)
    kept = {}
    for turn in range(45):
        layer, s = (int(torch.randint(0, n, (1,), generator=g)) for n in (layers, seqs))
        if turn % 15 == 14 and turn < 40:
            c.release(s)
            kept = {at: x for at, x in kept.items() if at[1] != s}
        n = int(torch.randint(1, 90, (1,), generator=g))
        x = [tokens(n, 2, dim, dt, 300 + 2 * turn + i, 0.3) for i in (0, 1)]
        if c.length(layer, s) + n > 700:
            continue
        c.append(layer, [s], [n], *x)
        kept[layer, s] = [torch.cat(p) for p in zip(kept[layer, s], x)] if (layer, s) in kept else x
    q = tokens(90, 8, dim, dt, 400, 0.3)
    assert sum(layer > 0 for layer, _ in kept) >= 4
    for layer in range(layers):
        ids = [s for s in range(seqs) if (layer, s) in kept]
        lens = [kept[layer, s][0].shape[0] for s in ids]
        assert lens == [c.length(layer, s) for s in ids]
        refs = [[held(x, 32, code) for x in kept[layer, s]] for s in ids]
        m = [min(n, 30) for n in lens]
        many, one, at = c.prefill_attention(layer, ids, m, q[:sum(m)]), c.decode_attention(layer, ids, q[:len(ids)]), 0
        back = c.read(layer, ids, None, lens, dtype=torch.float32)
        for i, (n, ref) in enumerate(zip(lens, refs)):
            want, tol = block_ref.attend(q[at:at + m[i]].cpu(), *ref, dim ** -0.5, list(range(n - m[i], n)))
            check(many[at:at + m[i]], want, tol, (layer, i))
            want, tol = block_ref.attend(q[i:i + 1].cpu(), *ref, dim ** -0.5, [n - 1])
            check(one[i:i + 1], want, tol, (layer, i))
            for x, y in zip(back, ref):
                assert torch.equal(x[sum(lens[:i]):sum(lens[:i + 1])].cpu(), y.float())
            at += m[i]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_queries_whose_every_logit_is_minus_infinity(dtype):
    """Zeros, as for an empty sequence; the other heads of the token are as without."""
    dt = TYPES[dtype]
    k, v, q = (tokens(m, h, 128, dt, s, 0.3) for m, h, s in ((20, 1, 501), (20, 1, 502), (3, 2, 503)))
    k[:, 0, 5] = float("inf")
    q[:, :, 5] = torch.tensor([-1.0, 0.5], dtype=dt).cuda()
    c = make(num_q_heads=2, num_kv_heads=1, dtype=dt, max_seqs=1)
    c.append(0, [0], [20], k, v)
    for out in (c.decode_attention(0, [0], q[2:]), c.prefill_attention(0, [0], [3], q)):
        assert not out[:, 0].any() and bool(out[:, 1].isnan().all())
