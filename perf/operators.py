"""Workloads of the query/key norm + rotation and of the 8-bit block cache (append, read, decode and prefill
attention): for each case its inputs, one pass in plain torch operations, one pass through the library, and
the operator's definition in 64 bits.

The cache holds K and V in blocks of ``block`` tokens. A full block is held as 8-bit codes with one scale per
(block, KV head, K or V); the last, partial block is exact. Codes: ``e4m3`` with the smallest power-of-two scale that
fits, or ``int8`` with scale amax / 127; scales are 2^-100 at least, and 1 where all values are zero.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step's queries and keys: Llama-3.1-8B heads, batch 16, far positions; latency counts
        dict(name="norm_rope step b16", op="norm_rope", tokens=16, hq=32, hkv=8, dim=128, rot=128, norm=True,
             interleaved=False, packed=False, dtype="fp16", out="fp16", far=131072),
        # a 4096-token prompt of Qwen3-4B heads (with head norms), bf16 projections written as fp16 for the cache
        dict(name="norm_rope prompt 4096", op="norm_rope", tokens=4096, hq=32, hkv=8, dim=128, rot=128, norm=True,
             interleaved=False, packed=True, dtype="bf16", out="fp16", far=4096),
        # a large batch of prompts, Phi-4-14B heads, no norm, read from the packed projection; odd token count
        dict(name="norm_rope packed 49157", op="norm_rope", tokens=49157, hq=40, hkv=10, dim=128, rot=128, norm=False,
             interleaved=False, packed=True, dtype="bf16", out="bf16", far=16384),
        # short prompts of odd lengths written and read back; latency counts
        dict(name="write_read short b3", op="write_read", batch=3, low=33, high=300, hkv=8, dim=128, block=64,
             code="e4m3", dtype="fp16", shape_seed=1),
        # one 4096-token prompt of Qwen3-4B heads, int8
        dict(name="write_read prompt 4096", op="write_read", batch=1, low=4096, high=4096, hkv=8, dim=128, block=64,
             code="int8", dtype="fp16", shape_seed=2),
        # the ragged batch: 64 sequences of 1k..16k tokens, Phi-4-14B heads
        dict(name="write_read ragged b64", op="write_read", batch=64, low=1024, high=16384, hkv=10, dim=128, block=128,
             code="e4m3", dtype="bf16", shape_seed=3),
        # a single sequence at 4096 tokens, Qwen3-4B heads: the smallest decode call
        dict(name="decode b1 4k", op="decode", batch=1, low=4096, high=4096, hq=32, hkv=8, dim=128, block=64,
             code="e4m3", dtype="fp16", shape_seed=4),
        # the headline decode: Llama-3.1-8B heads, batch 16, 32k context with ragged tails
        dict(name="decode b16 32k", op="decode", batch=16, low=32768, high=32895, hq=32, hkv=8, dim=128, block=64,
             code="e4m3", dtype="fp16", shape_seed=5),
        # the ragged batch: 64 sequences of 1k..16k tokens, Phi-4-14B heads, int8, bf16 queries
        dict(name="decode ragged b64", op="decode", batch=64, low=1024, high=16384, hq=40, hkv=10, dim=128, block=32,
             code="int8", dtype="bf16", shape_seed=6),
        # a whole 4096-token prompt attended causally, Qwen3-4B heads
        dict(name="prefill prompt 4096", op="prefill", batch=1, low=4096, high=4096, qlow=4096, qhigh=4096, hq=32, hkv=8,
             dim=128, block=64, code="e4m3", dtype="fp16", shape_seed=7),
        # a 512-token chunk against 32k cached tokens: few query rows, a long axis
        dict(name="prefill chunk 512 of 32k", op="prefill", batch=1, low=32768, high=32768, qlow=512, qhigh=512, hq=32,
             hkv=8, dim=128, block=128, code="e4m3", dtype="fp16", shape_seed=8),
        # ragged chunks of several sequences, odd lengths, int8 cache of a bf16 model
        dict(name="prefill ragged b6", op="prefill", batch=6, low=700, high=6000, qlow=1, qhigh=700, hq=40, hkv=10,
             dim=128, block=32, code="int8", dtype="bf16", shape_seed=9),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "write_read", "decode", "prefill"])
    dtype = rng.choice(["fp16", "bf16"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 10])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "norm_rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        tokens = _log(rng, 1, min(65536, 300_000_000 // ((hq + hkv) * dim)))
        return dict(op=op, tokens=tokens, hq=hq, hkv=hkv, dim=dim, rot=dim if rng.random() < 0.6 else dim // 16 * 8,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.3, packed=rng.random() < 0.5, dtype=dtype,
                    out=rng.choice(["fp16", "bf16"]) if dtype == "bf16" else "fp16", far=_log(rng, tokens, 262144))
    case = dict(op=op, batch=_log(rng, 1, 64), hkv=hkv, dim=rng.choice([64, 128, 128]), block=rng.choice([32, 64, 128]),
                code=rng.choice(["e4m3", "int8"]), dtype=dtype, shape_seed=rng.randrange(1 << 30))
    if op == "write_read":
        most = min(32768, 500_000_000 // (case["batch"] * hkv * case["dim"]))
        high = _log(rng, 1, most)
        return dict(case, low=_log(rng, 1, high), high=high)
    case["hq"] = hq
    if op == "decode":
        most = min(65536, 500_000_000 // (case["batch"] * hkv * case["dim"]))
        high = _log(rng, 1, most)
        return dict(case, low=_log(rng, 1, high), high=high)
    case["batch"] = _log(rng, 1, 8)
    qhigh = _log(rng, 1, 2048)
    # scores of the padded batch: at most the 4096-token prompt's
    most = max(qhigh, min(32768, 500_000_000 // (case["batch"] * hq * qhigh)))
    high = _log(rng, qhigh, most)
    return dict(case, low=_log(rng, qhigh, high), high=high, qlow=_log(rng, 1, qhigh), qhigh=qhigh)


def _lengths(case):
    """Tokens of each sequence, and queries of each for prefill: part of the case's shape, not of the seed."""
    rng = random.Random(case["shape_seed"])
    lens = [rng.randint(case["low"], case["high"]) for _ in range(case["batch"])]
    if case["op"] != "prefill":
        return lens, None
    return lens, [min(n, rng.randint(case["qlow"], case["qhigh"])) for n in lens]


def work(case):
    if case["op"] == "norm_rope":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 8 * n}
    lens, qlens = _lengths(case)
    d, hkv, b = case["dim"], case["hkv"], case["block"]
    full = sum(n // b * b for n in lens)
    rest = sum(lens) - full
    held = 2 * hkv * (full * d + full // b * 4 + rest * d * 2)  # the cache: codes, scales, exact rows
    if case["op"] == "write_read":
        # tokens in, cache out; cache in, tokens out
        return {"bytes": 2 * held + 2 * (2 * sum(lens) * hkv * d * 2), "flops": 4 * 2 * sum(lens) * hkv * d}
    hq = case["hq"]
    if case["op"] == "decode":
        return {"bytes": held + 2 * len(lens) * hq * d * 2, "flops": 4 * sum(lens) * hq * d}
    pairs = sum(q * n - q * (q - 1) // 2 for n, q in zip(lens, qlens))  # visible (query, key) pairs of a head
    return {"bytes": held + 2 * sum(qlens) * hq * d * 2, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)


def _tokens(g, n, hkv, dim, dtype):
    """K and V rows [n][hkv][dim] as a model makes them: scales by channel with outlier channels, norms by token."""
    chan = torch.empty((2, hkv, dim), device="cuda").log_normal_(0.0, 0.5, generator=g)
    chan[:, :, :2] *= 20.0
    chan /= 4.0
    norm = torch.empty((n, 1, 1), device="cuda").log_normal_(0.0, 0.7, generator=g)
    return [torch.randn((n, hkv, dim), device="cuda", generator=g).mul_(chan[i]).mul_(norm).clamp_(-6e4, 6e4).to(dtype)
            for i in (0, 1)]


def _starts(lens):
    return [sum(lens[:i]) for i in range(len(lens))]


def _padded(x, lens, width):
    """Rows of the sequences, back to back in x, as [batch][width][heads][dim], zeros behind each."""
    y = torch.zeros((len(lens), width) + x.shape[1:], dtype=x.dtype, device=x.device)
    at = 0
    for i, n in enumerate(lens):
        y[i, :n] = x[at:at + n]
        at += n
    return y


def _quantised(x, case):
    """Codes and scales of whole blocks, x: [batch][n][heads][dim] (n a multiple of the block)."""
    b, n, h, d = x.shape
    x = x.view(b, n // case["block"], case["block"], h, d)
    amax = x.abs().amax(dim=(2, 4)).float()
    if case["code"] == "e4m3":
        m, e = torch.frexp(amax)
        # the power of two from its bits: pow() is not exact
        scale = ((torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-100) + 127) << 23).view(torch.float32)
        scale = torch.where(amax == 0, torch.ones_like(scale), scale)
        codes = (x.float() / scale[:, :, None, :, None]).to(torch.float8_e4m3fn)
    else:
        scale = torch.where(amax == 0, torch.ones_like(amax), (amax / 127).clamp(min=2.0 ** -100))
        # in 64 bits: a quotient next to the middle of two codes
        codes = (x.double() / scale[:, :, None, :, None].double()).round_().clamp_(-127, 127).to(torch.int8)
    return codes, scale  # [batch][blocks][block][heads][dim], [batch][blocks][heads]


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "norm_rope":
        t, hq, hkv, d, rot = (case[k] for k in ("tokens", "hq", "hkv", "dim", "rot"))
        if case["packed"]:  # q and k are parts of the projection's rows, before v
            qkv = torch.randn((t, hq + 2 * hkv, d), device="cuda", generator=g).to(dtype)
            q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            q = torch.randn((t, hq, d), device="cuda", generator=g).to(dtype)
            k = torch.randn((t, hkv, d), device="cuda", generator=g).to(dtype)
        weights = [torch.empty(d, device="cuda").log_normal_(0.0, 0.3, generator=g) if case["norm"] else None
                   for _ in (0, 1)]
        freqs = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        if case["far"] > t:
            pos = torch.randint(0, case["far"], (t,), device="cuda", generator=g, dtype=torch.int32)
        else:
            pos = torch.arange(t, device="cuda", dtype=torch.int32) % case["far"]
        return dict(case=case, q=q, k=k, weights=weights, freqs=freqs, pos=pos, eps=1e-6, out=DTYPES[case["out"]])
    lens, qlens = _lengths(case)
    k, v = _tokens(g, sum(lens), case["hkv"], case["dim"], dtype)
    state = dict(case=case, lens=lens, ids=list(range(len(lens))), qlens=qlens)
    if "hq" in case:
        rows = sum(qlens) if qlens else len(lens)
        state["q"] = torch.randn((rows, case["hq"], case["dim"]), device="cuda", generator=g).to(dtype)
        state["scale"] = case["dim"] ** -0.5
    if own:  # the cache that a program keeps; for attention, with the tokens in it
        from quantized_kv_cache_seal_gb300.block_cache import BlockCache
        cache = BlockCache(num_layers=1, max_seqs=len(lens), num_q_heads=case.get("hq", case["hkv"]),
                        num_kv_heads=case["hkv"], head_dim=case["dim"], block_tokens=case["block"], code=case["code"],
                        dtype=dtype, max_seq_len=max(lens), pool_blocks=sum(n // case["block"] for n in lens))
        if case["op"] == "write_read":
            return dict(state, cache=cache, k=k, v=v)
        cache.append(0, state["ids"], lens, k, v)
        return dict(state, cache=cache)
    block = case["block"]
    width = -(-max(lens) // block) * block
    state["lengths"] = torch.tensor(lens, device="cuda")
    state["full"] = state["lengths"] // block * block
    # where each token stands in the padded batch, and each padded place's token
    start = torch.tensor(_starts(lens), device="cuda")
    state["batch_of"] = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), state["lengths"])
    state["place_of"] = torch.arange(sum(lens), device="cuda") - start[state["batch_of"]]
    if case["op"] == "write_read":
        return dict(state, k=k, v=v, width=width)
    for name, x in (("k", k), ("v", v)):
        x = _padded(x, lens, width)
        state[name + "_codes"], state[name + "_scale"] = _quantised(x, case)
        at = (state["full"][:, None] + torch.arange(block, device="cuda")).clamp_(max=width - 1)
        state[name + "_tail"] = x[torch.arange(len(lens), device="cuda")[:, None], at]  # [batch][block][heads][dim]
    if qlens:
        most = max(qlens)
        qstart = torch.tensor(_starts(qlens), device="cuda")
        q_lengths = torch.tensor(qlens, device="cuda")
        t = torch.arange(most, device="cuda")
        state["q_rows"] = torch.minimum(qstart[:, None] + t, (qstart + q_lengths - 1)[:, None])  # [batch][most]
        state["q_pos"] = state["lengths"][:, None] - q_lengths[:, None] + t
        state["q_batch"] = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), q_lengths)
        state["q_place"] = torch.arange(sum(qlens), device="cuda") - qstart[state["q_batch"]]
    return state


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"norm_rope": _norm_rope, "write_read": _write_read, "decode": _decode, "prefill": _prefill}[
        state["case"]["op"]](state)


def _run_own(state):
    case = state["case"]
    if case["op"] == "norm_rope":
        from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
        return qk_norm_rope(state["q"], state["k"], state["pos"], state["freqs"], q_weight=state["weights"][0],
                            k_weight=state["weights"][1], eps=state["eps"], interleaved=case["interleaved"],
                            dtype=state["out"])
    cache = state["cache"]
    if case["op"] == "write_read":
        cache.release(state["ids"])
        cache.append(0, state["ids"], state["lens"], state["k"], state["v"])
        return cache.read(0, state["ids"], None, state["lens"])
    if case["op"] == "decode":
        return cache.decode_attention(0, state["ids"], state["q"], scale=state["scale"])
    return cache.prefill_attention(0, state["ids"], state["qlens"], state["q"], scale=state["scale"])


def _rotated(x, weight, cos, sin, interleaved, eps, dtype):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * weight
    half = cos.shape[-1]
    a, b, rest = (y[..., 0:2 * half:2], y[..., 1:2 * half:2], y[..., 2 * half:]) if interleaved else (
        y[..., :half], y[..., half:2 * half], y[..., 2 * half:])
    c, s = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((c, s), -1).flatten(-2) if interleaved else torch.cat((c, s), -1)
    return torch.cat((turned, rest), -1).to(dtype)


def _norm_rope(state):
    angle = state["pos"].double()[:, None, None] * state["freqs"]  # 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    return tuple(_rotated(x, w, cos, sin, state["case"]["interleaved"], state["eps"], state["out"])
                 for x, w in ((state["q"], state["weights"][0]), (state["k"], state["weights"][1])))


def _write_read(state):
    out = []
    case, lengths = state["case"], state["lengths"]
    for x in (state["k"], state["v"]):
        y = torch.zeros((len(state["lens"]), state["width"]) + x.shape[1:], dtype=x.dtype, device=x.device)
        y[state["batch_of"], state["place_of"]] = x
        codes, scale = _quantised(y, case)
        values = (codes.float() * scale[:, :, None, :, None]).flatten(1, 2)
        values = values[state["batch_of"], state["place_of"]]
        exact = state["place_of"] >= state["full"][state["batch_of"]]
        most = torch.finfo(x.dtype).max
        out.append(torch.where(exact[:, None, None], x.float(), values.clamp(-most, most)).to(x.dtype))
    return tuple(out)


def _held(state, name):
    """The cached values in 32 bits, [batch][n][heads][dim]: dequantised blocks, then the exact rows."""
    values = (state[name + "_codes"].float() * state[name + "_scale"][:, :, None, :, None]).flatten(1, 2)
    n = torch.arange(values.shape[1], device=values.device)
    exact = n[None] >= state["full"][:, None]
    tail = state[name + "_tail"].float()
    at = (n[None] - state["full"][:, None]).clamp(0, tail.shape[1] - 1)
    picked = tail[torch.arange(len(at), device=at.device)[:, None], at]
    return torch.where(exact[:, :, None, None], picked, values)


def _attended(q, k, v, seen, scale):
    """q: [batch][kv heads][rows][dim]; k, v: [batch][n][kv heads][dim]; seen: broadcast over [batch][kv heads][rows][n]."""
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * scale
    s = torch.where(seen, s, float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return torch.matmul(p / p.sum(-1, keepdim=True), v.permute(0, 2, 1, 3))


def _decode(state):
    q = state["q"]
    k, v = _held(state, "k"), _held(state, "v")
    seen = torch.arange(k.shape[1], device=q.device)[None] < state["lengths"][:, None]
    o = _attended(q.float().view(q.shape[0], k.shape[2], -1, q.shape[2]), k, v, seen[:, None, None], state["scale"])
    return o.reshape(q.shape).to(q.dtype)


def _prefill(state):
    q = state["q"]
    k, v = _held(state, "k"), _held(state, "v")
    x = q.float()[state["q_rows"]]  # [batch][most][hq][dim]
    b, most, hq, d = x.shape
    hkv = k.shape[2]
    x = x.view(b, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, hq // hkv * most, d)
    seen = torch.arange(k.shape[1], device=q.device)[None, None] <= state["q_pos"][:, :, None]  # [batch][most][n]
    seen = seen[:, None, None].expand(b, 1, hq // hkv, most, k.shape[1]).reshape(b, 1, hq // hkv * most, k.shape[1])
    # padding rows of a shorter sequence see a later position: they are left out below
    o = _attended(x, k, v, seen, state["scale"])
    o = o.view(b, hkv, hq // hkv, most, d).permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)
    return o[state["q_batch"], state["q_place"]].to(q.dtype)


# ---------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _power(e):
    """2^e in 64 bits, from its bits, for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest_even(x, step):
    """Multiples of step (an exact power of two, or 1) nearest to x, ties to even multiples, in 64 bits."""
    low = torch.floor(x / step)
    over = x / step - low
    up = (over > 0.5) | ((over == 0.5) & (low % 2 == 1))
    return (low + up.double()) * step


def _exact_block(x, code):
    """Values that a full block x [block][heads][dim] (64 bits) is held as."""
    top = x.abs().amax(dim=(0, 2), keepdim=True)
    one = torch.ones_like(top)
    if code == "int8":
        scale = torch.where(top == 0, one, (top / 127).float().double().clamp(min=2.0 ** -100))  # held in 32 bits
        return _nearest_even(x / scale, 1.0).clamp(-127, 127) * scale
    exponent = torch.ceil(torch.log2(torch.where(top == 0, 448 * one, top) / 448))
    exponent = torch.where(448 * _power(exponent - 1) >= top, exponent - 1, exponent)  # log2 next to a whole number
    exponent = torch.where(448 * _power(exponent) < top, exponent + 1, exponent)
    scale = torch.where(top == 0, one, _power(exponent.clamp(min=-100)))
    y = (x / scale).abs()
    # e4m3: three bits behind the leading one, down to steps of 2^-9
    lead = torch.floor(torch.log2(torch.where(y == 0, torch.ones_like(y), y)))
    lead = torch.where(_power(lead) > y, lead - 1, lead)
    lead = torch.where(_power(lead + 1) <= y, lead + 1, lead)
    step = _power(lead.clamp(min=-6) - 3)
    return torch.sign(x) * _nearest_even(y, step).clamp(max=448) * scale


def _exact_cache(x, lens, case):
    """What the cache holds for each sequence, a list of [n][heads][dim] in 64 bits."""
    held, at = [], 0
    for n in lens:
        y = x[at:at + n].double()
        b = case["block"]
        done = n // b * b
        step = max(1, (1 << 25) // (b * x.shape[1] * x.shape[2])) * b  # some blocks at a time
        for i in range(0, done, step):
            part = y[i:min(done, i + step)]
            whole = part.view(-1, b, *part.shape[1:]).permute(1, 0, 2, 3)  # [block][blocks][heads][dim]
            flat = whole.reshape(b, -1, whole.shape[-1])
            y[i:i + part.shape[0]] = _exact_block(flat, case["code"]).view(whole.shape).permute(1, 0, 2, 3).reshape(
                part.shape)
        held.append(y)
        at += n
    return held


def exact(case, seed):
    if case["op"] == "norm_rope":
        s = prepare(case, seed)
        out = []
        for x, w in ((s["q"], s["weights"][0]), (s["k"], s["weights"][1])):
            y = x.double()
            if w is not None:
                y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.double()
            turn = torch.exp(1j * (s["pos"].double()[:, None, None] * s["freqs"]))
            half = case["rot"] // 2
            index = torch.arange(half, device=x.device)
            first, second = (2 * index, 2 * index + 1) if case["interleaved"] else (index, index + half)
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
        return tuple(out)
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    lens, qlens = _lengths(case)
    k, v = _tokens(g, sum(lens), case["hkv"], case["dim"], dtype)
    if case["op"] == "write_read":
        most = torch.finfo(dtype).max
        return tuple(torch.cat(_exact_cache(x, lens, case)).clamp_(-most, most) for x in (k, v))
    if work(case)["flops"] > 1.2e12:
        return None  # too long in 64 bits
    rows = sum(qlens) if qlens else len(lens)
    q = torch.randn((rows, case["hq"], case["dim"]), device="cuda", generator=g).to(dtype).double()
    out, at = torch.empty_like(q), 0
    keys, values = _exact_cache(k, lens, case), _exact_cache(v, lens, case)
    for i, n in enumerate(lens):
        m = qlens[i] if qlens else 1
        part = q[at:at + m].view(m, case["hkv"], -1, case["dim"])
        last = torch.arange(n - m, n, device="cuda")
        for h in range(case["hkv"]):
            s = torch.einsum("mrd,nd->mrn", part[:, h], keys[i][:, h]) * case["dim"] ** -0.5
            s.masked_fill_((torch.arange(n, device="cuda")[None] > last[:, None])[:, None], float("-inf"))
            r = case["hq"] // case["hkv"]
            out[at:at + m, h * r:(h + 1) * r] = torch.einsum("mrn,nd->mrd", torch.softmax(s, -1), values[i][:, h])
        at += m
    return out
