"""Workloads of the rotation by several position axes, of attention over prefixes that sequences share, and of eviction
from the block cache by accumulated attention weight: for each case its inputs, one pass in plain torch operations,
one pass through the library, and the operator's definition in 64 bits.

Rotation: pair i of a head turns by positions[axes[i]] * freqs[i] (text has the same position on every axis, an
image's tokens their time, row and column). Shared prefix: a query attends the tokens of its sequence's prefix and those
of the sequence itself under one softmax. Weights: what each block of a sequence has received of the softmax
weights of the queries so far, summed over the query heads of a KV head. Eviction: each KV head keeps the blocks of
most weight, its first and last ones in any case, in their order.

The cache holds full blocks as 8-bit codes with one scale per (block, KV head, K or V), and the last, partial
block exact. Codes: ``e4m3`` with the smallest power-of-two scale that fits, or ``int8`` with scale amax / 127; scales
are 2^-100 at least, and 1 where all values are zero.
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
        # one decode step's queries and keys of a model with three axes, batch 16; latency counts
        dict(name="axes_rope step b16", op="axes_rope", tokens=16, hq=32, hkv=8, dim=128, rot=128, axes=3, mixed=False,
             norm=True, interleaved=False, packed=False, dtype="fp16", out="fp16"),
        # a large batch of prompts with images in them, read from the packed projection; odd token count, axes in turn
        dict(name="axes_rope packed 49157", op="axes_rope", tokens=49157, hq=40, hkv=10, dim=128, rot=128, axes=3,
             mixed=True, norm=True, interleaved=False, packed=True, dtype="bf16", out="bf16"),
        # four answers sampled from one short prompt; latency counts
        dict(name="shared_decode b4 1k", op="shared_decode", groups=1, batch=4, plow=1000, phigh=1000, low=1, high=100,
             hq=32, hkv=8, dim=128, block=64, code="e4m3", dtype="fp16", shape_seed=21),
        # two long documents, 32 ragged conversations about each; Phi-4-14B heads
        dict(name="shared_decode b64 32k", op="shared_decode", groups=2, batch=64, plow=32000, phigh=32768, low=1,
             high=1024, hq=40, hkv=10, dim=128, block=32, code="int8", dtype="bf16", shape_seed=22),
        # eight short questions behind a system prompt, ragged
        dict(name="shared_prefill b8 2k", op="shared_prefill", groups=1, batch=8, plow=2048, phigh=2048, low=17, high=200,
             hq=32, hkv=8, dim=128, block=64, code="e4m3", dtype="fp16", shape_seed=23),
        # four longer questions about one 16k document
        dict(name="shared_prefill b4 16k", op="shared_prefill", groups=1, batch=4, plow=16384, phigh=16384, low=400,
             high=700, hq=32, hkv=8, dim=128, block=128, code="e4m3", dtype="fp16", shape_seed=24),
        # a single sequence's step that also notes the weights: the smallest call
        dict(name="weighed_decode b1 4k", op="weighed_decode", batch=1, low=4096, high=4096, hq=32, hkv=8, dim=128, block=64,
             code="e4m3", dtype="fp16", shape_seed=25),
        # the headline decode (Llama-3.1-8B heads, batch 16, 32k, ragged tails), noting the weights
        dict(name="weighed_decode b16 32k", op="weighed_decode", batch=16, low=32768, high=32895, hq=32, hkv=8, dim=128,
             block=64, code="e4m3", dtype="fp16", shape_seed=26),
        # the last 16 queries of one 4096-token prompt say what it needs (Qwen3-4B heads)
        dict(name="window 16 of 4k", op="window", batch=1, low=4096, high=4096, qlow=16, qhigh=16, hq=32, hkv=8, dim=128,
             block=64, code="int8", dtype="fp16", shape_seed=27),
        # the last 32 queries of 16 ragged prompts, Phi-4-14B heads
        dict(name="window 32 ragged b16", op="window", batch=16, low=1024, high=16384, qlow=32, qhigh=32, hq=40, hkv=10,
             dim=128, block=32, code="e4m3", dtype="bf16", shape_seed=28),
        # short prompts written, cut to a small budget, read back; latency counts
        dict(name="evict short b3", op="evict", batch=3, low=300, high=700, keep=4, first=1, last=1, hkv=8, dim=128, block=64,
             code="e4m3", dtype="fp16", shape_seed=29),
        # 16 ragged prompts written, cut to about 4k tokens each, read back; Phi-4-14B heads
        dict(name="evict ragged b16", op="evict", batch=16, low=1024, high=16384, keep=64, first=1, last=4, hkv=10, dim=128,
             block=64, code="int8", dtype="bf16", shape_seed=30),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["axes_rope", "shared_decode", "shared_prefill", "weighed_decode", "window", "evict"])
    dtype = rng.choice(["fp16", "bf16"])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 10])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "axes_rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        tokens = _log(rng, 1, min(49157, 300_000_000 // ((hq + hkv) * dim)))
        return dict(op=op, tokens=tokens, hq=hq, hkv=hkv, dim=dim, rot=dim if rng.random() < 0.6 else dim // 16 * 8,
                    axes=rng.choice([2, 3, 3, 4]), mixed=rng.random() < 0.5, norm=rng.random() < 0.6,
                    interleaved=rng.random() < 0.3, packed=rng.random() < 0.5, dtype=dtype,
                    out=rng.choice(["fp16", "bf16"]) if dtype == "bf16" else "fp16")
    case = dict(op=op, batch=_log(rng, 1, 64), hkv=hkv, dim=rng.choice([64, 128, 128]), block=rng.choice([32, 64, 128]),
                code=rng.choice(["e4m3", "int8"]), dtype=dtype, shape_seed=rng.randrange(1 << 30))
    width = hkv * case["dim"]
    if op == "evict":
        case["batch"] = _log(rng, 1, 16)
        most = min(16384, 300_000_000 // (case["batch"] * width))
        high = _log(rng, 1, most)
        keep = _log(rng, 1, max(1, high // case["block"]))
        first = rng.randint(0, min(2, keep))
        return dict(case, low=_log(rng, 1, high), high=high, keep=keep, first=first, last=rng.randint(0, min(4, keep - first)))
    case["hq"] = hq
    if op == "weighed_decode":
        most = min(32768, 500_000_000 // (case["batch"] * width))
        high = _log(rng, 1, most)
        return dict(case, low=_log(rng, 1, high), high=high)
    if op == "window":
        case["batch"] = _log(rng, 1, 16)
        qhigh = _log(rng, 1, 64)
        # scores of the padded batch
        most = max(qhigh, min(16384, 350_000_000 // (case["batch"] * hq * qhigh), 300_000_000 // (case["batch"] * width)))
        high = _log(rng, qhigh, most)
        return dict(case, low=_log(rng, qhigh, high), high=high, qlow=_log(rng, 1, qhigh), qhigh=qhigh)
    groups = min(case["batch"], rng.choice([1, 1, 2, 3]))
    if op == "shared_decode":
        high = _log(rng, 1, max(1, min(1024, 80_000_000 // (case["batch"] * width))))
        phigh = _log(rng, 1, min(32768, 80_000_000 // (groups * width)))
    else:
        case["batch"] = _log(rng, 1, 8)
        groups = min(case["batch"], groups)
        high = _log(rng, 1, 700)
        phigh = _log(rng, 1, min(16384, 400_000_000 // (case["batch"] * high * hq)))
    return dict(case, groups=groups, low=_log(rng, 1, high), high=high, plow=_log(rng, 1, phigh), phigh=phigh)


def _lengths(case):
    """Tokens of each sequence, then of each prefix, and queries of each sequence: part of the case's shape, not of
    the seed."""
    rng = random.Random(case["shape_seed"])
    lens = [rng.randint(case["low"], case["high"]) for _ in range(case["batch"])]
    if case["op"] in ("shared_decode", "shared_prefill"):
        prefixes = [rng.randint(case["plow"], case["phigh"]) for _ in range(case["groups"])]
        return lens, prefixes, lens if case["op"] == "shared_prefill" else [1] * len(lens)
    if case["op"] == "window":
        return lens, [], [min(n, rng.randint(case["qlow"], case["qhigh"])) for n in lens]
    return lens, [], [1] * len(lens)


def _group(case):
    """The prefix of each sequence, in order: runs of about the same number of sequences."""
    return [i * case["groups"] // case["batch"] for i in range(case["batch"])]


def _columns(case):
    """Places of a sequence's weights for one KV head: its blocks, the partial one among them."""
    return case["high"] // case["block"] + 1


def work(case):
    if case["op"] == "axes_rope":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * case["dim"]
        return {"bytes": 4 * n + 4 * case["axes"] * case["tokens"], "flops": 8 * n}
    lens, prefixes, qlens = _lengths(case)
    d, hkv, b = case["dim"], case["hkv"], case["block"]

    def held(n):  # codes, scales, exact rows of K and V
        return 2 * hkv * (n // b * b * d + n // b * 4 + n % b * d * 2)

    cache = sum(held(n) for n in lens + prefixes)
    weights = 2 * 4 * hkv * sum(n // b + 1 for n in lens)
    if case["op"] == "evict":
        left = [min(n, case["keep"] * b + n % b) for n in lens]
        # tokens in; the cache that stays, written and read; tokens out; weights and the blocks' numbers
        return {"bytes": 2 * hkv * d * 2 * (sum(lens) + sum(left)) + 2 * sum(held(n) for n in left) + weights
                + 4 * hkv * case["keep"] * len(lens), "flops": 4 * 2 * sum(lens) * hkv * d}
    hq = case["hq"]
    # visible (query, key) pairs of a head: all of the prefix, the sequence's own up to the query
    pairs = sum(q * n - q * (q - 1) // 2 for n, q in zip(lens, qlens))
    if prefixes:
        pairs += sum(q * prefixes[g] for q, g in zip(qlens, _group(case)))
    rows = 2 * sum(qlens) * hq * d
    if case["op"] == "window":  # keys alone; queries in, no rows out
        return {"bytes": cache // 2 + rows + weights, "flops": 2 * pairs * hq * d}
    return {"bytes": cache + 2 * rows + (weights if case["op"] == "weighed_decode" else 0), "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)


def _tokens(g, n, hkv, dim, dtype):
    """K and V rows [n][hkv][dim] as a model makes them: scales by channel with outlier channels, norms by token."""
    chan = torch.empty((2, hkv, dim), device="cuda").log_normal_(0.0, 0.5, generator=g)
    chan[:, :, :2] *= 20.0
    chan /= 4.0
    norm = torch.empty((n, 1, 1), device="cuda").log_normal_(0.0, 0.7, generator=g)
    return [torch.randn((n, hkv, dim), device="cuda", generator=g).mul_(chan[i]).mul_(norm).clamp_(-6e4, 6e4).to(dtype)
            for i in (0, 1)]


def _axis_of(case):
    """The axis of each pair: in sections of about the same length, or in turn."""
    pairs, axes = case["rot"] // 2, case["axes"]
    return tuple(i % axes if case["mixed"] else i * axes // pairs for i in range(pairs))


def _data(case, seed):
    """Tokens of the sequences and then the prefixes, back to back; queries; weights received before this call."""
    g = _generator(seed)
    lens, prefixes, qlens = _lengths(case)
    k, v = _tokens(g, sum(lens) + sum(prefixes), case["hkv"], case["dim"], DTYPES[case["dtype"]])
    q = weights = None
    if "hq" in case:
        q = torch.randn((sum(qlens), case["hq"], case["dim"]), device="cuda", generator=g).to(DTYPES[case["dtype"]])
    if case["op"] in ("weighed_decode", "window", "evict"):
        weights = torch.empty((case["batch"], case["hkv"], _columns(case)), device="cuda").log_normal_(-3.0, 2.0, generator=g)
        blocks = torch.tensor([-(-n // case["block"]) for n in lens], device="cuda")
        weights *= torch.arange(weights.shape[2], device="cuda") < blocks[:, None, None]
    return k, v, q, weights


def _places(lens):
    """Of tokens back to back: their sequence and their place in it."""
    lens = torch.tensor(lens, device="cuda")
    which = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), lens)
    return which, torch.arange(len(which), device="cuda") - (lens.cumsum(0) - lens)[which]


def _padded(x, which, place, count, width):
    """[count][width][heads][dim] of tokens back to back, zeros behind each sequence."""
    y = torch.zeros((count, width) + x.shape[1:], dtype=x.dtype, device=x.device)
    y[which, place] = x
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


def _width(lens, block):
    return (max(lens) // block + 1) * block


def _held_in(x, lens, case):
    """A cache in plain tensors: codes, scales, exact rows and where they begin, of tokens back to back."""
    which, place = _places(lens)
    width = _width(lens, case["block"])
    y = _padded(x, which, place, len(lens), width)
    codes, scale = _quantised(y, case)
    full = torch.tensor([n // case["block"] for n in lens], device="cuda")
    tail = y.view(codes.shape)[torch.arange(len(lens), device="cuda"), full]  # [batch][block][heads][dim]
    return dict(codes=codes, scale=scale, tail=tail, full=full)


def prepare(case, seed):
    if case["op"] == "axes_rope":
        return _prepare_rope(case, seed)
    lens, prefixes, qlens = _lengths(case)
    k, v, q, weights = _data(case, seed)
    state = dict(case=case, lens=lens, prefixes=prefixes, qlens=qlens, q=q, weights=weights, ids=list(range(len(lens))))
    if prefixes:
        state["prefix_ids"] = [len(lens) + g for g in _group(case)]
    if own:  # the cache that a program keeps; for attention, with the tokens in it
        from quantized_kv_cache_seal_gb300.block_cache import BlockCache
        every = lens + prefixes
        cache = BlockCache(num_layers=1, max_seqs=len(every), num_q_heads=case.get("hq", case["hkv"]),
                           num_kv_heads=case["hkv"], head_dim=case["dim"], block_tokens=case["block"], code=case["code"],
                           dtype=DTYPES[case["dtype"]], max_seq_len=max([case["high"]] + prefixes),
                           pool_blocks=sum(n // case["block"] for n in every))
        if case["op"] == "evict":
            return dict(state, cache=cache, k=k, v=v)
        cache.append(0, list(range(len(every))), every, k, v)
        return dict(state, cache=cache)
    own_tokens = sum(lens)
    if case["op"] == "evict":
        left = [min(n, case["keep"] * case["block"] + n % case["block"]) for n in lens]
        return dict(state, k=k, v=v, lengths=torch.tensor(lens, device="cuda"), places=_places(lens), left=_places(left))
    for name, x in (("k", k), ("v", v)):
        state[name] = _held_in(x[:own_tokens], lens, case)
        if prefixes:
            state["p" + name] = _held_in(x[own_tokens:], prefixes, case)
    state["lengths"] = torch.tensor(lens, device="cuda")
    # queries in a padded batch: [batch][most]
    state["q_at"] = _places(qlens)
    state["q_pos"] = (state["lengths"] - torch.tensor(qlens, device="cuda"))[:, None] + torch.arange(max(qlens), device="cuda")
    if prefixes:
        # the sequences of each prefix in a padded batch: [groups][most]
        counts = [_group(case).count(g) for g in range(case["groups"])]
        state["s_at"], state["s_width"] = _places(counts), max(counts)
        state["p_lengths"] = torch.tensor(prefixes, device="cuda")
    return state


def _prepare_rope(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    t, hq, hkv, d, rot = (case[k] for k in ("tokens", "hq", "hkv", "dim", "rot"))
    if case["packed"]:  # q and k are parts of the projection's rows, before v
        qkv = torch.randn((t, hq + 2 * hkv, d), device="cuda", generator=g).to(dtype)
        q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    else:
        q = torch.randn((t, hq, d), device="cuda", generator=g).to(dtype)
        k = torch.randn((t, hkv, d), device="cuda", generator=g).to(dtype)
    weights = [torch.empty(d, device="cuda").log_normal_(0.0, 0.3, generator=g) if case["norm"] else None for _ in (0, 1)]
    freqs = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    # text and images of 32 columns in turn, 512 tokens each: time, row, column (and one more), from some place on
    i = torch.arange(t, device="cuda")
    start = i // 512 * 512
    image = (i // 512 % 2 == 1).long()
    steps = torch.stack((i * 0, (i - start) // 32, (i - start) % 32, (i - start) % 7))[:case["axes"]]
    pos = start + torch.where(image == 1, steps, i - start) + torch.randint(0, 100000, (1,), device="cuda", generator=g)
    return dict(case=case, q=q, k=k, norm=weights, freqs=freqs, pos=pos.to(torch.int32), axes=_axis_of(case),
                axis=torch.tensor(_axis_of(case), device="cuda"), eps=1e-6, out=DTYPES[case["out"]])


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"axes_rope": _axes_rope, "shared_decode": _shared, "shared_prefill": _shared, "weighed_decode": _weighed_decode,
            "window": _window, "evict": _evict}[state["case"]["op"]](state)


def _run_own(state):
    case = state["case"]
    if case["op"] == "axes_rope":
        from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
        return qk_norm_rope(state["q"], state["k"], state["pos"], state["freqs"], q_weight=state["norm"][0],
                            k_weight=state["norm"][1], eps=state["eps"], interleaved=case["interleaved"],
                            dtype=state["out"], axes=state["axes"])
    cache, ids = state["cache"], state["ids"]
    if case["op"] == "shared_decode":
        return cache.decode_attention(0, ids, state["q"], prefix_ids=state["prefix_ids"])
    if case["op"] == "shared_prefill":
        return cache.prefill_attention(0, ids, state["qlens"], state["q"], prefix_ids=state["prefix_ids"])
    weights = state["weights"].clone()  # what was received before this call
    if case["op"] == "weighed_decode":
        return cache.decode_attention(0, ids, state["q"], weights=weights), weights
    if case["op"] == "window":
        cache.window_weights(0, ids, state["qlens"], state["q"], weights)
        return weights
    cache.release(ids)
    cache.append(0, ids, state["lens"], state["k"], state["v"])
    kept = cache.evict(0, ids, weights, case["keep"], first=case["first"], last=case["last"])
    b = case["block"]
    return kept, weights, cache.read(0, ids, None, [min(n, case["keep"] * b + n % b) for n in state["lens"]])


def _axes_rope(state):
    angle = (state["pos"].double()[state["axis"]] * state["freqs"][:, None]).T[:, None]  # 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    half, interleaved = cos.shape[-1], state["case"]["interleaved"]

    def rotated(x, weight):
        y = x.float()
        if weight is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + state["eps"]) * weight
        a, b, rest = (y[..., 0:2 * half:2], y[..., 1:2 * half:2], y[..., 2 * half:]) if interleaved else (
            y[..., :half], y[..., half:2 * half], y[..., 2 * half:])
        c, s = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack((c, s), -1).flatten(-2) if interleaved else torch.cat((c, s), -1)
        return torch.cat((turned, rest), -1).to(state["out"])

    return rotated(state["q"], state["norm"][0]), rotated(state["k"], state["norm"][1])


def _values(h):
    """The cached values in 32 bits, [batch][n][heads][dim]: dequantised blocks, then the exact rows."""
    values = h["codes"].float() * h["scale"][:, :, None, :, None]
    values[torch.arange(len(values), device=values.device), h["full"]] = h["tail"].float()
    return values.flatten(1, 2)


def _queries(state):
    """[batch][kv heads][r * most][dim] of the padded batch, in 32 bits, and [batch][1][r * most] positions."""
    case, (which, place) = state["case"], state["q_at"]
    q = _padded(state["q"], which, place, case["batch"], max(state["qlens"])).float()
    r = case["hq"] // case["hkv"]
    q = q.view(q.shape[:2] + (case["hkv"], r, case["dim"])).permute(0, 2, 3, 1, 4).flatten(2, 3)
    return q, state["q_pos"].repeat(1, r)[:, None]


def _logits(state, q, pos, k):
    """Of a sequence's own tokens: those up to the query (padding queries see what they see and are left out)."""
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * state["case"]["dim"] ** -0.5
    n = torch.arange(k.shape[1], device=q.device)
    seen = (n <= pos[..., None]) & (n < state["lengths"][:, None, None, None])
    return torch.where(seen, s, float("-inf"))


def _rows(state, o):
    """Rows of the padded batch back in their order, in the case's type."""
    case, (which, place) = state["case"], state["q_at"]
    o = o.view(case["batch"], case["hkv"], case["hq"] // case["hkv"], -1, case["dim"]).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return o[which, place].to(state["q"].dtype)


def _shared(state):
    case, (group, place) = state["case"], state["s_at"]
    q, pos = _queries(state)
    s = _logits(state, q, pos, _values(state["k"]))
    # the queries of all sequences of a prefix as rows of one product: [groups][kv heads][sequences * rows][dim]
    groups, rows = case["groups"], q.shape[2]
    gq = _padded(q, group, place, groups, state["s_width"]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    pk, pv = _values(state["pk"]), _values(state["pv"])
    ps = torch.matmul(gq, pk.permute(0, 2, 3, 1)) * case["dim"] ** -0.5
    seen = torch.arange(pk.shape[1], device=q.device) < state["p_lengths"][:, None]
    ps = torch.where(seen[:, None, None], ps, float("-inf"))
    m, pm = s.amax(-1, keepdim=True), ps.amax(-1, keepdim=True)

    def of_sequences(x):  # [groups][kv heads][sequences * rows][..] -> [batch][kv heads][rows][..]
        return x.unflatten(2, (-1, rows)).permute(0, 2, 1, 3, 4)[group, place]

    e, pe = torch.exp(s - m), torch.exp(ps - pm)
    top = torch.maximum(m, of_sequences(pm))
    f, pf = torch.exp(m - top), torch.exp(of_sequences(pm) - top)
    o = torch.matmul(e, _values(state["v"]).permute(0, 2, 1, 3)) * f + of_sequences(torch.matmul(pe, pv.permute(0, 2, 1, 3))) * pf
    total = e.sum(-1, keepdim=True) * f + of_sequences(pe.sum(-1, keepdim=True)) * pf
    return _rows(state, o / total)


def _add_to_blocks(state, p):
    """The weights with p [batch][kv heads][rows][n] added by block."""
    case = state["case"]
    p = p.sum(2).unflatten(-1, (-1, case["block"])).sum(-1)
    weights = state["weights"].clone()
    n = min(p.shape[-1], weights.shape[-1])
    weights[..., :n] += p[..., :n]
    return weights


def _shares(s):
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _weighed_decode(state):
    q, pos = _queries(state)
    p = _shares(_logits(state, q, pos, _values(state["k"])))
    o = torch.matmul(p, _values(state["v"]).permute(0, 2, 1, 3))
    return _rows(state, o), _add_to_blocks(state, p)


def _window(state):
    q, pos = _queries(state)
    p = _shares(_logits(state, q, pos, _values(state["k"])))
    valid = pos < state["lengths"][:, None, None]  # padding queries stand behind the last token
    return _add_to_blocks(state, torch.where(valid[..., None], p, 0.0))


def _evict(state):
    case, weights, (which, place) = state["case"], state["weights"], state["places"]
    keep, block = case["keep"], case["block"]
    index = torch.arange(weights.shape[2], device=weights.device)
    full = (state["lengths"] // block)[:, None, None]
    rank = torch.where((index < case["first"]) | (index >= full - case["last"]), float("inf"), weights)
    rank = torch.where(index < full, rank, float("-inf"))
    kept = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values  # ties: the lowest first
    over = full > keep
    order = torch.cat((kept, kept.new_zeros(kept.shape[:2] + (keep - kept.shape[2],))), -1)
    order = torch.where(over, order, torch.arange(keep, device=order.device))
    n = torch.where(over, keep, full)  # full blocks that stay
    # the blocks in their new places, the partial one behind them
    source = torch.cat((order, torch.zeros_like(order[..., :1])), -1).scatter(-1, n.expand(order.shape[:2] + (1,)),
                                                                             full.expand(order.shape[:2] + (1,)))
    place_of = torch.arange(keep + 1, device=order.device)
    source = torch.where(place_of <= n, source, 0).clamp(max=weights.shape[2] - 1)  # [batch][heads][keep + 1]
    moved = torch.zeros_like(weights)
    c = min(keep + 1, weights.shape[2])
    moved[..., :c] = torch.where(place_of <= n, weights.gather(-1, source), 0.0)[..., :c]
    out = []
    for x in (state["k"], state["v"]):
        y = _padded(x, which, place, case["batch"], _width(state["lens"], block))
        codes, scale = _quantised(y, case)
        most = torch.finfo(x.dtype).max
        held = (codes.float() * scale[:, :, None, :, None]).clamp(-most, most).to(x.dtype)
        is_full = torch.arange(held.shape[1], device=x.device) < full[:, :, 0]
        held = torch.where(is_full[:, :, None, None, None], held, y.view(held.shape))
        at = source.clamp(max=held.shape[1] - 1).transpose(1, 2)[:, :, None, :, None]  # [batch][keep + 1][1][heads][1]
        held = held.gather(1, at.expand(-1, -1, block, -1, x.shape[2]))
        out.append(held.flatten(1, 2)[state["left"]])
    return torch.where(torch.arange(keep, device=order.device) < n, order, -1).to(torch.int32), moved, tuple(out)


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


def _exact_rope(case, seed):
    s = _prepare_rope(case, seed)
    out = []
    pos = s["pos"].double()
    turn = torch.exp(1j * torch.stack([pos[a] * f for a, f in zip(s["axes"], s["freqs"])], -1)[:, None])
    for x, w in ((s["q"], s["norm"][0]), (s["k"], s["norm"][1])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.double()
        half = case["rot"] // 2
        index = torch.arange(half, device=x.device)
        first, second = (2 * index, 2 * index + 1) if case["interleaved"] else (index, index + half)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_evict(case, k, v, weights):
    lens = _lengths(case)[0]
    b, keep = case["block"], case["keep"]
    kept = torch.full((len(lens), case["hkv"], keep), -1, dtype=torch.int32)
    moved = weights.cpu().double()
    held = [_exact_cache(x, lens, case) for x in (k, v)]
    out = ([], [])
    for i, n in enumerate(lens):
        full = n // b
        always = set(range(min(case["first"], full))) | set(range(max(0, full - case["last"]), full))
        heads = ([], [])
        for h in range(case["hkv"]):
            w = moved[i, h].tolist()
            blocks = list(range(full))
            if full > keep:
                rest = sorted((x for x in blocks if x not in always), key=lambda x: (-w[x], x))
                blocks = sorted(list(always) + rest[:keep - len(always)])
                row = [w[x] for x in blocks + ([full] if full < len(w) else [])]
                moved[i, h] = torch.tensor((row + [0.0] * len(w))[:len(w)], dtype=torch.float64)
            kept[i, h, :len(blocks)] = torch.tensor(blocks, dtype=torch.int32)
            for side in (0, 1):
                y = held[side][i][:, h]
                heads[side].append(torch.cat([y[x * b:(x + 1) * b] for x in blocks] + [y[full * b:]]))
        for side in (0, 1):
            out[side].append(torch.stack(heads[side], 1))
    most = torch.finfo(k.dtype).max
    return kept, moved, tuple(torch.cat(x).clamp_(-most, most) for x in out)


def exact(case, seed):
    if case["op"] == "axes_rope":
        return _exact_rope(case, seed)
    lens, prefixes, qlens = _lengths(case)
    k, v, q, weights = _data(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, k, v, weights)
    if work(case)["flops"] > 1.2e12:
        return None  # too long in 64 bits
    q = q.double()
    out, at = torch.empty_like(q), 0
    received = None if weights is None else weights.double()
    keys, values = _exact_cache(k, lens + prefixes, case), _exact_cache(v, lens + prefixes, case)
    group = _group(case) if prefixes else None
    r, b = case["hq"] // case["hkv"], case["block"]
    for i, n in enumerate(lens):
        m = qlens[i]
        part = q[at:at + m].view(m, case["hkv"], -1, case["dim"])
        last = torch.arange(n - m, n, device="cuda")
        for h in range(case["hkv"]):
            kh, vh = keys[i][:, h], values[i][:, h]
            s = torch.einsum("mrd,nd->mrn", part[:, h], kh) * case["dim"] ** -0.5
            s.masked_fill_((torch.arange(n, device="cuda")[None] > last[:, None])[:, None], float("-inf"))
            if prefixes:
                pk, pv = keys[len(lens) + group[i]][:, h], values[len(lens) + group[i]][:, h]
                s = torch.cat((torch.einsum("mrd,nd->mrn", part[:, h], pk) * case["dim"] ** -0.5, s), -1)
                vh = torch.cat((pv, vh))
            p = torch.softmax(s, -1)
            out[at:at + m, h * r:(h + 1) * r] = torch.einsum("mrn,nd->mrd", p, vh)
            if received is not None:
                p = torch.cat((p.sum((0, 1)), p.new_zeros(-n % b)))
                received[i, h, :len(p) // b] += p.view(-1, b).sum(-1)
        at += m
    return received if case["op"] == "window" else (out, received) if case["op"] == "weighed_decode" else out
