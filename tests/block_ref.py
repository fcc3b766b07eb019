"""The block cache, its attention and the norm + rotation from their definitions, in 64 bits on the CPU (test
infrastructure; no code shared with the library)."""
import torch


def f64(x):
    return x.detach().cpu().double()


def hold(x, block, code):
    """What the cache holds for one sequence x [n][heads][dim] (fp16 or bf16): [n][heads][dim] in 64 bits."""
    x = x.detach().cpu()
    y = x.double().clone()
    n = x.shape[0]
    for b in range(n // block):
        part = x[b * block:(b + 1) * block]
        for h in range(x.shape[1]):
            y[b * block:(b + 1) * block, h] = _sealed(part[:, h].double(), code)
    return y


def _sealed(v, code):
    if not bool(torch.isfinite(v).all()):
        return torch.full_like(v, float("nan"))
    amax = float(v.abs().max())
    if amax == 0:
        return v * 0
    if code == "int8":
        s = max(float((torch.tensor(amax, dtype=torch.float32) / 127).double()), 2.0 ** -100)
        n = torch.round(v / s).clamp(-127, 127)  # 64-bit quotients of 11-bit by 24-bit numbers: ties come out exact
        return n * s
    e = -100
    while 448.0 * 2.0 ** e < amax:
        e += 1
    s = 2.0 ** e
    y = (v / s).abs()
    step = torch.full_like(y, 2.0 ** -9)
    for k in range(-6, 9):  # binades of e4m3: steps of an eighth of the leading bit
        step = torch.where(y >= 2.0 ** k, torch.full_like(y, 2.0 ** (k - 3)), step)
    return torch.sign(v) * torch.round(y / step) * step * s


def attend(q, k, v, scale, last):
    """o [rows][hq][dim] and a bound on a kernel's error. q [rows][hq][dim] in the inputs' type; k, v [n][hkv][dim] in
    64 bits; row i sees positions <= last[i].

    The bound: each weight is rounded to f16 (half a step: 2^-11 of it, or 2^-25 where it is under f16's normal
    range); logits are off by (dim + 8) roundings of 2^-24 of sum |q k| scale (each changes a weight by that share,
    numerator and denominator); sums and divisions a further 2^-16; and the output's own rounding. A weight stands
    for p s (s: V's scale in its block) in units in which the largest of the row is at least 2^7, so 2^-25 is at
    most 2^-32 max(p s), and its error meets a code of at most 512: over n tokens n 2^-32 512 max(p s). A block
    whose largest |v| is a has 512 s <= 4.1 a (int8: s = a / 127; e4m3: s <= 2 a / 448; exact tokens: 512 s <= 2 a),
    so with the largest |v| of all blocks for a: n 2^-29 max(p) max|v|. (A block of zeros counts as s = 2^-60, less
    than that of any other here.)"""
    dtype = q.dtype
    q = f64(q)
    rows, hq, dim = q.shape
    n, hkv, _ = k.shape
    r = hq // hkv
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    seen = torch.arange(n)[None] <= torch.as_tensor(last)[:, None]
    for h in range(hq):
        kh, vh = k[:, h // r], v[:, h // r]
        s = (q[:, h] @ kh.T) * scale
        s = torch.where(seen, s, torch.tensor(float("-inf"), dtype=torch.float64))
        m = s.amax(-1, keepdim=True) if n else s
        p = torch.where(seen, torch.exp(s - torch.where(torch.isfinite(m), m, torch.zeros_like(m))), torch.zeros_like(s))
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, torch.zeros_like(p))
        o[:, h] = p @ vh
        off = (q[:, h].abs() @ kh.abs().T) * abs(scale) * (dim + 8) * 2.0 ** -24
        off = torch.where(seen, off, torch.zeros_like(off)).amax(-1, keepdim=True) if n else total
        mass = p @ vh.abs()
        small = n * 2.0 ** -29 * p.amax(-1, keepdim=True) * vh.abs().max() if n else total
        tol[:, h] = mass * (2.0 ** -11 + 2 * off + 2.0 ** -16) + small
    return o, tol + o.abs() * torch.finfo(dtype).eps / 2 + float(torch.finfo(dtype).smallest_normal) * 2.0 ** -7


def norm_rope(x, weight, pos, freqs, interleaved, eps):
    """y and a bound on a kernel's error before the output's rounding: a few fp32 roundings of the pair's size."""
    y = f64(x)
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * f64(weight)
    phi = f64(pos)[:, None, None] * f64(freqs)
    half = freqs.shape[0]
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    size = y.abs()
    out = y.clone()
    out[..., a] = y[..., a] * phi.cos() - y[..., b] * phi.sin()
    out[..., b] = y[..., b] * phi.cos() + y[..., a] * phi.sin()
    size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, size * 2.0 ** -20
