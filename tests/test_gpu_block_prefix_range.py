"""GPU tests of attention behind a shared prefix (include/kvarn.h) at the ends of bf16's range: V near its largest and
smallest values, on both sides and on one, in every form that such calls take. Bounds: block_ref.attend's (test_gpu_block_prefix.py)."""
import pytest
import torch

from tests import block_ref
from tests.test_gpu_block import check, make, tokens
from tests.test_gpu_block_evict import near, received, some_weights
from tests.test_gpu_block_prefix import want_of

pytestmark = pytest.mark.gpu

# sequences, queries of each (None: one, as decode), tokens of the prefix
FORMS = {"decode, walked once": (40, None, 2100), "decode, each": (3, None, 300), "prompts, walked once": (60, 6, 4001),
         "prompts, walked once in pairs": (150, 6, 700), "prompts, in front": (3, 40, 700)}


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("prefix,own", [(120, 120), (-88, -88), (120, 90), (90, 120), (-88, -60)])
@pytest.mark.parametrize("form", FORMS)
def test_values_at_the_ends_of_the_range(form, prefix, own, code):
    seqs, m, n = FORMS[form]
    lens = [9 + (37 * i) % 90 for i in range(seqs)] + [n]
    lens[0] = 70
    c = make(max_seqs=seqs + 1, num_q_heads=32, num_kv_heads=8, block_tokens=64, code=code, dtype=torch.bfloat16, max_seq_len=4096,
             pool_blocks=sum(x // 64 for x in lens))
    k, v = (list(torch.split(tokens(sum(lens), 8, 128, torch.bfloat16, s, 0.3), lens)) for s in (1101, 1102))
    v = [x.clamp(-100, 100) * 2.0 ** (prefix if i == seqs else own) for i, x in enumerate(v)]
    assert all(bool(torch.isfinite(x).all()) for x in v)
    for s in range(seqs + 1):
        c.append(0, [s], [lens[s]], k[s], v[s])
    ids, count = list(range(seqs)), 1 if m is None else m
    q = tokens(seqs * count, 32, 128, torch.bfloat16, 1103, 0.3)
    out = c.decode_attention(0, ids, q, prefix_ids=[seqs] * seqs) if m is None else c.prefill_attention(
        0, ids, [m] * seqs, q, prefix_ids=[seqs] * seqs)
    for s in {0, 1, seqs - 1}:
        want, tol = want_of(q, s * count, k, v, seqs, s, lens[s], count, 64, code, 128)
        check(out[s * count:(s + 1) * count], want, tol, s)
    assert c.check_device_error() == 0


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("prefix,own", [(120, 120), (-88, -88), (120, 90), (-88, -60)])
@pytest.mark.parametrize("form", ["decode, walked once", "decode, each"])
def test_weights_at_the_ends_of_the_range(form, prefix, own, code):
    """V's scale, which decode carries in its weights, must not show in what blocks receive. Beside received()'s bound, which is for
    a log2 of the scale under 2^5: under 2^7 its roundings are 8 * 2^7 * 2^-24 = 2^-14 of a weight, and 1 / scale, below fp32's normal
    range, has 16 bits in a tile's sum and in the row's: under 2^-13 in all."""
    seqs, _, n = FORMS[form]
    lens = [9 + (37 * i) % 90 for i in range(seqs)] + [n]
    c = make(max_seqs=seqs + 1, num_q_heads=32, num_kv_heads=8, block_tokens=64, code=code, dtype=torch.bfloat16, max_seq_len=4096,
             pool_blocks=sum(x // 64 for x in lens))
    k, v = (list(torch.split(tokens(sum(lens), 8, 128, torch.bfloat16, s, 0.3), lens)) for s in (1111, 1112))
    for s in range(seqs + 1):
        c.append(0, [s], [lens[s]], k[s], v[s].clamp(-100, 100) * 2.0 ** (prefix if s == seqs else own))
    q = tokens(seqs, 32, 128, torch.bfloat16, 1113, 0.3)
    w = some_weights(c, 1114)
    before = w.clone()
    c.decode_attention(0, list(range(seqs)), q, prefix_ids=[seqs] * seqs, weights=w)
    for s in {0, 1, seqs - 1}:
        held = torch.cat([block_ref.hold(k[x], 64, code) for x in (seqs, s)])
        want, tol = received(q[s:s + 1], held, 128 ** -0.5, [n + lens[s] - 1], 64, n)
        near(w[s], before[s], want, tol + want * 2.0 ** -13, s)
    assert c.check_device_error() == 0
