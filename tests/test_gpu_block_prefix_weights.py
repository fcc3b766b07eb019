"""GPU tests of the weights that blocks receive behind a shared prefix (include/kvarn.h) where the prefix's part of a row's
denominator is nothing, far from 1, or walked by each sequence itself."""
import pytest
import torch

from tests import block_ref
from tests.test_gpu_block import TYPES, make, tokens
from tests.test_gpu_block_evict import near, some_weights

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
