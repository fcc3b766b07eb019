"""GPU tests of the weights that blocks receive behind a shared prefix (include/kvarn.h) where the prefix's part of a row's
denominator is nothing, far from 1, or walked by each sequence itself."""
import pytest
import torch

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
