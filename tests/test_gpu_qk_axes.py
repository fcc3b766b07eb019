"""GPU tests of the norm + rotation by several axes of positions (include/kvarn.h) against 64 bits."""
import pytest
import torch

from tests import block_ref
from tests.test_gpu_block import TYPES, tokens

pytestmark = pytest.mark.gpu


def turned(x, weight, pos, axes, freqs, interleaved, eps):
    """block_ref.norm_rope's value and bound, pair by pair of its own axis."""
    out, tol = block_ref.norm_rope(x, weight, pos[0], freqs, interleaved, eps)
    half = freqs.shape[0]
    for a in sorted(set(axes)):
        y, t = block_ref.norm_rope(x, weight, pos[a], freqs, interleaved, eps)
        pairs = torch.tensor([i for i in range(half) if axes[i] == a])
        for at in ((2 * pairs, 2 * pairs + 1) if interleaved else (pairs, pairs + half)):
            out[..., at], tol[..., at] = y[..., at], t[..., at]
    return out, tol


@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (128, 64), (80, 80), (96, 48), (256, 256), (192, 96), (8, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("types", [("fp16", "fp16"), ("bf16", "fp16"), ("bf16", "bf16")])
def test_axes(dim, rot, interleaved, types):
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    src, dst = TYPES[types[0]], TYPES[types[1]]
    half = rot // 2
    freqs = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    for t, hq, hkv, count in ((1, 1, 1, 3), (7, 5, 2, 2), (1000, 16, 3, 4), (33, 70, 20, 3)):
        qkv = tokens(t, hq + 2 * hkv, dim, src, t, 0.3)
        g = torch.Generator().manual_seed(t)
        pos = torch.randint(-5, 300000, (count, t), generator=g, dtype=torch.int32).cuda()
        w = torch.rand(dim, generator=g).cuda() + 0.5
        for axes in (tuple(i * count // half for i in range(half)), tuple(i % count for i in range(half)), [count - 1] * half):
            q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
            got = qk_norm_rope(q, k, pos, freqs, w, None, eps=1e-5, interleaved=interleaved, dtype=dst, axes=axes)
            for x, wt, y in ((q, w, got[0]), (k, None, got[1])):
                want, tol = turned(x, wt, pos, axes, freqs, interleaved, 1e-5)
                tol = tol + want.abs() * torch.finfo(dst).eps / 2 + float(torch.finfo(dst).smallest_normal)
                assert y.dtype == dst and float(((y.cpu().double() - want).abs() / tol).max()) <= 1


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (128, 64), (96, 96)])
def test_one_axis_is_the_plain_call(dim, rot, interleaved):
    """The same bits: one axis, and several that say the same (one row for all of them)."""
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    freqs = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    q = tokens(300, 12, dim, torch.bfloat16, 3, 0.3)
    pos = torch.randint(0, 2 ** 31 - 1, (300,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    want, _ = qk_norm_rope(q, None, pos, freqs, interleaved=interleaved)
    for positions, axes in ((pos[None], [0] * (rot // 2)), (pos.expand(3, 300), [i % 3 for i in range(rot // 2)]),
                            (torch.stack((pos, pos)), [0, 1] * (rot // 4))):
        got, _ = qk_norm_rope(q, None, positions, freqs, interleaved=interleaved, axes=axes)
        assert torch.equal(got, want)


def test_rows_of_a_longer_table_in_place_and_captured():
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    freqs = 1e4 ** (-torch.arange(0, 128, 2, dtype=torch.float64, device="cuda") / 128)
    axes = tuple([0] * 16 + [1] * 24 + [2] * 24)
    q = tokens(100, 8, 128, torch.float16, 4, 0.3)
    table = torch.randint(0, 100000, (3, 500), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    want, _ = qk_norm_rope(q, None, table[:, 40:140].contiguous(), freqs, axes=axes)
    assert torch.equal(qk_norm_rope(q, None, table[:, 40:140], freqs, axes=axes)[0], want)
    other, _ = qk_norm_rope(q, None, table[:, 41:141].contiguous(), freqs, axes=axes)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work, pos = q.clone(), table[:, 40:140].clone()
        with torch.cuda.graph(g, stream=s):
            qk_norm_rope(work, None, pos, freqs, q_out=work, axes=axes)
        g.replay()
        assert torch.equal(work, want)
        work.copy_(q)
        pos.copy_(table[:, 41:141])
        g.replay()
        assert torch.equal(work, other)
    s.synchronize()


def test_refusals():
    from quantized_kv_cache_seal_gb300.qk import qk_norm_rope
    q = tokens(4, 2, 64, torch.float16, 1)
    pos = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    ok = [i % 3 for i in range(32)]
    for p, axes in ((pos, ok[:-1]), (pos, ok + [0]), (pos, [3] * 32), (pos, [-1] * 32), (pos[0], ok), (pos[:, :3], ok), (pos.long(), ok),
                    (pos.cpu(), ok), (pos.t().contiguous().t(), ok), (pos[:0], ok), (pos, None)):
        with pytest.raises(ValueError):
            qk_norm_rope(q, None, p, f, axes=axes)
    empty, _ = qk_norm_rope(q[:0], None, pos[:, :0], f, axes=ok)
    assert empty.shape == (0, 2, 64)
