"""RMS norm of query and key heads with the position rotation in the same pass (``kvarn_qk_norm_rope``,
``include/kvarn.h``): makes the post-rotation queries and keys that the caches take."""
from __future__ import annotations

import contextlib
import functools
from typing import Optional

import torch

from . import kvarn as K

_TYPES = {torch.float16: K.KVARN_TYPE_F16, torch.bfloat16: K.KVARN_TYPE_BF16}
_HERE = contextlib.nullcontext()


def _refuse(name, x, want):
    raise ValueError(f"{name} must be {want}, got {x.dtype} {tuple(x.shape)} with strides {x.stride()} on {x.device}")


def _stride(x, name, dtype, device, tokens, heads, dim):
    """Elements between the tokens of x: [tokens][heads][dim], heads and channels dense."""
    stride = x.stride()
    if (x.dtype != dtype or x.device != device or x.shape != (tokens, heads, dim)
            or (stride[2] != 1 or (heads > 1 and stride[1] != dim)) and x.numel() > 0):
        _refuse(name, x, f"a {dtype} tensor {(tokens, heads, dim)} on {device} with dense heads")
    return stride[0] if tokens > 1 else heads * dim


@functools.lru_cache(maxsize=64)
def _config(hq, hkv, dim, rot, interleaved, in_type, out_type, eps):
    return K.kvarn_qk_config(hq, hkv, dim, rot, interleaved, in_type, out_type, eps)


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, freqs: torch.Tensor,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False, dtype: Optional[torch.dtype] = None, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, stream=None):
    """Normalise (where a weight is given) and rotate every head of q [T][Hq][D] and k [T][Hkv][D] (or None).

    positions: int32 [T]; freqs: float64 [R / 2], radians per position, R <= D a multiple of 8 (channels from R on
    pass); weights: float32 [D]. q and k are fp16 or bf16 and may be parts of a packed projection (any stride between
    tokens). Results are ``dtype`` (default: the inputs'; fp16 for a KVarN cache) or go to q_out and k_out, which
    may be q and k themselves. Returns (q, k)."""
    if q.dim() != 3 or (k is not None and k.dim() != 3) or not q.is_cuda or q.dtype not in _TYPES:
        _refuse("q", q, "a CUDA tensor [tokens][heads][dim] of fp16 or bf16, as k")
    tokens, hq, dim = q.shape
    hkv = 0 if k is None else k.shape[1]
    device, in_type = q.device, q.dtype
    given = q_out if q_out is not None else k_out
    out_type = dtype or (in_type if given is None else given.dtype)
    if out_type not in _TYPES:
        raise ValueError(f"dtype must be fp16 or bf16, got {out_type}")
    if k is None and (k_out is not None or k_weight is not None):
        raise ValueError("k_out or k_weight without k")
    qs = _stride(q, "q", in_type, device, tokens, hq, dim)
    ks = 0 if k is None else _stride(k, "k", in_type, device, tokens, hkv, dim)
    if (positions.dtype != torch.int32 or positions.shape != (tokens,) or positions.device != device
            or not positions.is_contiguous()):
        _refuse("positions", positions, f"a contiguous int32 tensor [{tokens}] on {device}")
    if freqs.dtype != torch.float64 or freqs.dim() != 1 or freqs.device != device or not freqs.is_contiguous():
        _refuse("freqs", freqs, f"a contiguous float64 tensor [rot_dim / 2] on {device}")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype != torch.float32 or w.shape != (dim,) or w.device != device or not w.is_contiguous()):
            _refuse(name, w, f"a contiguous float32 tensor [{dim}] on {device}")
    cfg = _config(hq, hkv, dim, 2 * freqs.shape[0], int(interleaved), _TYPES[in_type], _TYPES[out_type], eps)
    with K.on_device(device):
        if stream is None:
            stream = K.current_stream(device)
            where = _HERE
        else:  # results are allocated on the stream that writes them
            where = torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)
        qos, kos = hq * dim, hkv * dim
        with where:
            if q_out is None:
                q_out = torch.empty((tokens, hq, dim), dtype=out_type, device=device)
            else:
                qos = _stride(q_out, "q_out", out_type, device, tokens, hq, dim)
            if k is not None:
                if k_out is None:
                    k_out = torch.empty((tokens, hkv, dim), dtype=out_type, device=device)
                else:
                    kos = _stride(k_out, "k_out", out_type, device, tokens, hkv, dim)
        K.kvarn_qk_norm_rope(cfg, tokens, q, qs, k, ks, q_weight, k_weight, positions, freqs, q_out, qos, k_out, kos, stream)
    return q_out, k_out
