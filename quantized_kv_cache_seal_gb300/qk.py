"""RMS norm of query and key heads with the position rotation in the same pass (``kvarn_qk_norm_rope``,
``include/kvarn.h``): makes the post-rotation queries and keys that the caches take."""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import kvarn as K

_TYPES = {torch.float16: K.KVARN_TYPE_F16, torch.bfloat16: K.KVARN_TYPE_BF16}


def _stride(x, name, tokens, dim):
    """Elements between the tokens of x: [tokens][heads][dim], heads and channels dense."""
    if x.dim() != 3 or x.shape[0] != tokens or x.shape[2] != dim or not x.is_cuda or (
            x.numel() > 0 and (x.stride(2) != 1 or (x.shape[1] > 1 and x.stride(1) != dim))):
        raise ValueError(f"{name} must be a CUDA tensor [{tokens}][heads][{dim}] with dense heads, got {tuple(x.shape)} "
                         f"with strides {x.stride()} on {x.device}")
    return x.stride(0) if tokens > 1 else x.shape[1] * dim


def _table(x, name, dtype, shape, device):
    if x.dtype != dtype or tuple(x.shape) != shape or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on {device}, got {x.dtype} "
                         f"{tuple(x.shape)} on {x.device}")
    return x


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, freqs: torch.Tensor,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False, dtype: Optional[torch.dtype] = None, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, stream=None):
    """Normalise (where a weight is given) and rotate every head of q [T][Hq][D] and k [T][Hkv][D] (or None).

    positions: int32 [T]; freqs: float64 [R / 2], radians per position, R <= D a multiple of 8 (channels from R on
    pass); weights: float32 [D]. q and k are fp16 or bf16 and may be parts of a packed projection (any stride between
    tokens). Results are ``dtype`` (default: the inputs'; fp16 for a KVarN cache) or go to q_out and k_out, which
    may be q and k themselves. Returns (q, k)."""
    if q.dim() != 3:
        raise ValueError(f"q must be [tokens][heads][dim], got {tuple(q.shape)}")
    tokens, hq, dim = q.shape
    given = q_out if q_out is not None else k_out
    out_type = dtype or (given.dtype if given is not None else q.dtype)
    for name, x in (("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out)):
        if x is None:
            continue
        want = out_type if name.endswith("out") else q.dtype
        if want not in _TYPES or x.dtype != want or x.device != q.device:
            raise ValueError(f"{name} must be fp16 or bf16 {want} on {q.device}, got {x.dtype} on {x.device}")
    qs = _stride(q, "q", tokens, dim)
    ks = 0 if k is None else _stride(k, "k", tokens, dim)
    _table(positions, "positions", torch.int32, (tokens,), q.device)
    if freqs.dim() != 1:
        raise ValueError("freqs must have one dimension")
    _table(freqs, "freqs", torch.float64, (freqs.shape[0],), q.device)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _table(w, name, torch.float32, (dim,), q.device)
    if k is None and (k_out is not None or k_weight is not None):
        raise ValueError("k_out or k_weight without k")
    if out_type not in _TYPES:
        raise ValueError(f"dtype must be fp16 or bf16, got {out_type}")
    with torch.cuda.device(q.device):
        if stream is None:
            stream, where = torch.cuda.current_stream(), contextlib.nullcontext()
        else:  # results are allocated on the stream that writes them
            where = torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)
        with where:
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=out_type, device=q.device)
            if k is not None and k_out is None:
                k_out = torch.empty(k.shape, dtype=out_type, device=q.device)
        for name, x, y in (("q_out", q, q_out), ("k_out", k, k_out)):
            if x is not None and y.shape != x.shape:
                raise ValueError(f"{name} must have its input's shape {tuple(x.shape)}, got {tuple(y.shape)}")
        cfg = K.kvarn_qk_config(hq, 0 if k is None else k.shape[1], dim, 2 * freqs.shape[0], int(interleaved),
                                _TYPES[q.dtype], _TYPES[out_type], eps)
        K.kvarn_qk_norm_rope(cfg, tokens, q, qs, k, ks, q_weight, k_weight, positions, freqs, q_out,
                             _stride(q_out, "q_out", tokens, dim), k_out,
                             0 if k is None else _stride(k_out, "k_out", tokens, dim), stream)
    return q_out, k_out
