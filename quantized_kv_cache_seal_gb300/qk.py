"""RMS norm of query and key heads with the position rotation in the same pass (``kvarn_qk_norm_rope``,
``include/kvarn.h``): makes the post-rotation queries and keys that the caches take."""
from __future__ import annotations

import functools
from typing import Optional, Sequence

import torch

from . import kvarn as K

_TYPES = {torch.float16: K.KVARN_TYPE_F16, torch.bfloat16: K.KVARN_TYPE_BF16}


def _refuse(name, x, want):
    raise ValueError(f"{name} must be {want}, got {x.dtype} {tuple(x.shape)} with strides {x.stride()} on {x.device}")


def _stride(x, name, dtype, index, tokens, heads, dim):
    """Elements between the tokens of x: [tokens][heads][dim] on CUDA device `index`, heads and channels dense."""
    if x.dtype is dtype and x.get_device() == index and x.shape == (tokens, heads, dim):
        if x.is_contiguous():
            return heads * dim
        between, head, channel = x.stride()
        if channel == 1 and (heads == 1 or head == dim):
            return between if tokens > 1 else heads * dim
    _refuse(name, x, f"a {dtype} tensor {(tokens, heads, dim)} on cuda:{index} with dense heads")


def _table(x, name, dtype, index, shape):
    if x.dtype is not dtype or x.get_device() != index or x.shape != shape or not x.is_contiguous():
        _refuse(name, x, f"a contiguous {dtype} tensor {shape} on cuda:{index}")


@functools.lru_cache(maxsize=64)
def _config(hq, hkv, dim, rot, interleaved, in_type, out_type, eps):
    return K.kvarn_qk_config(hq, hkv, dim, rot, interleaved, in_type, out_type, eps)


@functools.lru_cache(maxsize=64)
def _axes(axes, pairs, count):
    """One axis a pair, each below `count`, as the bytes that the library takes."""
    if len(axes) != pairs or not all(0 <= a < count for a in axes) or not 1 <= count <= 255:
        raise ValueError(f"axes must be {pairs} numbers from 0 to {count - 1} (1 to 255 axes), got {axes}")
    return bytes(axes)


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, freqs: torch.Tensor,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False, dtype: Optional[torch.dtype] = None, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, stream=None, axes: Optional[Sequence[int]] = None):
    """Normalise (where a weight is given) and rotate every head of q [T][Hq][D] and k [T][Hkv][D] (or None).

    positions: int32 [T]; freqs: float64 [R / 2], radians per position, R <= D a multiple of 8 (channels from R on
    pass); weights: float32 [D]. With ``axes`` (R / 2 ints, a tuple is quickest) positions are int32 [A][T], any
    stride between the axes, and pair i turns by positions[axes[i]] freqs[i]: sections of an image's time, row and
    column, or axes in turn, as the model has them. q and k are fp16 or bf16 and may be parts of a packed projection (any stride between
    tokens). Results are ``dtype`` (default: the inputs'; fp16 for a KVarN cache) or go to q_out and k_out, which
    may be q and k themselves. Returns (q, k); no gradient is recorded. A torch.cuda.Stream given as ``stream`` holds the
    tensors' memory until it is through with them; one given by its address does not."""
    index = q.get_device()
    if q.dim() != 3 or (k is not None and k.dim() != 3) or index < 0 or q.dtype not in _TYPES:
        _refuse("q", q, "a CUDA tensor [tokens][heads][dim] of fp16 or bf16, as k")
    tokens, hq, dim = q.shape
    hkv = 0 if k is None else k.shape[1]
    in_type = q.dtype
    given = q_out if q_out is not None else k_out
    out_type = dtype or (in_type if given is None else given.dtype)
    if out_type not in _TYPES:
        raise ValueError(f"dtype must be fp16 or bf16, got {out_type}")
    if k is None and (k_out is not None or k_weight is not None):
        raise ValueError("k_out or k_weight without k")
    qs = _stride(q, "q", in_type, index, tokens, hq, dim)
    ks = 0 if k is None else _stride(k, "k", in_type, index, tokens, hkv, dim)
    if axes is None:
        _table(positions, "positions", torch.int32, index, (tokens,))
    else:
        if positions.dim() != 2 or positions.shape[1] != tokens or positions.dtype is not torch.int32 or (
                positions.get_device() != index or (tokens > 1 and positions.stride(1) != 1)):
            _refuse("positions", positions, f"a torch.int32 tensor (axes, {tokens}) with dense rows on cuda:{index}")
        axes = _axes(tuple(axes), freqs.numel(), positions.shape[0])
    _table(freqs, "freqs", torch.float64, index, (freqs.numel(),))
    if q_weight is not None:
        _table(q_weight, "q_weight", torch.float32, index, (dim,))
    if k_weight is not None:
        _table(k_weight, "k_weight", torch.float32, index, (dim,))
    qos = hq * dim if q_out is None else _stride(q_out, "q_out", out_type, index, tokens, hq, dim)
    kos = hkv * dim if k_out is None else _stride(k_out, "k_out", out_type, index, tokens, hkv, dim)
    cfg = _config(hq, hkv, dim, 2 * freqs.shape[0], int(interleaved), _TYPES[in_type], _TYPES[out_type], eps)
    with K.on_device(q.device, stream) as s:  # results are allocated on the stream that writes them
        if q_out is None:
            q_out = torch.empty((tokens, hq, dim), dtype=out_type, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty((tokens, hkv, dim), dtype=out_type, device=q.device)
        if axes is None:
            K.kvarn_qk_norm_rope(cfg, tokens, q, qs, k, ks, q_weight, k_weight, positions, freqs, q_out, qos, k_out, kos, s)
        else:
            K.kvarn_qk_norm_rope_axes(cfg, tokens, q, qs, k, ks, q_weight, k_weight, positions, positions.stride(0),
                                      positions.shape[0], axes, freqs, q_out, qos, k_out, kos, s)
        if stream is not None:
            K.hold(stream, q, k, positions, freqs, q_weight, k_weight, q_out, k_out)
    return q_out, k_out
