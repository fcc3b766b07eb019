"""Owner object of a block cache (8-bit codes, one scale per block of tokens and KV head): allocates its device
block with torch, checks tensors and forwards every call to libkvarn.so (``include/kvarn.h``, "Block cache")."""
from __future__ import annotations

import math
from typing import Optional, Sequence, Union

import torch

from . import kvarn as K

_TYPES = {torch.float16: K.KVARN_TYPE_F16, torch.bfloat16: K.KVARN_TYPE_BF16}
_CODES = {"e4m3": K.KVARN_CODE_E4M3, "int8": K.KVARN_CODE_INT8}


class BlockCache:
    """K and V of ``num_layers`` layers and ``max_seqs`` sequences in blocks of ``block_tokens`` (32, 64 or 128)
    tokens, sealed at 8 bits when full and exact until then. ``code``: "e4m3" (power-of-two scales; keeps small
    channels beside outliers) or "int8" (scale amax / 127; finer where values are alike). Tensors are ``dtype``
    (fp16 or bf16) on ``device``; calls go to ``stream`` or the device's current stream and do not synchronise.

    A torch.cuda.Stream given as ``stream`` holds the memory of a call's tensors until it is through with them, and the
    cache's own memory is held by every such or current stream that calls went to. A stream given by its address holds
    nothing: keep the tensors and the cache until its work is done. Results belong to the stream that wrote them."""

    def __init__(self, num_layers=1, max_seqs=1, num_q_heads=32, num_kv_heads=8, head_dim=128, block_tokens=64,
                 code="e4m3", dtype=torch.float16, max_seq_len=32768, pool_blocks=None, device="cuda", flags=0):
        if code not in _CODES or dtype not in _TYPES:
            raise ValueError(f"code must be one of {sorted(_CODES)} and dtype fp16 or bf16, got {code!r}, {dtype}")
        if pool_blocks is None:
            pool_blocks = max_seqs * num_layers * (max_seq_len // max(1, block_tokens))
        self.cfg = K.kvarn_block_config(num_layers, max_seqs, num_q_heads, num_kv_heads, head_dim, block_tokens,
                                        _CODES[code], _TYPES[dtype], max_seq_len, pool_blocks, flags)
        self.handle = None
        self.dtype = dtype
        self.heads, self.kv_heads, self.dim = num_q_heads, num_kv_heads, head_dim
        self.scale = 1.0 / math.sqrt(head_dim)
        self.nbytes = K.kvarn_block_required_bytes(self.cfg)
        self.mem = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        self.device = self.mem.device
        self.index = self.mem.get_device()  # -1: the CPU
        # streams that hold the cache's memory: the one that it was allocated on, then others as they come
        self._holders = {None if self.index < 0 else K.current_stream(self.device)}
        base = (self.mem.data_ptr() + 255) // 256 * 256
        with K.on_device(self.device):
            self.handle = K.kvarn_block_create(self.cfg, base, self.nbytes)

    def close(self):
        if self.handle:
            K.kvarn_block_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- tensors ---------------------------------------------------------------------------------------------
    def _refuse(self, name, x, what):
        raise ValueError(f"{name} must be {what} on {self.device}, got {x.dtype} {tuple(x.shape)} with strides "
                         f"{x.stride()} on {x.device}")

    def _dense(self, x, rows, name):
        want = (rows, self.heads, self.dim)
        if x.shape != want or x.dtype is not self.dtype or x.get_device() != self.index or not x.is_contiguous():
            self._refuse(name, x, f"a contiguous {self.dtype} tensor {want}")

    def _tokens(self, x, rows, name):
        """Elements between the tokens of k or v; its heads and channels are dense."""
        heads, dim = self.kv_heads, self.dim
        if x.shape == (rows, heads, dim) and x.dtype is self.dtype and x.get_device() == self.index:
            if x.is_contiguous():
                return heads * dim
            between, head, channel = x.stride()
            if channel == 1 and (heads == 1 or head == dim):
                return between if rows > 1 else heads * dim
        self._refuse(name, x, f"a {self.dtype} tensor {(rows, heads, dim)} with dense heads")

    def _used(self, given, stream, *tensors):
        """A call went to `stream` (an address), which the caller gave as `given` (None: the current one)."""
        if given is not None:
            K.hold(given, *tensors)
        if stream not in self._holders and not isinstance(given, int):
            K.hold(given or torch.cuda.current_stream(self.device), self.mem)
            self._holders.add(stream)

    # -- calls -----------------------------------------------------------------------------------------------
    def append(self, layer: int, seq_ids: Sequence[int], n_tokens: Sequence[int], k: torch.Tensor, v: torch.Tensor,
               stream=None):
        """Append n_tokens[i] tokens to each sequence; k, v: [sum(n_tokens)][Hkv][D], any stride between tokens."""
        rows = sum(n_tokens)
        ks, vs = self._tokens(k, rows, "k"), self._tokens(v, rows, "v")
        _same_length(seq_ids, n_tokens)
        with K.on_device(self.device, stream) as s:
            K.kvarn_block_append(self.handle, layer, seq_ids, n_tokens, k, ks, v, vs, s)
            self._used(stream, s, k, v)

    def read(self, layer: int, seq_ids: Sequence[int], starts: Optional[Sequence[int]], counts: Sequence[int],
             dtype: Optional[torch.dtype] = None, stream=None):
        """(k, v) of tokens starts[i] .. starts[i] + counts[i] - 1 (starts None: from 0) of each sequence, back to
        back, [sum(counts)][Hkv][D] of the cache's dtype or torch.float32."""
        dtype = dtype or self.dtype
        if dtype not in (self.dtype, torch.float32):
            raise ValueError(f"dtype must be {self.dtype} or torch.float32, got {dtype}")
        _same_length(seq_ids, counts)
        if starts is not None:
            _same_length(seq_ids, starts)
        if len(counts) and min(counts) < 0:
            raise ValueError("counts must not be negative")
        shape = (sum(counts), self.kv_heads, self.dim)
        with K.on_device(self.device, stream) as s:
            k = torch.empty(shape, dtype=dtype, device=self.device)
            v = torch.empty_like(k)
            K.kvarn_block_read(self.handle, layer, seq_ids, starts, counts, k, v, dtype is torch.float32, s)
            self._used(stream, s)
        return k, v

    def _queries(self, q, rows, out):
        self._dense(q, rows, "q")
        if out is not None:
            self._dense(out, rows, "out")

    def decode_attention(self, layer: int, seq_ids: Sequence[int], q: torch.Tensor, out: Optional[torch.Tensor] = None,
                         scale: Optional[float] = None, stream=None) -> torch.Tensor:
        """One query token per sequence over all its cached tokens; q, out: [len(seq_ids)][Hq][D]."""
        self._queries(q, len(seq_ids), out)
        with K.on_device(self.device, stream) as s:
            if out is None:
                out = torch.empty_like(q)
            K.kvarn_block_decode_attention(self.handle, layer, seq_ids, q, out, self.scale if scale is None else scale, s)
            self._used(stream, s, q, out)
        return out

    def decode_step(self, layer: int, seq_ids: Sequence[int], k: torch.Tensor, v: torch.Tensor, q: torch.Tensor,
                    out: Optional[torch.Tensor] = None, scale: Optional[float] = None, stream=None) -> torch.Tensor:
        """Append one token per sequence and attend its query; k, v: [len(seq_ids)][Hkv][D]."""
        n = len(seq_ids)
        ks, vs = self._tokens(k, n, "k"), self._tokens(v, n, "v")
        self._queries(q, n, out)
        with K.on_device(self.device, stream) as s:
            if out is None:
                out = torch.empty_like(q)
            K.kvarn_block_decode_step(self.handle, layer, seq_ids, k, ks, v, vs, q, out,
                                      self.scale if scale is None else scale, s)
            self._used(stream, s, k, v, q, out)
        return out

    def prefill_attention(self, layer: int, seq_ids: Sequence[int], q_lens: Sequence[int], q: torch.Tensor,
                          out: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                          stream=None) -> torch.Tensor:
        """Causal attention of the last q_lens[i] tokens of each sequence; q, out: [sum(q_lens)][Hq][D]."""
        _same_length(seq_ids, q_lens)
        self._queries(q, sum(q_lens), out)
        with K.on_device(self.device, stream) as s:
            if out is None:
                out = torch.empty_like(q)
            K.kvarn_block_prefill_attention(self.handle, layer, seq_ids, q_lens, q, out,
                                            self.scale if scale is None else scale, s)
            self._used(stream, s, q, out)
        return out

    def prefill(self, layer: int, seq_ids: Sequence[int], n_tokens: Sequence[int], k: torch.Tensor, v: torch.Tensor,
                q: torch.Tensor, out: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                stream=None) -> torch.Tensor:
        """Append a prompt chunk and attend its queries."""
        _same_length(seq_ids, n_tokens)
        rows = sum(n_tokens)
        ks, vs = self._tokens(k, rows, "k"), self._tokens(v, rows, "v")
        self._queries(q, rows, out)
        with K.on_device(self.device, stream) as s:
            if out is None:
                out = torch.empty_like(q)
            K.kvarn_block_prefill(self.handle, layer, seq_ids, n_tokens, k, ks, v, vs, q, out,
                                  self.scale if scale is None else scale, s)
            self._used(stream, s, k, v, q, out)
        return out

    def release(self, seq_ids: Union[int, Sequence[int]]):
        """Drop sequences in every layer. A later append may reuse their blocks: it must follow, on the GPU, the
        calls that still read them (issue both to one stream)."""
        K.kvarn_block_release(self.handle, [seq_ids] if isinstance(seq_ids, int) else seq_ids)

    def length(self, layer: int, seq_id: int) -> int:
        return K.kvarn_block_length(self.handle, layer, seq_id)

    def check_device_error(self, stream=None) -> int:
        with K.on_device(self.device, stream) as s:
            self._used(stream, s)
            return K.kvarn_block_check_device_error(self.handle, s)


def _same_length(seq_ids, counts):
    if len(seq_ids) != len(counts):
        raise ValueError(f"{len(seq_ids)} sequences, but {len(counts)} counts")
