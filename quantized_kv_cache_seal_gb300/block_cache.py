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
    nothing: keep the tensors and the cache until its work is done. Results belong to the stream that wrote them.

    Attention takes ``prefix_ids``, one a sequence (None or -1: none): sequences of the cache whose tokens stand in front
    of the sequence's own; neighbours in the call that name the same one share its reading where that is quicker. (Calls with
    prefixes or weights take kernels of their own, of the same definition and bounds but not always the same last bits; single
    queries of many short sequences are quicker there also with no prefix named, ``prefix_ids=[None] * n``.) With ``weights``, a layer of
    ``new_weights()``, single queries add up what each block receives of their softmax weights, ``window_weights`` adds
    the last queries' of prompts, and ``evict`` keeps the blocks with the most."""

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
        # places of the blocks' weights in a layer
        self.weights_shape = (max_seqs, num_kv_heads, max_seq_len // max(1, block_tokens) + 1)
        self.nbytes = K.kvarn_block_required_bytes(self.cfg)
        self.mem = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        self.device = self.mem.device
        self.index = self.mem.get_device()  # -1: the CPU
        self._spaces = [torch.empty(1 << 20, dtype=torch.uint8, device=device)]  # workspaces of calls that want one, the last in use
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
            K.hold(given or torch.cuda.current_stream(self.device), self.mem, *self._spaces)
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

    def new_weights(self) -> torch.Tensor:
        """float32 zeros [num_layers][max_seqs][Hkv][blocks]: the weights that blocks receive, by sequence id. Yours to
        keep, one or more; calls take one layer of it. Zero a sequence's when it begins."""
        return torch.zeros((self.cfg.num_layers,) + self.weights_shape, dtype=torch.float32, device=self.device)

    def _weights(self, x):
        if x.shape != self.weights_shape or x.dtype is not torch.float32 or x.get_device() != self.index or (
                not x.is_contiguous()):
            self._refuse("weights", x, f"a contiguous torch.float32 tensor {self.weights_shape}")

    def _attend(self, layer, seq_ids, prefix_ids, counts, q, out, scale, weights, stream, k=None, ks=0, v=None, vs=0):
        """The calls with prefixes or weights; counts: queries of each sequence (None: one), or tokens to append if k."""
        prefix_ids = _prefixes(prefix_ids)
        if weights is not None:
            self._weights(weights)
        with K.on_device(self.device, stream) as s:
            if out is None:
                out = torch.empty_like(q)
            scale = self.scale if scale is None else scale

            def call(space, n):
                if k is None:
                    K.kvarn_block_attend(self.handle, layer, seq_ids, prefix_ids, counts, q, out, scale, weights, space, n, s)
                else:
                    K.kvarn_block_append_attend(self.handle, layer, seq_ids, prefix_ids, counts, k, ks, v, vs, q, out, scale,
                                                weights, space, n, s)

            self._in_space(stream, call, lambda: K.kvarn_block_attend_workspace(self.handle, layer, seq_ids, prefix_ids, counts,
                                                                                k is not None, weights is not None))
            self._used(stream, s, k, v, q, out, weights)
        return out

    def _in_space(self, given, call, need):
        """call(workspace, bytes) with the cache's own, which grows where need() says that it is too small. Calls of one
        cache are ordered on the GPU, so that they can share it. Spaces that were outgrown stay, since captured graphs use
        them; each is at least twice as large as the one before, so that all of them together take less than the last one."""
        space = self._spaces[-1]
        try:
            return call(space, space.numel())
        except K.KVarNError as e:
            if e.status != 1:
                raise
            try:
                n = need()
            except K.KVarNError:
                raise e from None
            if n <= space.numel():
                raise
        # while a stream captures, memory belongs to its graph: for this call alone
        capturing = self.index >= 0 and torch.cuda.is_current_stream_capturing()
        space = torch.empty(n if capturing else max(n, 2 * space.numel()), dtype=torch.uint8, device=self.device)
        if not capturing:
            self._spaces.append(space)
            # held anew by the streams that calls go to, but for the one that it was allocated on (one given by its
            # address holds nothing)
            self._holders = set()
            if not isinstance(given, int):
                self._holders.add(None if self.index < 0 else K.current_stream(self.device))
                if self.index >= 0:
                    self.mem.record_stream(torch.cuda.current_stream(self.device))
        return call(space, space.numel())

    def decode_attention(self, layer: int, seq_ids: Sequence[int], q: torch.Tensor, out: Optional[torch.Tensor] = None,
                         scale: Optional[float] = None, stream=None, prefix_ids: Optional[Sequence[Optional[int]]] = None,
                         weights: Optional[torch.Tensor] = None) -> torch.Tensor:
        """One query token per sequence over all its cached tokens; q, out: [len(seq_ids)][Hq][D]."""
        self._queries(q, len(seq_ids), out)
        if prefix_ids is not None or weights is not None:
            return self._attend(layer, seq_ids, prefix_ids, None, q, out, scale, weights, stream)
        with K.on_device(self.device, stream) as s:
            if out is None:
                out = torch.empty_like(q)
            K.kvarn_block_decode_attention(self.handle, layer, seq_ids, q, out, self.scale if scale is None else scale, s)
            self._used(stream, s, q, out)
        return out

    def decode_step(self, layer: int, seq_ids: Sequence[int], k: torch.Tensor, v: torch.Tensor, q: torch.Tensor,
                    out: Optional[torch.Tensor] = None, scale: Optional[float] = None, stream=None,
                    prefix_ids: Optional[Sequence[Optional[int]]] = None,
                    weights: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Append one token per sequence and attend its query; k, v: [len(seq_ids)][Hkv][D]."""
        n = len(seq_ids)
        ks, vs = self._tokens(k, n, "k"), self._tokens(v, n, "v")
        self._queries(q, n, out)
        if prefix_ids is not None or weights is not None:
            return self._attend(layer, seq_ids, prefix_ids, [1] * n, q, out, scale, weights, stream, k, ks, v, vs)
        with K.on_device(self.device, stream) as s:
            if out is None:
                out = torch.empty_like(q)
            K.kvarn_block_decode_step(self.handle, layer, seq_ids, k, ks, v, vs, q, out,
                                      self.scale if scale is None else scale, s)
            self._used(stream, s, k, v, q, out)
        return out

    def prefill_attention(self, layer: int, seq_ids: Sequence[int], q_lens: Sequence[int], q: torch.Tensor,
                          out: Optional[torch.Tensor] = None, scale: Optional[float] = None, stream=None,
                          prefix_ids: Optional[Sequence[Optional[int]]] = None) -> torch.Tensor:
        """Causal attention of the last q_lens[i] tokens of each sequence; q, out: [sum(q_lens)][Hq][D]."""
        _same_length(seq_ids, q_lens)
        self._queries(q, sum(q_lens), out)
        if prefix_ids is not None:
            return self._attend(layer, seq_ids, prefix_ids, q_lens, q, out, scale, None, stream)
        with K.on_device(self.device, stream) as s:
            if out is None:
                out = torch.empty_like(q)
            K.kvarn_block_prefill_attention(self.handle, layer, seq_ids, q_lens, q, out,
                                            self.scale if scale is None else scale, s)
            self._used(stream, s, q, out)
        return out

    def prefill(self, layer: int, seq_ids: Sequence[int], n_tokens: Sequence[int], k: torch.Tensor, v: torch.Tensor,
                q: torch.Tensor, out: Optional[torch.Tensor] = None, scale: Optional[float] = None, stream=None,
                prefix_ids: Optional[Sequence[Optional[int]]] = None) -> torch.Tensor:
        """Append a prompt chunk and attend its queries."""
        _same_length(seq_ids, n_tokens)
        rows = sum(n_tokens)
        ks, vs = self._tokens(k, rows, "k"), self._tokens(v, rows, "v")
        self._queries(q, rows, out)
        if prefix_ids is not None:
            return self._attend(layer, seq_ids, prefix_ids, n_tokens, q, out, scale, None, stream, k, ks, v, vs)
        with K.on_device(self.device, stream) as s:
            if out is None:
                out = torch.empty_like(q)
            K.kvarn_block_prefill(self.handle, layer, seq_ids, n_tokens, k, ks, v, vs, q, out,
                                  self.scale if scale is None else scale, s)
            self._used(stream, s, k, v, q, out)
        return out

    def window_weights(self, layer: int, seq_ids: Sequence[int], q_lens: Sequence[int], q: torch.Tensor,
                       weights: torch.Tensor, scale: Optional[float] = None, stream=None,
                       prefix_ids: Optional[Sequence[Optional[int]]] = None):
        """Add to ``weights`` what the last q_lens[i] (128 at most) tokens of each sequence give its blocks, each over
        the tokens up to its own, behind those of its prefix; q: [sum(q_lens)][Hq][D], their queries. Name the prefixes that the
        sequences are attended with: shares of another softmax do not compare with those of ``decode_attention``."""
        _same_length(seq_ids, q_lens)
        self._dense(q, sum(q_lens), "q")
        self._weights(weights)
        prefix_ids = _prefixes(prefix_ids)
        with K.on_device(self.device, stream) as s:
            scale = self.scale if scale is None else scale
            self._in_space(stream, lambda space, n: K.kvarn_block_window_weights_prefixes(
                self.handle, layer, seq_ids, prefix_ids, q_lens, q, scale, weights, space, n, s),
                           lambda: K.kvarn_block_window_workspace_prefixes(self.handle, layer, seq_ids, prefix_ids, q_lens))
            self._used(stream, s, q, weights)

    def evict(self, layer: int, seq_ids: Sequence[int], weights: torch.Tensor, keep: int, first: int = 1, last: int = 1,
              stream=None) -> torch.Tensor:
        """Cut each sequence's full blocks in ``layer`` to ``keep`` where it has more: its first ``first``, its last
        ``last`` and those of most weight, for each KV head its own, in their order; the partial block stays. Returns
        int32 [len(seq_ids)][Hkv][keep]: the number that each block had before (-1: none). ``weights`` move along.
        The blocks that leave are free at once: later appends go to the same stream, as after ``release``."""
        self._weights(weights)
        if not 0 <= keep < 1 << 31:
            raise ValueError(f"keep must be a number of blocks, got {keep}")
        with K.on_device(self.device, stream) as s:
            kept = torch.empty((len(seq_ids), self.kv_heads, keep), dtype=torch.int32, device=self.device)
            K.kvarn_block_evict(self.handle, layer, seq_ids, keep, first, last, weights, kept, s)
            self._used(stream, s, weights, kept)
        return kept

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


def _prefixes(ids):
    """One prefix a sequence as the library takes them: -1 for none."""
    return [-1 if x is None else x for x in ids] if ids is not None and None in ids else ids


def _same_length(seq_ids, counts):
    if len(seq_ids) != len(counts):
        raise ValueError(f"{len(seq_ids)} sequences, but {len(counts)} counts")
