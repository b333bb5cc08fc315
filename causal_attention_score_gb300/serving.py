"""Rotary positions, the paged 8-bit cache of keys and values, and attention over it:
Python binding of their C entry points (argument marshalling only, as in ops.py).

``RotaryTable``, ``KvCache`` and ``KvBatch`` are checked and marshalled once and may be
used for any number of calls; each keeps references to its tensors.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from .ops import _need

CSA_BF16, CSA_F16, CSA_F32 = 0, 1, 2
CSA_KV_INT8, CSA_KV_E4M3 = 0, 1
_DTYPE = {torch.bfloat16: CSA_BF16, torch.float16: CSA_F16, torch.float32: CSA_F32}
_HALF = (torch.bfloat16, torch.float16)
_FORMAT = {torch.int8: CSA_KV_INT8, torch.float8_e4m3fn: CSA_KV_E4M3}
_SCALING = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}


def _on_device(t: torch.Tensor, name: str) -> None:
    """Every call works on the current device: its tensors must be there."""
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, but calls work on the current device "
                         f"cuda:{torch.cuda.current_device()}")


def _stream_ptr(stream) -> int:
    """The raw handle of ``stream``, by default of the current device's current stream
    (asked for directly: building a torch.cuda.Stream takes as long as a launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _rows(t: torch.Tensor, name: str, shape, dtypes) -> tuple[int, int]:
    """(token stride, head stride) of a [tokens, heads, size] tensor of the given shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    token, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    _on_device(t, name)
    # the stride of a dimension of one entry means nothing
    n, heads, size = shape
    head = head if heads > 1 else size
    return (token if n > 1 else heads * size), head


def _same_storage(tensors, ptrs, what: str) -> None:
    for t, p in zip(tensors, ptrs):
        if t.data_ptr() != p:
            raise ValueError(f"a tensor of this {what} no longer has the storage it was made "
                             f"with; make a new {what}")


class RotaryTable:
    """Frequencies of rotary positions, on the device, and the amplitude of the result.

    ``scaling``: "none", "linear" (``factor``), "ntk" (``factor``) or "by_parts" (``factor``,
    ``original_length``, ``slow``, ``fast``); see csa_rotary_turns in include/csa.h.
    """

    def __init__(self, rot_dim: int, base: float = 10000.0, scaling: str = "none",
                 factor: float = 1.0, original_length: float = 0.0, slow: float = 1.0,
                 fast: float = 32.0, amplitude: float = 1.0, device="cuda"):
        if scaling not in _SCALING:
            raise ValueError(f"unknown scaling {scaling!r}: one of {tuple(_SCALING)}")
        host = (ctypes.c_uint64 * max(1, rot_dim // 2))()
        _lib.check(_lib.load().csa_rotary_turns(host, rot_dim, base, _SCALING[scaling], factor,
                                                original_length, slow, fast), "csa_rotary_turns")
        self.rot_dim = int(rot_dim)
        self.amplitude = float(amplitude)
        signed = [v - (1 << 64) if v >> 63 else v for v in host]
        self.turns = torch.tensor(signed, dtype=torch.int64).to(device)


def _rotary(which: str, out, x, table, positions, start, period, interleaved, stream) -> None:
    if x.dim() == 4:  # (B, T, heads, size) whose batches follow one another
        if x.shape[0] > 1 and x.stride(0) != x.shape[1] * x.stride(1):
            raise ValueError("x: a 4-D tensor's batches must follow one another")
        if out.shape[0] > 1 and out.stride(0) != out.shape[1] * out.stride(1):
            raise ValueError("out: a 4-D tensor's batches must follow one another")
        if out.shape != x.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(x.shape)}")
        B, T = x.shape[0], x.shape[1]
        x = x.as_strided((B * T, x.shape[2], x.shape[3]), x.stride()[1:])
        out = out.as_strided(x.shape, out.stride()[1:])
    if x.dim() != 3:
        raise ValueError("x must be [tokens, heads, size] or [B, T, heads, size]")
    xt, xh = _rows(x, "x", x.shape, tuple(_DTYPE))
    ot, oh = _rows(out, "out", x.shape, (x.dtype,))
    n, heads, size = x.shape
    pos = None
    if positions is not None:
        _need(positions, "positions", torch.int32, n)
        _on_device(positions, "positions")
        pos = positions.data_ptr()
    _on_device(table.turns, "the rotary table")
    lib = _lib.load()
    fn = lib.rotary_backward if which == "rotary_backward" else lib.rotary_forward
    _lib.check(fn(out.data_ptr(), x.data_ptr(), _DTYPE[x.dtype], n, heads, size, table.rot_dim,
                  ot, oh, xt, xh, table.turns.data_ptr(), table.amplitude, pos, start, period,
                  1 if interleaved else 0, _stream_ptr(stream)), which)


def rotary_forward(out: torch.Tensor, x: torch.Tensor, table: RotaryTable, positions=None,
                   start: int = 0, period: int = 0, interleaved: bool = False,
                   stream=None) -> None:
    """Turns every head's first ``table.rot_dim`` elements by its token's position into
    ``out`` (``x`` itself, or a tensor apart from it): [tokens, heads, size] or
    [B, T, heads, size], bf16, fp16 or fp32. ``positions`` int32, one per token (negative:
    padding, left as it is), or None for ``start + (t % period if period else t)``; see
    rotary_forward in include/csa.h."""
    _rotary("rotary_forward", out, x, table, positions, start, period, interleaved, stream)


def rotary_backward(dx: torch.Tensor, dy: torch.Tensor, table: RotaryTable, positions=None,
                    start: int = 0, period: int = 0, interleaved: bool = False,
                    stream=None) -> None:
    """The gradient of rotary_forward: ``dy`` turned by the opposite angles into ``dx``."""
    _rotary("rotary_backward", dx, dy, table, positions, start, period, interleaved, stream)


def rotary_qkv(qkv: torch.Tensor, table: RotaryTable, start: int = 0, interleaved: bool = False,
               backward: bool = False, stream=None) -> None:
    """Rotates the Q and K of packed ``qkv`` (B, T, 3, NH, HS) in place, token t of each
    batch at position ``start + t``: what trimul and causal_softmax then read.
    ``backward`` turns the gradient of such a tensor back."""
    B, T, three, NH, HS = qkv.shape
    if three != 3 or not qkv.is_contiguous():
        raise ValueError("qkv must be contiguous with shape (B, T, 3, NH, HS)")
    qk = qkv.view(B * T, 3 * NH, HS)[:, : 2 * NH]
    _rotary("rotary_backward" if backward else "rotary_forward", qk, qk, table, None, start, T,
            interleaved, stream)


class _KvCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int), ("heads", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("head_size", ctypes.c_int),
                ("format", ctypes.c_int)]


class _KvBatchStruct(ctypes.Structure):
    _fields_ = [("offsets", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("sequences", ctypes.c_int),
                ("table_width", ctypes.c_int), ("rows", ctypes.c_int), ("max_new", ctypes.c_int)]


class KvCache:
    """A paged cache of keys and values in 8 bits (csa_kv_cache in include/csa.h): codes
    ``k`` and ``v`` [pages, heads, page_tokens, head_size], torch.int8 or
    torch.float8_e4m3fn, and fp32 scales ``k_scale`` and ``v_scale`` [pages, heads]."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        if k.dim() != 4:
            raise ValueError("k must be [pages, heads, page_tokens, head_size]")
        if k.dtype not in _FORMAT:
            raise TypeError(f"codes must be int8 or float8_e4m3fn, got {k.dtype}")
        pages, heads, page_tokens, head_size = k.shape
        for name, t in (("k", k), ("v", v)):
            _need(t, name, k.dtype, k.numel())
            if t.shape != k.shape:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(k.shape)}")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(t, name, torch.float32, pages * heads)
        for t in (v, k_scale, v_scale):
            if t.device != k.device:
                raise ValueError("the tensors of a cache must be on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_tokens, self.head_size = pages, heads, page_tokens, head_size
        self._tensors = (k, v, k_scale, v_scale)
        self._ptrs = [t.data_ptr() for t in self._tensors]
        self._struct = _KvCacheStruct(*self._ptrs, pages, heads, page_tokens, head_size,
                                      _FORMAT[k.dtype])
        self._ref = ctypes.addressof(self._struct)
        # page and head sizes the library does not take are refused here
        n = ctypes.c_size_t(0)
        _lib.check(_lib.load().cache_attention_workspace_size(self._ref, heads, ctypes.byref(n)),
                   "KvCache")

    @classmethod
    def empty(cls, pages: int, heads: int, page_tokens: int, head_size: int,
              dtype: torch.dtype = torch.int8, device="cuda") -> "KvCache":
        """A new cache (its content is never interpreted before it is written)."""
        shape = (pages, heads, page_tokens, head_size)
        codes = [torch.empty(shape, dtype=dtype, device=device) for _ in range(2)]
        scales = [torch.empty(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales)

    def _pointer(self) -> int:
        _same_storage(self._tensors, self._ptrs, "KvCache")
        _on_device(self.k, "the cache")
        return self._ref


class KvBatch:
    """Which rows of a call are which tokens (csa_kv_batch in include/csa.h): int32 tensors
    ``offsets`` [S + 1], ``lengths`` [S] (including the rows) and ``table`` [S, width], which
    may change between calls in place. ``rows`` is the number of rows the calls' tensors
    have, ``max_new`` at least any sequence's rows (default: ``rows``)."""

    def __init__(self, offsets: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
                 rows: int, max_new: int | None = None):
        if table.dim() != 2:
            raise ValueError("table must be [sequences, width]")
        S, width = table.shape
        _need(offsets, "offsets", torch.int32, S + 1)
        _need(lengths, "lengths", torch.int32, S)
        _need(table, "table", torch.int32, S * width)
        if lengths.device != offsets.device or table.device != offsets.device:
            raise ValueError("the tensors of a batch must be on one device")
        self.offsets, self.lengths, self.table = offsets, lengths, table
        self.rows, self.max_new = int(rows), int(rows if max_new is None else max_new)
        self._tensors = (offsets, lengths, table)
        self._ptrs = [t.data_ptr() for t in self._tensors]
        self._struct = _KvBatchStruct(*self._ptrs, S, width, self.rows, self.max_new)
        self._ref = ctypes.addressof(self._struct)

    def _pointer(self) -> int:
        _same_storage(self._tensors, self._ptrs, "KvBatch")
        _on_device(self.offsets, "the batch")
        return self._ref


def kv_cache_write(cache: KvCache, batch: KvBatch, k: torch.Tensor, v: torch.Tensor,
                   stream=None) -> None:
    """Quantises rows ``k`` and ``v`` [rows, heads, head_size] (bf16 or fp16) into the cache,
    as the last tokens of the batch's sequences; see kv_cache_write in include/csa.h."""
    shape = (batch.rows, cache.heads, cache.head_size)
    kt, kh = _rows(k, "k", shape, _HALF)
    vt, vh = _rows(v, "v", shape, (k.dtype,))
    _lib.check(_lib.load().kv_cache_write(cache._pointer(), batch._pointer(), k.data_ptr(),
                                          v.data_ptr(), _DTYPE[k.dtype], kt, kh, vt, vh,
                                          _stream_ptr(stream)), "kv_cache_write")


def kv_cache_read(k: torch.Tensor, v: torch.Tensor, cache: KvCache, batch: KvBatch,
                  stream=None) -> None:
    """The values of the batch's rows (the last tokens of its sequences) into ``k`` and ``v``
    [rows, heads, head_size], bf16, fp16 or fp32; see kv_cache_read in include/csa.h."""
    shape = (batch.rows, cache.heads, cache.head_size)
    kt, kh = _rows(k, "k", shape, tuple(_DTYPE))
    vt, vh = _rows(v, "v", shape, (k.dtype,))
    _lib.check(_lib.load().kv_cache_read(k.data_ptr(), v.data_ptr(), _DTYPE[k.dtype], kt, kh, vt,
                                         vh, cache._pointer(), batch._pointer(),
                                         _stream_ptr(stream)), "kv_cache_read")


def cache_attention_workspace_size(cache: KvCache, batch: KvBatch, q_heads: int) -> int:
    """Bytes of workspace ``cache_attention_forward`` needs (the same for any batch)."""
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().cache_attention_workspace_size(cache._pointer(), q_heads,
                                                          ctypes.byref(n)),
               "cache_attention_workspace_size")
    return int(n.value)


def cache_attention_forward(out: torch.Tensor, q: torch.Tensor, cache: KvCache, batch: KvBatch,
                            scale: float | None = None, window: int = 0, sinks: int = 0,
                            workspace: torch.Tensor | None = None, stream=None) -> None:
    """Attention of the rows ``q`` [rows, q_heads, head_size] (bf16 or fp16) over the cache
    into ``out``: row p sees keys t <= p, with a ``window`` those with p - t < window or
    t < ``sinks``. ``scale`` defaults to 1/sqrt(head_size). Without a ``workspace`` (at least
    cache_attention_workspace_size bytes) one is taken from torch's caching allocator on the
    call's stream. See cache_attention_forward in include/csa.h."""
    if q.dim() != 3:
        raise ValueError("q must be [rows, q_heads, head_size]")
    shape = (batch.rows, q.shape[1], cache.head_size)
    qt, qh = _rows(q, "q", shape, _HALF)
    ot, oh = _rows(out, "out", shape, (q.dtype,))
    ref = cache._pointer()
    if workspace is None:
        if stream is None:
            st = torch.cuda.current_stream(q.device)
        elif isinstance(stream, torch.cuda.Stream):
            st = stream
        else:
            st = torch.cuda.ExternalStream(int(stream), device=q.device)
        with torch.cuda.stream(st):
            workspace = torch.empty(cache_attention_workspace_size(cache, batch, q.shape[1]),
                                    dtype=torch.uint8, device=q.device)
        stream = st
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    else:
        _on_device(workspace, "workspace")
    _lib.check(_lib.load().cache_attention_forward(
        out.data_ptr(), q.data_ptr(), _DTYPE[q.dtype], q.shape[1], ot, oh, qt, qh, ref,
        batch._pointer(), 1.0 / math.sqrt(cache.head_size) if scale is None else scale, window,
        sinks, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream_ptr(stream)), "cache_attention_forward")


def cache_attention(q: torch.Tensor, cache: KvCache, batch: KvBatch, scale: float | None = None,
                    window: int = 0, sinks: int = 0, stream=None) -> torch.Tensor:
    """Allocating form of cache_attention_forward; rows of no sequence are zero."""
    out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    cache_attention_forward(out, q, cache, batch, scale, window, sinks, None, stream)
    return out
