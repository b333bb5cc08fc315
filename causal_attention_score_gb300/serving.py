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
from .ops import _allocate, _need, _torch_stream

CSA_BF16, CSA_F16, CSA_F32 = 0, 1, 2
CSA_KV_INT8, CSA_KV_E4M3 = 0, 1
_DTYPE = {torch.bfloat16: CSA_BF16, torch.float16: CSA_F16, torch.float32: CSA_F32}
_HALF = (torch.bfloat16, torch.float16)
_FORMAT = {torch.int8: CSA_KV_INT8, torch.float8_e4m3fn: CSA_KV_E4M3}
_SCALING = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}


_ANY = tuple(_DTYPE)
_get_device, _get_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _elsewhere(device, name: str) -> ValueError:
    """Every call works on the current device: its tensors must be there."""
    return ValueError(f"{name} is on {device}, but calls work on the current device "
                      f"cuda:{torch.cuda.current_device()}")


def _device_of(t: torch.Tensor, name: str) -> int:
    """The current device, where ``t`` must be."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _get_device():
        raise _elsewhere(t.device, name)
    return dev


def _stream_ptr(stream, dev: int) -> int:
    """The raw handle of ``stream``, by default of device ``dev``'s current stream
    (asked for directly: building a torch.cuda.Stream takes as long as a launch)."""
    if stream is None:
        return _get_stream(dev)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _rows(t: torch.Tensor, name: str, shape, dtypes, dev: int) -> tuple[int, int]:
    """(token stride, head stride) of a [tokens, heads, size] tensor of the given shape on
    device ``dev``."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise _elsewhere(t.device, name)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    token, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    # the stride of a dimension of one entry means nothing
    n, heads, size = shape
    return (token if n > 1 else heads * size), (head if heads > 1 else size)


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


def _flat(t: torch.Tensor, name: str) -> torch.Tensor:
    """(B, T, heads, size) whose tokens are one stride apart, through all batches, as
    [B * T, heads, size]; with one token a batch that is the batches' stride."""
    B, T, heads, size = t.shape
    batch, token, head, one = t.stride()
    if T == 1:
        token = batch
    elif B > 1 and batch != T * token:
        raise ValueError(f"{name}: a 4-D tensor's batches must follow one another")
    return t.as_strided((B * T, heads, size), (token, head, one))


def _rotary(which: str, out, x, table, positions, start, period, interleaved, stream) -> None:
    if x.dim() == 4:
        if out.shape != x.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(x.shape)}")
        x, out = _flat(x, "x"), _flat(out, "out")
    if x.dim() != 3:
        raise ValueError("x must be [tokens, heads, size] or [B, T, heads, size]")
    dev = _device_of(x, "x")
    shape, dtype = x.shape, x.dtype
    xt, xh = _rows(x, "x", shape, _ANY, dev)
    ot, oh = _rows(out, "out", shape, (dtype,), dev)
    n, heads, size = shape
    pos = None
    if positions is not None:
        _need(positions, "positions", torch.int32, n)
        if positions.get_device() != dev:
            raise _elsewhere(positions.device, "positions")
        pos = positions.data_ptr()
    turns = table.turns
    if turns.get_device() != dev:
        raise _elsewhere(turns.device, "the rotary table")
    lib = _lib._lib or _lib.load()
    fn = lib.rotary_backward if which == "rotary_backward" else lib.rotary_forward
    rc = fn(out.data_ptr(), x.data_ptr(), _DTYPE[dtype], n, heads, size, table.rot_dim, ot, oh,
            xt, xh, turns.data_ptr(), table.amplitude, pos, start, period,
            1 if interleaved else 0, _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, which)


def rotary_forward(out: torch.Tensor, x: torch.Tensor, table: RotaryTable, positions=None,
                   start: int = 0, period: int = 0, interleaved: bool = False,
                   stream=None) -> None:
    """Turns every head's first ``table.rot_dim`` elements by its token's position into
    ``out`` (``x`` itself, or a tensor apart from it): [tokens, heads, size] or
    [B, T, heads, size], bf16, fp16 or fp32. ``positions`` int32, one per token (negative:
    padding, left as it is), or None for ``start + (t % period if period else t)``, t counting
    the tokens through all batches (``period=T`` starts each batch anew); see rotary_forward
    in include/csa.h."""
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


class _Marshalled:
    """Tensors (``_tensors``) whose addresses were written into a struct once."""

    def _pointer(self, dev: int) -> int:
        """Address of the struct, for a call on device ``dev``."""
        if [t.data_ptr() for t in self._tensors] != self._ptrs:
            raise ValueError(f"a tensor of this {type(self).__name__} no longer has the storage it "
                             f"was made with; make a new {type(self).__name__}")
        if self._device != dev:
            raise _elsewhere(self._tensors[0].device, f"the {type(self).__name__}")
        return self._ref


class KvCache(_Marshalled):
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
        self._device = k.get_device()
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


class KvBatch(_Marshalled):
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
        self._device = offsets.get_device()
        self._struct = _KvBatchStruct(*self._ptrs, S, width, self.rows, self.max_new)
        self._ref = ctypes.addressof(self._struct)


def kv_cache_write(cache: KvCache, batch: KvBatch, k: torch.Tensor, v: torch.Tensor,
                   stream=None) -> None:
    """Quantises rows ``k`` and ``v`` [rows, heads, head_size] (bf16 or fp16) into the cache,
    as the last tokens of the batch's sequences; see kv_cache_write in include/csa.h."""
    dev, dtype = _device_of(k, "k"), k.dtype
    shape = (batch.rows, cache.heads, cache.head_size)
    kt, kh = _rows(k, "k", shape, _HALF, dev)
    vt, vh = _rows(v, "v", shape, (dtype,), dev)
    rc = (_lib._lib or _lib.load()).kv_cache_write(
        cache._pointer(dev), batch._pointer(dev), k.data_ptr(), v.data_ptr(), _DTYPE[dtype], kt, kh,
        vt, vh, _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "kv_cache_write")


def kv_cache_read(k: torch.Tensor, v: torch.Tensor, cache: KvCache, batch: KvBatch,
                  stream=None) -> None:
    """The values of the batch's rows (the last tokens of its sequences) into ``k`` and ``v``
    [rows, heads, head_size], bf16, fp16 or fp32; see kv_cache_read in include/csa.h."""
    dev, dtype = _device_of(k, "k"), k.dtype
    shape = (batch.rows, cache.heads, cache.head_size)
    kt, kh = _rows(k, "k", shape, _ANY, dev)
    vt, vh = _rows(v, "v", shape, (dtype,), dev)
    rc = (_lib._lib or _lib.load()).kv_cache_read(
        k.data_ptr(), v.data_ptr(), _DTYPE[dtype], kt, kh, vt, vh, cache._pointer(dev),
        batch._pointer(dev), _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "kv_cache_read")


def cache_attention_workspace_size(cache: KvCache, batch: KvBatch, q_heads: int) -> int:
    """Bytes of workspace ``cache_attention_forward`` needs (the same for any batch)."""
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().cache_attention_workspace_size(cache._ref, q_heads,
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
    dev, dtype, q_heads = _device_of(q, "q"), q.dtype, q.shape[1]
    shape = (batch.rows, q_heads, cache.head_size)
    qt, qh = _rows(q, "q", shape, _HALF, dev)
    ot, oh = _rows(out, "out", shape, (dtype,), dev)
    ref = cache._pointer(dev)
    if workspace is None:
        size = cache_attention_workspace_size(cache, batch, q_heads)
        if stream is None:
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
        else:
            stream = _torch_stream(stream, q.device)
            with torch.cuda.stream(stream):
                workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev:
        if not workspace.is_cuda:
            raise ValueError("workspace must be a contiguous CUDA tensor")
        raise _elsewhere(workspace.device, "workspace")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    rc = (_lib._lib or _lib.load()).cache_attention_forward(
        out.data_ptr(), q.data_ptr(), _DTYPE[dtype], q_heads, ot, oh, qt, qh, ref,
        batch._pointer(dev), 1.0 / math.sqrt(cache.head_size) if scale is None else scale, window,
        sinks, workspace.data_ptr(), workspace.nbytes, _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "cache_attention_forward")


def cache_attention(q: torch.Tensor, cache: KvCache, batch: KvBatch, scale: float | None = None,
                    window: int = 0, sinks: int = 0, stream=None) -> torch.Tensor:
    """Allocating form of cache_attention_forward; rows of no sequence are zero. The output is
    allocated and cleared on the call's stream."""
    out = _allocate(torch.zeros, q.shape, q.dtype, q.device, stream)
    cache_attention_forward(out, q, cache, batch, scale, window, sinks, None, stream)
    return out
