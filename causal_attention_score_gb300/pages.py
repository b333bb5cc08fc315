"""The books of a paged cache (which pages each sequence has) and the calls that keep them:
Python binding of their C entry points (argument marshalling only, as in ops.py)."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .ops import _need
from .serving import (KvCache, _elsewhere, _get_device, _given, _Marshalled, _stream_ptr,
                      _workspace)


class _KvPagesStruct(ctypes.Structure):
    _fields_ = [("refs", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("pages", ctypes.c_int), ("sequences", ctypes.c_int),
                ("table_width", ctypes.c_int), ("page_tokens", ctypes.c_int)]


def _apart(spans) -> bool:
    """Whether no two of ``spans`` [(begin, end)] meet."""
    last = 0
    for begin, end in sorted(spans):
        if begin < last:
            return False
        last = end
    return True


class KvPages(_Marshalled):
    """The books of a cache (csa_kv_pages in include/csa.h): int32 tensors ``refs`` [pages] (how
    many table entries name a page; 0: free), ``lengths`` [S] (tokens of each place's sequence; 0:
    none) and ``table`` [S, width] (its pages). ``KvBatch(offsets, pages.lengths, pages.table, ...)``
    is a batch over all places."""

    def __init__(self, refs: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
                 page_tokens: int):
        if table.dim() != 2:
            raise ValueError("table must be [sequences, width]")
        if refs.dim() != 1:
            raise ValueError("refs must be [pages]")
        S, width = table.shape
        _need(refs, "refs", torch.int32, refs.numel())
        _need(lengths, "lengths", torch.int32, S)
        _need(table, "table", torch.int32, S * width)
        if lengths.device != refs.device or table.device != refs.device:
            raise ValueError("the tensors of the pages must be on one device")
        self.refs, self.lengths, self.table = refs, lengths, table
        self.page_tokens = int(page_tokens)
        self._tensors = (refs, lengths, table)
        self._ptrs = [t.data_ptr() for t in self._tensors]
        self._spans = [(p, p + 4 * t.numel()) for p, t in zip(self._ptrs, self._tensors)]
        if not _apart(self._spans):
            raise ValueError("refs, lengths and table must not overlap")
        self._device = refs.get_device()
        self._struct = _KvPagesStruct(*self._ptrs, refs.numel(), S, width, self.page_tokens)
        self._ref = ctypes.addressof(self._struct)
        n = ctypes.c_size_t(0)  # (sizes that the library does not take are refused here)
        _lib.check(_lib.load().kv_pages_workspace_size(self._ref, 0, ctypes.byref(n)), "KvPages")

    @classmethod
    def empty(cls, cache: KvCache, sequences: int, table_width: int) -> "KvPages":
        """Books of ``cache`` with every page free, for up to ``sequences`` sequences of at most
        ``table_width`` pages."""
        def zeros(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=cache.k.device)

        return cls(zeros(cache.pages), zeros(sequences), zeros(sequences, table_width),
                   cache.page_tokens)


def kv_pages_workspace_size(pages: KvPages, n: int) -> int:
    """Bytes of workspace that kv_pages_extend and kv_cache_fork with up to ``n`` entries, and
    kv_cache_compact, need."""
    size = ctypes.c_size_t(0)
    _lib.check(_lib.load().kv_pages_workspace_size(pages._ref, n, ctypes.byref(size)),
               "kv_pages_workspace_size")
    return int(size.value)


def _list(t: torch.Tensor, name: str, n: int, dev: int) -> int:
    """Address of an int32 list of n entries on device ``dev``."""
    if (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.get_device() == dev
            and t.numel() == n and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise _elsewhere(t.device, name)
    _need(t, name, torch.int32, n)
    return t.data_ptr()


def _entries(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t.numel()


def _scratch(workspace, pages: KvPages, n: int, stream, dev: int):
    """(workspace, stream): the caller's workspace checked, or one of our own."""
    if workspace is None:
        return _workspace(kv_pages_workspace_size(pages, n), pages.refs.device, stream)
    _given(workspace, dev)
    return workspace, stream


def kv_pages_extend(pages: KvPages, sequences: torch.Tensor, more: torch.Tensor, workspace=None,
                    stream=None) -> None:
    """Room for ``more[i]`` more tokens of sequence ``sequences[i]`` (int32 tensors): lengths grow,
    free pages are given to new blocks, lowest number first; see kv_pages_extend in
    include/csa.h."""
    dev, n = _get_device(), _entries(sequences, "sequences")
    ref = pages._pointer(dev)
    at, count = _list(sequences, "sequences", n, dev), _list(more, "more", n, dev)
    workspace, stream = _scratch(workspace, pages, n, stream, dev)
    rc = (_lib._lib or _lib.load()).kv_pages_extend(
        ref, at, count, n, workspace.data_ptr(), workspace.nbytes, _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "kv_pages_extend")


def kv_cache_fork(cache: KvCache, pages: KvPages, parents: torch.Tensor, children: torch.Tensor,
                  tokens: torch.Tensor | None = None, workspace=None, stream=None) -> None:
    """Place ``children[i]`` (of length 0) becomes a sequence of the first ``tokens[i]`` tokens of
    ``parents[i]`` (None: all of them): whole pages are shared, the written part of a last one is
    copied; see kv_cache_fork in include/csa.h."""
    dev, n = _get_device(), _entries(children, "children")
    ref, books = cache._pointer(dev), pages._pointer(dev)
    p, c = _list(parents, "parents", n, dev), _list(children, "children", n, dev)
    t = None if tokens is None else _list(tokens, "tokens", n, dev)
    workspace, stream = _scratch(workspace, pages, n, stream, dev)
    rc = (_lib._lib or _lib.load()).kv_cache_fork(
        ref, books, p, c, t, n, workspace.data_ptr(), workspace.nbytes, _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "kv_cache_fork")


def kv_pages_free(pages: KvPages, sequences: torch.Tensor, stream=None) -> None:
    """The sequences at ``sequences`` (int32) end: their lengths become 0, and pages that no other
    names are free; see kv_pages_free in include/csa.h."""
    dev, n = _get_device(), _entries(sequences, "sequences")
    rc = (_lib._lib or _lib.load()).kv_pages_free(
        pages._pointer(dev), _list(sequences, "sequences", n, dev), n, _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "kv_pages_free")


def kv_cache_copy(to: KvCache, from_: KvCache, to_pages: torch.Tensor, from_pages: torch.Tensor,
                  stream=None) -> None:
    """Page ``to_pages[i]`` of cache ``to`` becomes a copy of page ``from_pages[i]`` of ``from_``
    (int32 tensors; the caches' pages are alike); see kv_cache_copy in include/csa.h."""
    dev, n = _get_device(), _entries(to_pages, "to_pages")
    rc = (_lib._lib or _lib.load()).kv_cache_copy(
        to._pointer(dev), from_._pointer(dev), _list(to_pages, "to_pages", n, dev),
        _list(from_pages, "from_pages", n, dev), n, _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "kv_cache_copy")


def kv_cache_compact(cache: KvCache, pages: KvPages, moves: torch.Tensor, in_use: torch.Tensor,
                     workspace=None, stream=None) -> None:
    """Moves the pages in use to the lowest numbers, with the table's entries: ``moves`` (int32
    [pages]) becomes each page's new number (-1: it was free), ``in_use`` (int32 [1]) how many
    there are; see kv_cache_compact in include/csa.h."""
    dev = _get_device()
    ref, books = cache._pointer(dev), pages._pointer(dev)
    m, u = _list(moves, "moves", pages.refs.numel(), dev), _list(in_use, "in_use", 1, dev)
    if not _apart([*pages._spans, (m, m + 4 * pages.refs.numel()), (u, u + 4)]):
        raise ValueError("moves and in_use must not overlap the books or each other")
    workspace, stream = _scratch(workspace, pages, 0, stream, dev)
    rc = (_lib._lib or _lib.load()).kv_cache_compact(
        ref, books, m, u, workspace.data_ptr(), workspace.nbytes, _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "kv_cache_compact")
