"""Refusals of the calls on a cache's books: on the host, before anything touches a device."""
import ctypes

import pytest
import torch

import causal_attention_score_gb300 as csa
from causal_attention_score_gb300 import _lib, build_lib
from causal_attention_score_gb300.pages import _KvPagesStruct
from causal_attention_score_gb300.serving import _KvCacheStruct

N, SH, AL, UN, WS = (_lib.CSA_ERR_NULL, _lib.CSA_ERR_SHAPE, _lib.CSA_ERR_ALIGN,
                     _lib.CSA_ERR_UNSUPPORTED, _lib.CSA_ERR_WORKSPACE)
BIG = 1 << 32


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _lib.load()


CACHE = dict(k=4096, v=8192, k_scale=64, v_scale=64, pages=4, heads=2, page_tokens=16, head_size=64,
             format=0)
PAGES = dict(refs=64, lengths=64, table=64, pages=4, sequences=3, table_width=4, page_tokens=16)


ALL = ("extend", "fork", "free", "copy", "compact")


def calls(lib, which, cache=None, pages=None, other=None, a=64, b=64, c=64, n=2, ws=1 << 20, size=BIG):
    """The calls in `which` with these arguments: {name: status}. (Those that are not to be refused
    are not made where there is a device: the addresses are made up.)"""
    k = _KvCacheStruct(*{**CACHE, **(cache or {})}.values())
    o = _KvCacheStruct(*{**CACHE, **(cache or {}), **(other or {})}.values())
    p = _KvPagesStruct(*{**PAGES, **(pages or {})}.values())
    k, o, p = ctypes.byref(k), ctypes.byref(o), ctypes.byref(p)
    make = {"extend": lambda: lib.kv_pages_extend(p, a, b, n, ws, size, None),
            "fork": lambda: lib.kv_cache_fork(k, p, a, b, c, n, ws, size, None),
            "free": lambda: lib.kv_pages_free(p, a, n, None),
            "copy": lambda: lib.kv_cache_copy(o, k, a, b, n, None),
            "compact": lambda: lib.kv_cache_compact(k, p, a, b, ws, size, None)}
    return {name: make[name]() for name in which}


OF_PAGES, OF_CACHE = ("extend", "fork", "free", "compact"), ("fork", "copy", "compact")


@pytest.mark.parametrize("kw,code,which", [
    (dict(pages=dict(refs=None)), N, OF_PAGES), (dict(pages=dict(lengths=None)), N, OF_PAGES),
    (dict(pages=dict(table=None)), N, OF_PAGES), (dict(pages=dict(sequences=0)), SH, OF_PAGES),
    (dict(pages=dict(table_width=-1)), SH, OF_PAGES), (dict(pages=dict(refs=66)), AL, OF_PAGES),
    (dict(pages=dict(page_tokens=8), cache=dict(page_tokens=8)), UN, OF_PAGES),
    (dict(pages=dict(pages=0)), SH, ("extend", "free")),
    (dict(pages=dict(pages=(1 << 30) + 1)), UN, ("extend", "free")),
    (dict(pages=dict(pages=5)), SH, ("fork", "compact")),
    (dict(pages=dict(page_tokens=32)), SH, ("fork", "compact")),
    (dict(cache=dict(k=None)), N, OF_CACHE), (dict(cache=dict(v_scale=None)), N, OF_CACHE),
    (dict(cache=dict(heads=0)), SH, OF_CACHE), (dict(cache=dict(head_size=40)), AL, OF_CACHE),
    (dict(cache=dict(format=7)), UN, OF_CACHE), (dict(cache=dict(k=4104)), AL, OF_CACHE),
    (dict(cache=dict(heads=1 << 21)), UN, OF_CACHE),
    (dict(other=dict(heads=3)), SH, ("copy",)), (dict(other=dict(page_tokens=32)), SH, ("copy",)),
    (dict(other=dict(head_size=32)), SH, ("copy",)), (dict(other=dict(format=1)), SH, ("copy",)),
    (dict(other=dict(v=None)), N, ("copy",)),
    (dict(a=None), N, ("extend", "fork", "free", "copy", "compact")),
    (dict(b=None), N, ("extend", "fork", "copy", "compact")),
    (dict(a=66), AL, ("extend", "fork", "free", "copy", "compact")),
    (dict(b=66), AL, ("extend", "fork", "copy", "compact")), (dict(c=66), AL, ("fork",)),
    (dict(n=0), SH, ("extend", "fork", "free", "copy")),
    (dict(n=-1), SH, ("extend", "fork", "free", "copy")),
    (dict(ws=None), WS, ("extend", "fork", "compact")),
    (dict(size=4000), WS, ("extend", "fork", "compact")),
    (dict(ws=(1 << 20) + 8), AL, ("extend", "fork", "compact")),
])
def test_refusals(lib, kw, code, which):
    got = calls(lib, which, **kw)
    assert set(got.values()) == {code}, got


def test_null_structs_and_workspace_size(lib):
    size = ctypes.c_size_t(5)
    p = _KvPagesStruct(*PAGES.values())
    assert lib.kv_pages_workspace_size(None, 1, ctypes.byref(size)) == N and size.value == 0
    assert lib.kv_pages_workspace_size(ctypes.byref(p), 1, None) == N
    assert lib.kv_pages_workspace_size(ctypes.byref(p), -1, ctypes.byref(size)) == SH
    sizes = []
    for n in (0, 1, 1000):
        assert lib.kv_pages_workspace_size(ctypes.byref(p), n, ctypes.byref(size)) == 0
        sizes.append(size.value)
    assert sizes[0] < sizes[1] < sizes[2]
    assert lib.kv_pages_extend(None, 64, 64, 1, 64, BIG, None) == N
    assert lib.kv_cache_fork(None, ctypes.byref(p), 64, 64, None, 1, 64, BIG, None) == N
    assert lib.kv_cache_copy(None, None, 64, 64, 1, None) == N


def test_accepted_calls_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for kw in (dict(), dict(c=None), dict(n=1), dict(other=dict(pages=9))):
        assert set(calls(lib, ALL, **kw).values()) == {_lib.CSA_ERR_CUDA}, kw


def test_binding_refusals():
    t = torch.zeros((4,), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        csa.KvPages(t, t[:2], torch.zeros((2, 3), dtype=torch.int32), 16)
    with pytest.raises(ValueError, match="sequences, width"):
        csa.KvPages(t, t, t, 16)
    assert csa.CSA_ERR_PAGES == -13
