"""Refusals of attention with shared beginnings: on the host, before anything touches a device."""
import ctypes
import math

import pytest
import torch

from causal_attention_score_gb300 import _lib, build_lib
from causal_attention_score_gb300.serving import _KvBatchStruct, _KvCacheStruct

N, SH, AL, UN, WS = (_lib.CSA_ERR_NULL, _lib.CSA_ERR_SHAPE, _lib.CSA_ERR_ALIGN,
                     _lib.CSA_ERR_UNSUPPORTED, _lib.CSA_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _lib.load()


CACHE = dict(k=4096, v=8192, k_scale=64, v_scale=64, pages=4, heads=2, page_tokens=16, head_size=64,
             format=0)
BATCH = dict(offsets=64, lengths=64, table=64, sequences=1, table_width=4, rows=4, max_new=4)
ARGS = dict(out=1 << 24, q=1 << 20, dtype=0, q_heads=4, ot=256, oh=64, qt=256, qh=64, groups=64,
            shared=64, count=1, scale=1.0, ws=1 << 28, size=1 << 32)


def call(lib, cache=None, batch=None, **change):
    c = _KvCacheStruct(*{**CACHE, **(cache or {})}.values())
    b = _KvBatchStruct(*{**BATCH, **(batch or {})}.values())
    a = {**ARGS, **change}
    return lib.cache_attention_shared_forward(
        a["out"], a["q"], a["dtype"], a["q_heads"], a["ot"], a["oh"], a["qt"], a["qh"], ctypes.byref(c),
        ctypes.byref(b), a["groups"], a["shared"], a["count"], a["scale"], a["ws"], a["size"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(cache=dict(k=None)), N), (dict(cache=dict(page_tokens=8)), UN), (dict(cache=dict(head_size=40)), AL),
    (dict(batch=dict(table=None)), N), (dict(batch=dict(rows=0)), SH), (dict(batch=dict(sequences=0)), SH),
    (dict(batch=dict(rows=1 << 29)), UN),
    (dict(out=None), N), (dict(q=None), N), (dict(groups=None), N), (dict(shared=None), N),
    (dict(dtype=2), UN), (dict(q_heads=3), SH), (dict(q_heads=0), SH), (dict(count=0), SH), (dict(count=-2), SH),
    (dict(count=2 ** 31 - 1), UN),
    (dict(scale=math.nan), SH), (dict(scale=math.inf), SH), (dict(out=(1 << 24) + 8), AL), (dict(qt=260), AL),
    (dict(ot=0), SH), (dict(groups=66), AL), (dict(shared=66), AL), (dict(q=(1 << 24) + 128), UN),
    (dict(ws=None), WS), (dict(size=1 << 20), WS), (dict(ws=(1 << 28) + 8), AL),
])
def test_refusals(lib, kw, code):
    assert call(lib, **kw) == code
    assert lib.csa_last_error()


def test_accepted_calls_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for kw in (dict(), dict(out=1 << 20), dict(count=5), dict(scale=-1.0), dict(qt=0)):
        assert call(lib, **kw) == _lib.CSA_ERR_CUDA, kw


def test_workspace_size(lib):
    c, n = _KvCacheStruct(*CACHE.values()), ctypes.c_size_t(7)
    ref = ctypes.byref(c)

    def size(*args):
        rc = lib.cache_attention_shared_workspace_size(ref, *args, ctypes.byref(n))
        return rc, n.value

    assert lib.cache_attention_shared_workspace_size(ref, 4, 1, 1, 1, None) == N
    for args in ((3, 1, 1, 1), (4, 0, 1, 1), (4, 1, 0, 1), (4, 1, 1, 0)):
        assert size(*args) == (SH, 0)
    assert size(4, 1 << 29, 1, 1) == (UN, 0)
    small = size(4, 1, 1, 1)[1]
    assert 0 < small < size(4, 1000, 1, 1)[1] and small < size(4, 1, 1000, 1)[1] and small < size(4, 1, 1, 1000)[1]


def test_modes_of_the_shared_part(lib):
    for mode in (-1, 2):
        assert lib.csa_set_shared_part(mode) == SH
    assert lib.csa_set_shared_part(1) == 0 and lib.csa_set_shared_part(0) == 0
