"""Refusals of the rotary, cache and cache-attention calls, and csa_rotary_turns: on the host,
before anything touches a device."""
import ctypes
import math

import pytest
import torch

import causal_attention_score_gb300 as csa
from causal_attention_score_gb300 import _lib, build_lib
from causal_attention_score_gb300.serving import _KvBatchStruct, _KvCacheStruct

N, SH, AL, UN = (_lib.CSA_ERR_NULL, _lib.CSA_ERR_SHAPE, _lib.CSA_ERR_ALIGN,
                 _lib.CSA_ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _lib.load()


ROT = dict(out=1 << 20, x=1 << 24, dtype=0, tokens=4, heads=2, size=64, rd=64, ot=128, oh=64, xt=128,
           xh=64, turns=4096, amp=1.0, pos=None, start=0, period=0, inter=0, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(out=None), N), (dict(x=None), N), (dict(turns=None), N),
    (dict(dtype=3), UN), (dict(dtype=-1), UN),
    (dict(tokens=0), SH), (dict(heads=0), SH), (dict(size=1, rd=2), SH),
    (dict(rd=0), SH), (dict(rd=63), SH), (dict(rd=66), SH),
    (dict(amp=math.inf), SH), (dict(amp=math.nan), SH),
    (dict(start=-1), SH), (dict(period=-1), SH), (dict(start=2 ** 31 - 2), SH),
    (dict(pos=4096, start=3), UN), (dict(pos=4096, period=3), UN),
    (dict(out=(1 << 20) + 1), AL), (dict(x=(1 << 24) + 1), AL), (dict(turns=4100), AL),
    (dict(pos=4098), AL), (dict(dtype=2, out=(1 << 20) + 2), AL),
    (dict(xt=-128), SH), (dict(ot=64), SH), (dict(oh=32), SH), (dict(ot=0), SH),
    (dict(xt=1 << 60), SH),
    (dict(x=1 << 20, xt=256), UN),            # in place with other strides
    (dict(x=(1 << 20) + 256), UN),            # overlap in part
])
def test_rotary_refusals(lib, change, code):
    args = list({**ROT, **change}.values())
    for fn in (lib.rotary_forward, lib.rotary_backward):
        assert fn(*args) == code, change
        assert lib.csa_last_error()


def test_rotary_accepted_shapes_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for change in (dict(), dict(x=1 << 20), dict(size=66, rd=2, xt=200, ot=200, oh=70),
                   dict(xh=64 * 4, xt=64, oh=64 * 4, ot=64),  # head-major
                   dict(tokens=1, ot=0), dict(start=2 ** 31 - 4), dict(start=2 ** 31 - 2, period=2),
                   dict(xt=0)):                               # one token's x for all
        assert lib.rotary_forward(*{**ROT, **change}.values()) == _lib.CSA_ERR_CUDA, change


def test_rotary_turns(lib):
    def turns(rd, base=10000.0, scaling=0, factor=1.0, original=0.0, slow=1.0, fast=32.0):
        a = (ctypes.c_uint64 * (rd // 2))()
        assert lib.csa_rotary_turns(a, rd, base, scaling, factor, original, slow, fast) == 0
        return list(a)

    import serving_ref as ref
    for rd in (2, 8, 64, 128):
        for name, (i, kw) in {"none": (0, {}), "linear": (1, {"factor": 4.0}), "ntk": (2, {"factor": 4.0}),
                              "by_parts": (3, {"factor": 4.0, "original_length": 2048.0})}.items():
            f = ref.frequencies(rd, scaling=name, **kw).tolist()
            got = turns(rd, 10000.0, i, kw.get("factor", 1.0), kw.get("original_length", 0.0))
            for t, w in zip(got, f):
                # 64-bit fixed point of a 53-bit value, a few roundings apart
                assert abs(t * 2.0 ** -64 * 2 * math.pi / w - 1) < 2.0 ** -48 + 2.0 ** -64 / w
    a = (ctypes.c_uint64 * 4)()
    bad = [((None, 8, 1e4, 0, 1.0, 0.0, 1.0, 32.0), N), ((a, 7, 1e4, 0, 1.0, 0.0, 1.0, 32.0), SH),
           ((a, 0, 1e4, 0, 1.0, 0.0, 1.0, 32.0), SH), ((a, 8, 1.0, 0, 1.0, 0.0, 1.0, 32.0), SH),
           ((a, 8, math.nan, 0, 1.0, 0.0, 1.0, 32.0), SH), ((a, 8, 1e4, 4, 1.0, 0.0, 1.0, 32.0), UN),
           ((a, 8, 1e4, 1, 0.5, 0.0, 1.0, 32.0), SH), ((a, 8, 1e4, 3, 2.0, 0.0, 1.0, 32.0), SH),
           ((a, 8, 1e4, 3, 2.0, 64.0, 2.0, 2.0), SH)]
    for args, code in bad:
        assert lib.csa_rotary_turns(*args) == code


CACHE = dict(k=4096, v=8192, k_scale=64, v_scale=64, pages=4, heads=2, page_tokens=16, head_size=64,
             format=0)
BATCH = dict(offsets=64, lengths=64, table=64, sequences=1, table_width=4, rows=4, max_new=4)

CACHE_BAD = [
    (dict(k=None), N), (dict(v=None), N), (dict(k_scale=None), N), (dict(v_scale=None), N),
    (dict(pages=0), SH), (dict(heads=0), SH), (dict(head_size=0), SH),
    (dict(page_tokens=0), UN), (dict(page_tokens=8), UN), (dict(page_tokens=48), UN),
    (dict(page_tokens=256), UN), (dict(head_size=40), AL), (dict(head_size=144), UN),
    (dict(format=2), UN), (dict(k=4104), AL), (dict(v_scale=66), AL),
]
BATCH_BAD = [
    (dict(offsets=None), N), (dict(lengths=None), N), (dict(table=None), N),
    (dict(sequences=0), SH), (dict(table_width=0), SH), (dict(rows=0), SH), (dict(max_new=0), SH),
    (dict(table=66), AL),
]


def _refs(cache=None, batch=None):
    c = _KvCacheStruct(*{**CACHE, **(cache or {})}.values())
    b = _KvBatchStruct(*{**BATCH, **(batch or {})}.values())
    return c, b


def _calls(lib, c, b, **change):
    a = {**dict(x=1 << 20, y=1 << 24, dtype=0, t0=128, h0=64, t1=128, h1=64), **change}
    rows = (a["x"], a["y"], a["dtype"], a["t0"], a["h0"], a["t1"], a["h1"])
    pc, pb = ctypes.addressof(c) if c else None, ctypes.addressof(b) if b else None
    return {
        "write": lambda: lib.kv_cache_write(pc, pb, *rows, None),
        "read": lambda: lib.kv_cache_read(*rows, pc, pb, None),
        "attend": lambda: lib.cache_attention_forward(a["x"], a["y"], a["dtype"], 2, *rows[3:], pc, pb,
                                                      0.125, 0, 0, 1 << 28, 1 << 30, None),
    }


@pytest.mark.parametrize("change,code", CACHE_BAD)
def test_cache_refusals(lib, change, code):
    c, b = _refs(cache=change)
    for name, call in _calls(lib, c, b).items():
        assert call() == code, name
    n = ctypes.c_size_t(5)
    assert lib.cache_attention_workspace_size(ctypes.addressof(c), 2, ctypes.byref(n)) == code
    assert n.value == 0


@pytest.mark.parametrize("change,code", BATCH_BAD)
def test_batch_refusals(lib, change, code):
    c, b = _refs(batch=change)
    for name, call in _calls(lib, c, b).items():
        assert call() == code, name


@pytest.mark.parametrize("change,code,only", [
    (dict(x=None), N, None), (dict(y=None), N, None),
    (dict(dtype=3), UN, None), (dict(dtype=2, ), UN, ("write", "attend")),
    (dict(x=(1 << 20) + 8), AL, None), (dict(y=(1 << 24) + 8), AL, None),
    (dict(t0=132), AL, None), (dict(h1=68), AL, None), (dict(t1=-128), SH, None),
    (dict(t0=64), SH, ("read", "attend")), (dict(h0=32), SH, ("read", "attend")),
    (dict(t1=64), SH, ("read",)),
    # q over out in part: one element further, or in place with other strides
    (dict(y=(1 << 20) + 16), UN, ("attend",)), (dict(y=1 << 20, t1=136), UN, ("attend",)),
])
def test_row_refusals(lib, change, code, only):
    c, b = _refs()
    for name, call in _calls(lib, c, b, **change).items():
        if only is None or name in only:
            assert call() == code, name


def test_null_cache_and_batch(lib):
    c, b = _refs()
    for name, call in _calls(lib, None, b).items():
        assert call() == N, name
    for name, call in _calls(lib, c, None).items():
        assert call() == N, name
    assert lib.cache_attention_workspace_size(ctypes.addressof(c), 2, None) == N


def test_attention_refusals(lib):
    c, b = _refs()
    pc, pb = ctypes.addressof(c), ctypes.addressof(b)

    def call(q_heads=2, scale=0.125, window=0, sinks=0, ws=1 << 28, nbytes=1 << 30):
        t = q_heads * 64
        return lib.cache_attention_forward(1 << 20, 1 << 24, 0, q_heads, t, 64, t, 64, pc, pb, scale,
                                           window, sinks, ws, nbytes, None)

    n = ctypes.c_size_t(0)
    assert lib.cache_attention_workspace_size(pc, 2, ctypes.byref(n)) == 0 and n.value > 0
    assert call(q_heads=3) == SH and call(q_heads=0) == SH
    assert call(scale=math.nan) == SH and call(scale=math.inf) == SH
    assert call(window=-1) == SH and call(sinks=-1) == SH
    assert call(ws=None) == _lib.CSA_ERR_WORKSPACE
    assert call(nbytes=n.value - 1) == _lib.CSA_ERR_WORKSPACE
    assert call(ws=(1 << 28) + 8) == AL
    if not torch.cuda.is_available():
        assert call(nbytes=n.value) == _lib.CSA_ERR_CUDA
        for name, f in _calls(lib, c, b).items():
            assert f() == _lib.CSA_ERR_CUDA, name


def test_status_string_of_a_bad_index(lib):
    assert b"index" in lib.csa_status_string(_lib.CSA_ERR_INDEX)


def test_binding_refuses_wrong_tensors(lib):
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):   # CPU tensors
        csa.rotary_forward(x, x, csa.RotaryTable(64, device="cpu"))
    with pytest.raises(ValueError):
        csa.RotaryTable(64, scaling="other", device="cpu")
    with pytest.raises(csa.CsaError):
        csa.RotaryTable(63, device="cpu")
    with pytest.raises(ValueError):
        csa.rotary_qkv(torch.zeros((1, 2, 2, 1, 8)), csa.RotaryTable(8, device="cpu"))
    codes, scale = torch.zeros((1, 2, 16, 64), dtype=torch.int8), torch.zeros((1, 2))
    with pytest.raises(ValueError):
        csa.KvCache(codes, codes, scale, scale)
    with pytest.raises(TypeError):
        csa.KvCache(codes.to(torch.uint8), codes, scale, scale)
    with pytest.raises(ValueError):
        csa.KvCache(codes[0], codes, scale, scale)
    with pytest.raises(ValueError):
        csa.KvBatch(i, i[:1], i[:1].view(1, 1), rows=1)
    with pytest.raises(ValueError):
        csa.KvBatch(i, i[:1], i[:1], rows=1)
