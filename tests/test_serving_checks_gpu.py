"""The checking build (-DCSA_DEBUG) on the rotary, cache and cache-attention calls: no check of
decoded positions, ring places and TMEM columns fails, and the bits are the release library's
(GPU)."""
import ctypes

import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref
from causal_attention_score_gb300 import _lib, build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checking():
    lib = ctypes.CDLL(build_lib.build(debug=True))
    for name, (res, args) in _lib.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


@pytest.fixture
def both(checking, monkeypatch):
    """run(f): f() on either library, both without a failed check, their results equal."""
    def run(f):
        want = f()
        assert csa.get_status() == 0
        with monkeypatch.context() as m:
            m.setattr(_lib, "_lib", checking)
            got = f()
            assert csa.get_status() == 0, "a device check failed"
        assert len(want) == len(got) > 0
        for w, g in zip(want, got):
            assert torch.equal(w.contiguous().view(torch.uint8), g.contiguous().view(torch.uint8))
    return run


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,size,rd", [(1, 3, 64, 64), (500, 9, 80, 48), (333, 5, 34, 10),
                                                  (3000, 24, 64, 64)])
def test_rotary(both, tokens, heads, size, rd, interleaved, dtype):
    x = torch.randn((tokens, heads, size), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()

    def call():
        table = csa.RotaryTable(rd)
        out, y = torch.empty_like(x), x.clone()
        csa.rotary_forward(out, x, table, start=5, interleaved=interleaved)
        csa.rotary_backward(y, y, table, start=5, interleaved=interleaved)
        return out, y

    both(call)


@pytest.mark.parametrize("new,old,Hkv,D,P", [([1, 1, 3], [15, 16, 100], 3, 64, 16),
                                             ([200, 1, 65], [0, 63, 127], 2, 128, 64),
                                             ([300, 17], [5, 250], 4, 80, 128), ([9, 40], [0, 3], 1, 112, 32)])
def test_cache(both, new, old, Hkv, D, P):
    b = ref.Batch(new, old, Hkv, D, P, "int8", seed=D, extra_rows=1)
    k, v = (b.rows_of(Hkv, torch.bfloat16, 3.0, seed=s).cuda() for s in (1, 2))

    def call():
        cache, batch = b.device(csa)
        csa.kv_cache_write(cache, batch, k, v)
        back = [torch.zeros((b.rows, Hkv, D), device="cuda") for _ in range(2)]
        csa.kv_cache_read(*back, cache, batch)
        return [cache.k, cache.v, *back]

    both(call)


@pytest.mark.parametrize("sms", [0, 2])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new,old,Hq,Hkv,D,P,window,sinks", [
    ([1], [776], 12, 12, 64, 64, 0, 0),
    ([1, 2, 0, 9], [3000, 17, 4, 0], 8, 2, 128, 16, 0, 0),
    ([3, 150, 1], [130, 400, 0], 6, 2, 80, 64, 70, 5),
    ([300, 40, 260], [70, 600, 0], 8, 1, 64, 128, 0, 0),
    ([200, 131], [300, 0], 4, 2, 128, 32, 100, 0),
])
def test_attention(both, new, old, Hq, Hkv, D, P, window, sinks, fmt, sms):
    b = ref.Batch(new, old, Hkv, D, P, fmt, seed=D + P)
    q = b.rows_of(Hq, torch.float16, seed=3).cuda()

    def call():
        stream = torch.cuda.current_stream()
        csa.set_stream_sm_limit(stream, sms)
        try:
            cache, batch = b.device(csa)
            out = torch.empty_like(q)
            csa.cache_attention_forward(out, q, cache, batch, window=window, sinks=sinks)
            torch.cuda.synchronize()
            return [out]
        finally:
            csa.set_stream_sm_limit(stream, 0)

    both(call)
