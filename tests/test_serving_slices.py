"""Inputs and outputs that are slices of one tensor: taken where they lie side by side in it,
refused where they share elements. What is refused is on the host, before anything touches a
device."""
import ctypes

import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref
from causal_attention_score_gb300 import _lib, build_lib
from causal_attention_score_gb300.serving import _KvBatchStruct, _KvCacheStruct

UN, BASE = _lib.CSA_ERR_UNSUPPORTED, 1 << 24


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _lib.load()


# input offset, output offset (elements), token and head strides of each; 5 tokens, 2 heads of 64
SIDE_BY_SIDE = [
    (0, 128, (384, 64), (384, 64)), (256, 0, (384, 64), (384, 64)), (128, 256, (384, 64), (384, 64)),
    (0, 128 + 384, (384, 64), (384, 64)),          # the output a token further
    (384 * 3 + 128, 0, (384, 64), (384, 64)),      # and three back
    (0, 64, (384, 128), (384, 128)),               # heads take turns
    (0, 320, (64, 960), (64, 960)), (640, 320, (64, 960), (64, 960)),  # head-major
    (0, 128, (384, 0), (384, 64)),                 # one head's input for all
]
SHARED = [
    (0, 64, (384, 64), (384, 64)), (0, 384, (384, 64), (384, 64)), (0, 320, (384, 64), (384, 64)),
    (0, 384 - 64, (384, 64), (384, 64)), (0, 128, (384, 64), (256, 64)), (0, 256, (64, 960), (64, 960)),
    (0, 128 - 8, (384, 64), (384, 64)), (0, 128, (192, 64), (192, 64)), (0, 64, (0, 64), (384, 64)),
    (0, 32, (384, 128), (384, 128)), (0, 128, (384, 128), (384, 128)),
]


def rotary(lib, i, o, si, so):
    return lib.rotary_forward(BASE + 2 * o, BASE + 2 * i, 0, 5, 2, 64, 64, *so, *si, 4096, 1.0, None, 0, 0, 0,
                              None)


def attend(lib, i, o, si, so):
    c = _KvCacheStruct(4096, 8192, 64, 64, 4, 2, 16, 64, 0)
    b = _KvBatchStruct(64, 64, 64, 1, 4, 5, 5)
    return lib.cache_attention_forward(BASE + 2 * o, BASE + 2 * i, 0, 2, *so, *si, ctypes.addressof(c),
                                       ctypes.addressof(b), 0.125, 0, 0, 1 << 28, 1 << 30, None)


@pytest.mark.parametrize("call", [rotary, attend])
@pytest.mark.parametrize("i,o,si,so", SHARED)
def test_shared_elements_are_refused(lib, call, i, o, si, so):
    assert call(lib, i, o, si, so) == UN


@pytest.mark.parametrize("call", [rotary, attend])
@pytest.mark.parametrize("i,o,si,so", SIDE_BY_SIDE)
def test_slices_side_by_side_reach_the_device(lib, call, i, o, si, so):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    assert call(lib, i, o, si, so) == _lib.CSA_ERR_CUDA


@pytest.mark.parametrize("i,o,si,so", SIDE_BY_SIDE + SHARED)
def test_the_cases_are_what_they_are_called(i, o, si, so):
    t, h, d = torch.meshgrid(torch.arange(5), torch.arange(2), torch.arange(64), indexing="ij")
    got = [set((x + t * s[0] + h * s[1] + d).flatten().tolist()) for x, s in ((i, si), (o, so))]
    assert bool(got[0] & got[1]) == ((i, o, si, so) in SHARED)


@pytest.mark.gpu
@pytest.mark.parametrize("sms", [0, 2])
def test_slices_of_a_packed_tensor(sms):
    """Q turned into another slice of its packed row, attention into a third: the bits of tensors
    apart, every other element as it was."""
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, sms)
    try:
        b = ref.Batch([3, 70, 1], [100, 20, 0], 2, 64, 32, "int8", seed=2)
        q = b.rows_of(4, torch.bfloat16).cuda()
        cache, batch = b.device(csa)
        table = csa.RotaryTable(64)
        turned, out = torch.empty_like(q), torch.empty_like(q)
        csa.rotary_forward(turned, q, table, start=3)
        csa.cache_attention_forward(out, turned, cache, batch)
        packed = torch.full((b.rows, 14, 64), 7.0, dtype=q.dtype, device="cuda")
        packed[:, 1:5] = q
        csa.rotary_forward(packed[:, 9:13], packed[:, 1:5], table, start=3)
        csa.cache_attention_forward(packed[:, 5:9], packed[:, 9:13], cache, batch)
        assert csa.get_status() == 0
        for at, want in ((1, q), (5, out), (9, turned)):
            assert torch.equal(packed[:, at: at + 4], want)
        assert bool((packed[:, 0] == 7.0).all()) and bool((packed[:, 13] == 7.0).all())
    finally:
        torch.cuda.synchronize()
        csa.set_stream_sm_limit(stream, 0)
