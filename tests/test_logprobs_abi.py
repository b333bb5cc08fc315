"""Refusals of the calls on logits: on the host, before anything touches a device."""
import math

import pytest
import torch

import causal_attention_score_gb300 as csa
from causal_attention_score_gb300 import _lib, build_lib

N, SH, AL, UN = (_lib.CSA_ERR_NULL, _lib.CSA_ERR_SHAPE, _lib.CSA_ERR_ALIGN,
                 _lib.CSA_ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _lib.load()


FWD = dict(logprob=4096, entropy=8192, stats=16384, logits=1 << 20, dtype=0, rows=4, vocab=100,
           stride=100, tokens=64, scale=1.0, top=5, top_logprob=4096, top_token=4096, stream=None)
BWD = dict(dlogits=1 << 24, logits=1 << 20, dtype=0, rows=4, vocab=100, d_stride=100, stride=100,
           tokens=64, scale=1.0, stats=4096, entropy=4096, d_logprob=None, d_entropy=None, top=5,
           d_top=64, top_token=64, stream=None)
BOTH = [
    (dict(logits=None), N), (dict(tokens=None), N), (dict(stats=None), N), (dict(entropy=None), N),
    (dict(top_token=None), N), (dict(dtype=3), UN), (dict(dtype=-1), UN), (dict(rows=0), SH),
    (dict(rows=-1), SH), (dict(vocab=0), SH), (dict(vocab=(1 << 30) + 1, stride=1 << 31, top=0), UN),
    (dict(top=-1), SH), (dict(top=33), SH), (dict(vocab=4), SH), (dict(scale=0.0), SH),
    (dict(scale=-1.0), SH), (dict(scale=math.inf), SH), (dict(scale=math.nan), SH),
    (dict(scale=2.0 ** 65), SH), (dict(stride=99), SH), (dict(rows=1 << 40, stride=1 << 30), SH),
    (dict(logits=(1 << 20) + 1), AL), (dict(dtype=2, logits=(1 << 20) + 2), AL), (dict(tokens=66), AL),
    (dict(stats=4100), AL), (dict(entropy=4098), AL), (dict(top_token=66), AL),
]


@pytest.mark.parametrize("change,code", BOTH + [
    (dict(logprob=None), N), (dict(top_logprob=None), N), (dict(logprob=4097), AL),
    (dict(top_logprob=4098), AL)])
def test_forward_refusals(lib, change, code):
    assert lib.token_logprobs_forward(*{**FWD, **change}.values()) == code, change
    assert lib.csa_last_error()


@pytest.mark.parametrize("change,code", BOTH + [
    (dict(dlogits=None), N), (dict(d_logprob=66), AL), (dict(d_entropy=66), AL), (dict(d_top=66), AL),
    (dict(dlogits=(1 << 24) + 1), AL), (dict(d_stride=99), SH), (dict(d_stride=-100), SH),
    (dict(dlogits=1 << 20, d_stride=104), UN),            # in place with another stride
    (dict(dlogits=(1 << 20) + 16), UN)])                  # overlap in part
def test_backward_refusals(lib, change, code):
    assert lib.token_logprobs_backward(*{**BWD, **change}.values()) == code, change
    assert lib.csa_last_error()


def test_accepted_calls_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for change in (dict(), dict(top=0, top_logprob=None, top_token=None), dict(rows=1, stride=0),
                   dict(stride=1 << 20), dict(vocab=5)):
        assert lib.token_logprobs_forward(*{**FWD, **change}.values()) == _lib.CSA_ERR_CUDA, change
    for change in (dict(), dict(dlogits=1 << 20), dict(d_top=None, top_token=None), dict(rows=1, stride=0),
                   dict(top=0, d_top=None, top_token=None),
                   dict(dlogits=(1 << 20) + 200, d_stride=200, stride=200)):  # beside each other
        assert lib.token_logprobs_backward(*{**BWD, **change}.values()) == _lib.CSA_ERR_CUDA, change


def test_binding_refusals():
    x = torch.zeros((2, 10))
    with pytest.raises(ValueError, match="CUDA"):
        csa.token_logprobs(x, torch.zeros((2,), dtype=torch.int32))
    with pytest.raises(ValueError, match="rows, vocab"):
        csa.token_logprobs(x[0], torch.zeros((2,), dtype=torch.int32))
