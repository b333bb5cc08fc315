"""Arrays of the calls on logits that overlap: refused on the host, before anything touches a device."""
import pytest
import torch

from causal_attention_score_gb300 import _lib, build_lib
from test_logprobs_abi import BWD, FWD

UN = _lib.CSA_ERR_UNSUPPORTED
APART = dict(FWD, top_logprob=32768, top_token=65536)


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _lib.load()


@pytest.mark.parametrize("change", [
    dict(entropy=4096 + 12), dict(stats=8192 + 8), dict(logprob=64 - 12), dict(stats=64 - 24), dict(logprob=1 << 20),
    dict(entropy=(1 << 20) + 796), dict(entropy=(1 << 20) - 12), dict(top_logprob=16384 + 28), dict(top_token=8192 - 76),
    dict(top_token=64), dict(top_logprob=(1 << 20) + 400), dict(top_logprob=1 << 20, stride=256),
    dict(logprob=(1 << 20) + 4096 + 196, stride=2048), dict(logprob=(1 << 20) + 4096 - 4, stride=2048)])
def test_forward(lib, change):
    assert lib.token_logprobs_forward(*{**APART, **change}.values()) == UN, change
    assert b"overlap" in lib.csa_last_error()


@pytest.mark.parametrize("change", [
    dict(tokens=1 << 24), dict(stats=(1 << 24) + 792), dict(entropy=(1 << 24) - 12), dict(d_logprob=1 << 24),
    dict(d_entropy=(1 << 24) + 400), dict(d_top=(1 << 24) - 76), dict(top_token=(1 << 24) + 796),
    dict(d_logprob=(1 << 24) + 196, d_stride=104)])
def test_backward(lib, change):
    assert lib.token_logprobs_backward(*{**BWD, **change}.values()) == UN, change
    assert b"overlap" in lib.csa_last_error()


def test_side_by_side_reaches_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for change in (dict(entropy=4096 + 16), dict(stats=8192 + 16), dict(logprob=64 - 16), dict(entropy=(1 << 20) + 800),
                   dict(entropy=(1 << 20) - 16), dict(logprob=(1 << 20) + 4096 + 200, stride=2048),
                   dict(logprob=(1 << 20) + 4096 - 16, stride=2048), dict(top_logprob=1 << 20, top=0),
                   dict(logprob=(1 << 20) + 200, rows=1, stride=4096)):
        assert lib.token_logprobs_forward(*{**APART, **change}.values()) == _lib.CSA_ERR_CUDA, change
    for change in (dict(tokens=(1 << 24) - 16), dict(entropy=(1 << 24) + 800), dict(d_top=1 << 24, top_token=None, top=0),
                   dict(d_logprob=(1 << 24) + 4096 + 200, d_stride=2048)):
        assert lib.token_logprobs_backward(*{**BWD, **change}.values()) == _lib.CSA_ERR_CUDA, change
