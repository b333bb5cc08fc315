"""token_logprobs_forward on rows far longer than a vocabulary (GPU)."""
import math

import pytest
import torch

import causal_attention_score_gb300 as csa

pytestmark = pytest.mark.gpu
V = 1 << 26


@pytest.mark.parametrize("sms", [0, 1], ids=["all_sms", "1_sm"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [-0.05, -1.2])
def test_sums_of_long_rows(value, dtype, sms):
    """Every thread's first elements 0, which is the largest, and all others alike, so that the roundings of
    a sum that grows and grows are all to one side. A thread adds up chunks of 4 or 8 weights, at most 512 of them before they go to a sum of
    such runs, 128 of those where one SM's CTA has the whole row, and the threads' sums are added up in 13 steps;
    within a chunk there are 5 roundings: less than 670 half steps of 2^-24 of S. The weights themselves are off
    by 2^-21 + |d| 2^-22, d the logit (scale 1, largest 0): log S by that and 2^-23 of itself, log p by
    2^-22 |d| and its own rounding more. T / S = E d is off by twice S's error and its weights'."""
    x = torch.full((1, V), value, dtype=dtype, device="cuda")
    x.view(8, -1)[:, :8192] = 0  # (of the whole row, or of its part that a CTA of eight has)
    d, zeros = float(x[0, -1]), 8 * 8192
    S = zeros + (V - zeros) * math.exp(d)
    mean = (V - zeros) * math.exp(d) * d / S
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, sms)
    try:
        tokens = torch.tensor([V - 1], dtype=torch.int32, device="cuda")
        logprob, entropy, stats, top_logprob, top_token = (t.cpu().double() for t in csa.token_logprobs(x, tokens, 3))
        assert csa.get_status() == 0
    finally:
        csa.set_stream_sm_limit(stream, 0)
    ds = 670 * 2.0 ** -24 + 2.0 ** -21 + abs(d) * 2.0 ** -22
    d_log_s = ds + 2.0 ** -23 * math.log(S)
    d_log_p = d_log_s + 2.0 ** -22 * abs(d) + 2.0 ** -23 * (math.log(S) - d)
    assert abs(stats[0, 1] - math.log(S)) <= d_log_s
    assert abs(logprob[0] - (d - math.log(S))) <= d_log_p
    assert abs(entropy[0] - (math.log(S) - mean)) <= d_log_s + 2 * ds * abs(mean) + 2.0 ** -22 * (math.log(S) + abs(mean))
    assert top_token[0].tolist() == [0, 1, 2] and bool(((top_logprob[0] + math.log(S)).abs() <= d_log_p).all())
