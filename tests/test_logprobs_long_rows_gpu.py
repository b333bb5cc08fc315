"""token_logprobs_forward on rows far longer than a vocabulary (GPU)."""
import math

import pytest
import torch

import causal_attention_score_gb300 as csa

pytestmark = pytest.mark.gpu
V = 1 << 26


def off(mean_abs, log_s, d):
    """(S relatively, log S, log p of a logit d) may be off by, scale 1 and largest logit m: d = x - m. A thread
    adds up chunks of 4 or 8 weights, at most 512 of them before they go to a sum of such runs, 128 of those
    where one SM's CTA has a whole row of 2^26 words, and the threads' sums are added up in 13 steps; within a
    chunk there are 5 roundings: less than 670 half steps of 2^-24 of S. The weights themselves are off by
    2^-21 + |d| 2^-22: on average, their E|d| over p. log S is off by that and 2^-23 of itself, log p by
    2^-22 |d| and its own rounding more."""
    ds = 670 * 2.0 ** -24 + 2.0 ** -21 + mean_abs * 2.0 ** -22
    d_log_s = ds + 2.0 ** -23 * abs(log_s)
    return ds, d_log_s, d_log_s + 2.0 ** -22 * abs(d) + 2.0 ** -23 * abs(d - log_s)


@pytest.mark.parametrize("sms", [0, 1], ids=["all_sms", "1_sm"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [-0.05, -1.2])
def test_sums_of_long_rows(value, dtype, sms):
    """Every thread's first elements 0, which is the largest, and all others alike, so that the roundings of
    a sum that grows and grows are all to one side: the weights' bound of `off` beside the sums'."""
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
    ds, d_log_s, d_log_p = off(abs(d), math.log(S), d)
    assert abs(stats[0, 1] - math.log(S)) <= d_log_s
    assert abs(logprob[0] - (d - math.log(S))) <= d_log_p
    assert abs(entropy[0] - (math.log(S) - mean)) <= d_log_s + 2 * ds * abs(mean) + 2.0 ** -22 * (math.log(S) + abs(mean))
    assert top_token[0].tolist() == [0, 1, 2] and bool(((top_logprob[0] + math.log(S)).abs() <= d_log_p).all())


@pytest.mark.parametrize("sms", [0, 1], ids=["all_sms", "1_sm"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_where_runs_meet(dtype, sms):
    """Rows of two runs and more, with a head and a tail, whose weight is in what lies at the runs' (131072
    chunks) and the row's borders: none of it is lost or counted twice. Of the second row everything but the
    last elements is forbidden, the third is left out, the fourth has +inf in a later run."""
    per = 128 // torch.finfo(dtype).bits  # elements of a chunk
    run = 131072 * per
    vocab = 2 * run + 3 * per + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    held = torch.randn((4, vocab + 3), generator=g, device="cuda").mul_(0.25).to(dtype)
    x = held.view(-1)[1: 1 + 4 * (vocab + 3) - 3].as_strided((4, vocab), (vocab + 3, 1))
    for at in (0, run, 2 * run, vocab - 4):  # (a head is up to a chunk less one)
        for i in range(max(0, at - per), min(vocab, at + 2 * per)):
            x[:, i] = 9 + (i % 7) / 4
    x[1, : vocab - 9] = -math.inf
    x[3, run + 1000] = math.inf
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, sms)
    try:
        tokens = torch.tensor([run, vocab - 1, -1, 5], dtype=torch.int32, device="cuda")
        logprob, entropy, stats, top_logprob, top_token = (t.cpu().double() for t in csa.token_logprobs(x, tokens, 20))
        assert csa.get_status() == 0
    finally:
        csa.set_stream_sm_limit(stream, 0)
    for r in (0, 1):
        y = x[r].double()
        m = y.max()
        d = y - m
        w = d.exp()
        log_s, p = float(w.sum().log()), w / w.sum()
        dd = torch.where(p > 0, d, torch.zeros_like(d))
        mean, mean_abs, mean_sq = float((p * dd).sum()), float((p * dd.abs()).sum()), float((p * dd * dd).sum())
        t = float(d[int(tokens[r])])
        ds, d_log_s, d_log_p = off(mean_abs, log_s, t)
        assert stats[r, 0] == float(m) and abs(stats[r, 1] - log_s) <= d_log_s
        assert abs(logprob[r] - (t - log_s)) <= d_log_p
        assert abs(entropy[r] - (log_s - mean)) <= d_log_s + 2 * ds * mean_abs + 2.0 ** -22 * (mean_sq + mean_abs + log_s)
        order = torch.sort(y, descending=True, stable=True).indices[:20]
        live = y[order] > -math.inf
        assert top_token[r].tolist()[: int(live.sum())] == order[live].tolist()
        far = float(d[order[live]].abs().max())
        assert ((top_logprob[r][: int(live.sum())] - (d[order[live]].cpu() - log_s)).abs() <= off(mean_abs, log_s, far)[2]).all()
    assert logprob[2] == 0 and entropy[2] == 0 and not stats[2].any() and (top_token[2] == -1).all()
    assert logprob[3].isnan() and entropy[3].isnan() and top_logprob[3].isnan().all()
