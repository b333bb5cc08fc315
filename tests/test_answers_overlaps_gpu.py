"""The pages and logits calls refuse arrays that overlap where the header forbids it (GPU); what lies side by
side is taken."""
import pytest
import torch

import causal_attention_score_gb300 as csa

pytestmark = pytest.mark.gpu
ROWS, V, TOP = 6, 40, 3


def arrays():
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    return dict(logprob=f(ROWS), entropy=f(ROWS), stats=f(ROWS, 2), logits=torch.randn((ROWS, V), device="cuda"),
                tokens=torch.arange(ROWS, dtype=torch.int32, device="cuda"), top_logprob=f(ROWS, TOP),
                top_token=torch.zeros((ROWS, TOP), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("change", [
    lambda a: a.update(entropy=a["logprob"]),
    lambda a: a.update(logprob=a["stats"].view(-1)[ROWS: 2 * ROWS]),
    lambda a: a.update(stats=a["top_logprob"].view(-1)[2: 2 + 2 * ROWS].view(ROWS, 2)),
    lambda a: a.update(top_token=a["top_logprob"].view(torch.int32)),
    lambda a: a.update(logprob=a["tokens"].view(torch.float32)),
    lambda a: a.update(logprob=a["logits"].view(-1)[:ROWS]),
    lambda a: a.update(top_logprob=a["logits"].view(-1)[-ROWS * TOP:].view(ROWS, TOP)),
])
def test_forward(change):
    a = arrays()
    change(a)
    with pytest.raises((ValueError, csa.CsaError), match="overlap"):
        csa.token_logprobs_forward(a["logprob"], a["entropy"], a["stats"], a["logits"], a["tokens"], 1.0,
                                   a["top_logprob"], a["top_token"])


def test_outputs_side_by_side_and_between_the_rows():
    """Slices of one tensor, and of the padding of a row, are apart."""
    a = arrays()
    want = csa.token_logprobs(a["logits"], a["tokens"], TOP)
    one = torch.zeros((ROWS * 10 + 64,), device="cuda")
    got = (one[:ROWS], one[ROWS: 2 * ROWS], one[2 * ROWS: 4 * ROWS].view(ROWS, 2), a["logits"], a["tokens"], 1.0,
           one[4 * ROWS: 7 * ROWS].view(ROWS, TOP), one[7 * ROWS: 10 * ROWS].view(torch.int32).view(ROWS, TOP))
    csa.token_logprobs_forward(*got)
    for x, y in zip(want, (*got[:3], *got[6:])):
        assert torch.equal(x, y)
    wide = torch.zeros((ROWS, V + 4 * ROWS), device="cuda")
    wide[:, :V] = a["logits"]
    csa.token_logprobs_forward(wide[2, V: V + ROWS], wide[0, V + 2: V + 2 + ROWS],
                               wide[3, V + 2 * ROWS:].view(ROWS, 2), wide[:, :V], a["tokens"])
    assert torch.equal(wide[2, V: V + ROWS], want[0]) and torch.equal(wide[0, V + 2: V + 2 + ROWS], want[1])
    assert csa.get_status() == 0


def test_backward():
    a = arrays()
    f = csa.token_logprobs(a["logits"], a["tokens"], TOP)
    d = torch.ones((ROWS,), device="cuda")
    dx = torch.zeros((ROWS, V), device="cuda")
    flat = dx.view(-1)
    for bad in (dict(tokens=flat[:ROWS].view(torch.int32)), dict(stats=flat[-2 * ROWS:].view(ROWS, 2)),
                dict(entropy=flat[9: 9 + ROWS]), dict(d_logprob=flat[V: V + ROWS]), dict(d_entropy=flat[:ROWS]),
                dict(d_top=flat[:ROWS * TOP].view(ROWS, TOP)),
                dict(top_token=flat[:ROWS * TOP].view(torch.int32).view(ROWS, TOP))):
        given = dict(tokens=a["tokens"], stats=f[2], entropy=f[1], d_logprob=d, d_entropy=d, d_top=f[3], top_token=f[4])
        with pytest.raises(csa.CsaError, match="overlap"):
            csa.token_logprobs_backward(dx, a["logits"], **{**given, **bad})
    csa.token_logprobs_backward(dx, a["logits"], **given)  # (two inputs that are one array are fine)
    assert csa.get_status() == 0 and bool(dx.any())


def test_books():
    cache = csa.KvCache.empty(8, 1, 16, 16, torch.int8)
    one = torch.zeros((64,), dtype=torch.int32, device="cuda")
    for refs, lengths, table in ((one[:8], one[7:9], one[16:24]), (one[:8], one[8:10], one[9:17]),
                                 (one[:8], one[20:22], one[:8])):
        with pytest.raises(ValueError, match="overlap"):
            csa.KvPages(refs, lengths, table.view(2, 4), 16)
    books = csa.KvPages(one[:8], one[8:10], one[10:18].view(2, 4), 16)
    for moves, in_use in ((one[:8], one[40:41]), (one[17:25], one[40:41]), (one[20:28], one[9:10]),
                          (one[20:28], one[27:28])):
        with pytest.raises(ValueError, match="overlap"):
            csa.kv_cache_compact(cache, books, moves, in_use)
    csa.kv_cache_compact(cache, books, one[18:26], one[26:27])
    assert csa.get_status() == 0 and one[18:27].tolist() == [-1] * 8 + [0]
