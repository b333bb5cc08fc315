"""token_logprobs_forward / _backward against their definitions in 64 bits (GPU)."""
import math

import pytest
import torch

import causal_attention_score_gb300 as csa
import logprobs_ref as ref
from causal_attention_score_gb300 import _lib
from serving_ref import half_step

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def rows_of(kind, rows, vocab, g):
    x = torch.randn((rows, vocab), generator=g) * 3
    if kind == "equal":
        x = torch.full_like(x, 1.25)
    elif kind == "zeros":  # of both signs
        x = torch.where(torch.rand(x.shape, generator=g) < 0.5, 0.0, -0.0)
    elif kind == "rising":
        x = torch.arange(vocab, dtype=torch.float32).expand(rows, vocab) * (40.0 / vocab) - 20
    elif kind == "falling":
        x = 20 - torch.arange(vocab, dtype=torch.float32).expand(rows, vocab) * (40.0 / vocab)
    elif kind == "few":    # few values: ties everywhere
        x = torch.randint(0, 3, x.shape, generator=g).float()
    elif kind == "masked":
        x = x.masked_fill(torch.rand(x.shape, generator=g) < 0.8, -math.inf)
    elif kind == "lowest":
        x = x.masked_fill(torch.rand(x.shape, generator=g) < 0.8, -3.0e38)
    elif kind == "far":
        x = x + 1000
    elif kind == "peaked":
        x[:, vocab // 2] = 60
    elif kind == "columns":  # the largest, very many of them, in chunks of few threads
        at = torch.arange(vocab) // 4 % 512
        x = torch.where(at < 32, 30.0 + at, x)
    return x.clone()


def close(got, want, bound, what, dtype=torch.float32):
    got = got.cpu().double()
    same = (got == want) | (got.isnan() & want.isnan())
    err = (got - want).abs()
    bad = ~(same | (err <= bound + want.abs() * half_step(dtype)))
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err - bound)[bad].max())}"


def laid_out(x, dtype, pitch, shift):
    """x as [rows, vocab] on the GPU whose rows are vocab + pitch apart, `shift` elements into its storage."""
    rows, vocab = x.shape
    held = torch.full((rows * (vocab + pitch) + shift,), 99.0, dtype=dtype, device="cuda")
    view = held[shift:].view(rows, vocab + pitch)[:, :vocab]
    view.copy_(x.to(dtype))
    return view


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind,rows,vocab,pitch,shift,top,scale", [
    ("normal", 1, 1, 0, 0, 1, 1.0),
    ("normal", 3, 2, 1, 1, 2, 1.0),
    ("normal", 2, 17, 0, 3, 5, 0.5),
    ("normal", 700, 33, 0, 0, 32, 2.0),
    ("normal", 5, 511, 2, 1, 20, 1.0),
    ("normal", 48, 4097, 0, 0, 5, 1.0),
    ("normal", 1, 50257, 0, 1, 32, 1.0),
    ("normal", 31, 50257, 0, 0, 0, 0.7),
    ("peaked", 3, 128000, 8, 0, 20, 1.0),
    ("equal", 2, 50257, 0, 0, 32, 1.0),
    ("equal", 330, 5000, 0, 1, 7, 1.0),
    ("zeros", 3, 9000, 1, 0, 20, 1.0),
    ("few", 2, 20000, 0, 5, 32, 1.0),
    ("rising", 2, 50257, 0, 0, 32, 1.0),
    ("falling", 2, 50257, 0, 0, 32, 1.0),
    ("masked", 4, 3001, 0, 0, 32, 1.0),
    ("lowest", 4, 3001, 0, 0, 32, 1.0),
    ("far", 3, 10007, 0, 0, 5, 1.0),
    ("columns", 1, 200000, 0, 0, 32, 1.0),
    ("columns", 200, 30000, 0, 0, 32, 1.0),
])
def test_forward(kind, rows, vocab, pitch, shift, top, scale, dtype):
    if kind == "lowest" and dtype == torch.float16:
        pytest.skip("no such value in fp16")
    g = torch.Generator().manual_seed(rows + vocab)
    x = laid_out(rows_of(kind, rows, vocab, g), dtype, pitch, shift)
    tokens = torch.randint(0, vocab, (rows,), generator=g, dtype=torch.int32)
    if rows > 2:
        tokens[1] = -1
    want, bound = ref.forward(x.cpu(), tokens, scale, top)
    got = dict(zip(("logprob", "entropy", "stats", "top_logprob", "top_token"),
                   csa.token_logprobs(x, tokens.cuda(), top, scale)))
    torch.cuda.synchronize()
    assert csa.get_status() == 0
    assert torch.equal(got["top_token"].cpu().long(), want["top_token"].long())
    for name in ("logprob", "entropy", "stats", "top_logprob"):
        close(got[name], want[name], bound[name], name)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_without_numbers(dtype):
    """Every logit -inf; one NaN; one +inf; beside a row of numbers."""
    x = torch.randn((4, 3000), generator=torch.Generator().manual_seed(0))
    x[0] = -math.inf
    x[1, 7] = math.nan
    x[2, 9] = math.inf
    x = x.to(dtype)
    tokens = torch.tensor([5, 2999, 9, 3], dtype=torch.int32)
    logprob, entropy, stats, top_logprob, top_token = (t.cpu() for t in csa.token_logprobs(
        x.cuda(), tokens.cuda(), 4))
    assert logprob[0] == -math.inf and entropy[0] == 0 and (top_logprob[0] == -math.inf).all()
    assert stats[0, 0] == -math.inf and stats[0, 1] == 0 and top_token[0].tolist() == [0, 1, 2, 3]
    for r in (1, 2):
        assert logprob[r].isnan() and entropy[r].isnan() and top_logprob[r].isnan().all()
    order = torch.sort(torch.nan_to_num(x.double(), nan=-math.inf, posinf=math.inf), dim=1, descending=True,
                       stable=True)
    assert torch.equal(top_token[1:].long(), order.indices[1:, :4])
    want, bound = ref.forward(x[3:], tokens[3:], 1.0, 4)
    close(logprob[3:], want["logprob"], bound["logprob"], "logprob")
    # and their gradients: zeros; NaN; NaN; numbers
    d = torch.ones((4,), device="cuda")
    dx = torch.full_like(x, 5).cuda()
    f = csa.token_logprobs(x.cuda(), tokens.cuda())
    csa.token_logprobs_backward(dx, x.cuda(), tokens.cuda(), f[2], f[1], d, d)
    assert (dx[0] == 0).all() and dx[1].isnan().all() and dx[3].isfinite().all()
    assert dx[2].isnan().any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind,rows,vocab,pitch,d_pitch,shift,top,scale,terms", [
    ("normal", 1, 1, 0, 0, 0, 1, 1.0, "leh"),
    ("normal", 3, 2, 1, 0, 1, 2, 1.0, "leh"),
    ("normal", 40, 333, 0, 0, 0, 5, 1.5, "l"),
    ("normal", 40, 333, 0, 3, 1, 5, 1.5, "e"),
    ("normal", 2, 50257, 0, 0, 0, 32, 1.0, "leh"),
    ("normal", 3, 50257, 7, 7, 3, 20, 0.7, "h"),
    ("normal", 650, 2051, 0, 0, 0, 0, 1.0, "le"),
    ("masked", 7, 4000, 0, 0, 0, 20, 1.0, "leh"),
    ("peaked", 5, 9001, 0, 0, 0, 4, 1.0, "leh"),
    ("far", 3, 10007, 0, 0, 0, 5, 1.0, "le"),
    ("normal", 2, 700, 0, 0, 0, 3, 1.0, ""),
])
def test_backward(kind, rows, vocab, pitch, d_pitch, shift, top, scale, terms, dtype):
    g = torch.Generator().manual_seed(rows * 3 + vocab)
    x = laid_out(rows_of(kind, rows, vocab, g), dtype, pitch, shift)
    tokens = torch.randint(0, vocab, (rows,), generator=g, dtype=torch.int32)
    if rows > 2:
        tokens[2] = -100
    t = tokens.cuda()
    logprob, entropy, stats, _, top_token = csa.token_logprobs(x, t, top, scale)
    d = {"d_logprob": torch.randn((rows,), generator=g) if "l" in terms else None,
         "d_entropy": torch.randn((rows,), generator=g) if "e" in terms else None,
         "d_top": torch.randn((rows, top), generator=g) if "h" in terms else None}
    want, bound = ref.backward(x.cpu(), tokens, scale, **d, top_token=top_token.cpu())
    d = {k: None if v is None else v.cuda() for k, v in d.items()}
    dx = laid_out(torch.full((rows, vocab), 7.0), dtype, d_pitch, shift)
    csa.token_logprobs_backward(dx, x, t, stats, entropy, **d, top_token=top_token, scale=scale)
    # (fp16: half its smallest step)
    close(dx, want, bound + 2.0 ** -25 * (dtype == torch.float16), "apart", dtype)
    before = x.clone()
    csa.token_logprobs_backward(x, x, t, stats, entropy, **d, top_token=top_token, scale=scale)
    if pitch == d_pitch:
        assert torch.equal(x.cpu(), dx.cpu()), "in place"
    close(x, want, bound + 2.0 ** -25 * (dtype == torch.float16), "in place", dtype)
    assert before.shape == x.shape and csa.get_status() == 0


# Rows so short and so many that a warp takes each (up to 16384 bytes; more than 12 rows an SM), and their neighbours that a CTA takes. One after the other a lane of a warp
# adds up vocab / 256 chunks of 8 elements, 6 terms in the last of them and 6 of the lanes and what
# belongs to no chunk: at 8192 elements 44, and the bound counts vocab / 512 + 32 = 48. In fp32
# vocab / 128 chunks of 4 and 9 terms more: at 3900 elements 39.5 of 39.6.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind,rows,vocab,pitch,shift,top,scale", [
    ("normal", 2000, 1, 0, 0, 1, 1.0),
    ("normal", 40000, 64, 0, 0, 4, 1.0),
    ("normal", 1825, 255, 1, 1, 32, 2.0),
    ("equal", 1900, 300, 0, 0, 20, 1.0),     # more candidates than are kept
    ("equal", 9, 1023, 1, 0, 32, 1.0),
    ("masked", 1900, 257, 0, 5, 32, 1.0),
    ("few", 2100, 1500, 0, 0, 32, 1.0),
    ("zeros", 2000, 2048, 0, 0, 3, 1.0),
    ("rising", 2000, 2047, 0, 1, 32, 1.0),
    ("columns", 1900, 2048, 0, 0, 32, 1.0),
    ("lowest", 2000, 700, 4, 0, 5, 1.0),
    ("normal", 2000, 3900, 0, 0, 0, 0.7),
    ("far", 1900, 3899, 1, 3, 0, 1.0),
    ("normal", 2000, 8192, 0, 0, 0, 1.0),
    ("normal", 1900, 8001, 3, 0, 20, 1.0),
    ("rising", 1900, 3900, 0, 0, 32, 1.0),
    ("normal", 1824, 700, 0, 0, 6, 1.0),
])
def test_many_short_rows(kind, rows, vocab, pitch, shift, top, scale, dtype):
    test_forward(kind, rows, vocab, pitch, shift, top, scale, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind,rows,vocab,pitch,d_pitch,shift,top,scale,terms", [
    ("normal", 2000, 1, 0, 0, 0, 1, 1.0, "leh"),
    ("normal", 30000, 64, 0, 0, 0, 4, 1.0, "leh"),
    ("normal", 1900, 333, 0, 3, 1, 32, 1.5, "leh"),
    ("masked", 2000, 1001, 7, 7, 3, 32, 1.0, "leh"),
    ("equal", 1900, 256, 0, 0, 0, 32, 0.7, "lh"),
    ("peaked", 2000, 3900, 0, 0, 0, 0, 1.0, "le"),
    ("normal", 1824, 700, 0, 0, 0, 6, 1.0, "leh"),
])
def test_gradient_of_many_short_rows(kind, rows, vocab, pitch, d_pitch, shift, top, scale, terms, dtype):
    test_backward(kind, rows, vocab, pitch, d_pitch, shift, top, scale, terms, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_short_rows_without_numbers(dtype):
    """NaN, +inf and nothing but -inf in some of many short rows, tokens out of range and left out:
    their results, and the others' as if each were the only row."""
    rows, V, top = 2400, 200, 5
    x = torch.randn((rows, V), generator=torch.Generator().manual_seed(8)).to(dtype)
    tokens = torch.arange(rows, dtype=torch.int32) % V
    x[7, 150] = math.nan
    x[9, 3] = math.inf
    x[11] = -math.inf
    x[13, 4:] = -math.inf  # fewer than top are left
    tokens[15], tokens[17] = -5, V
    logprob, entropy, stats, top_logprob, top_token = (
        t.cpu() for t in csa.token_logprobs(x.cuda(), tokens.cuda(), top))
    assert csa.get_status() == _lib.CSA_ERR_INDEX
    for r in (7, 9):
        assert logprob[r].isnan() and entropy[r].isnan() and top_logprob[r].isnan().all()
    assert logprob[11] == -math.inf and entropy[11] == 0 and stats[11].tolist() == [-math.inf, 0]
    assert top_token[11].tolist() == [0, 1, 2, 3, 4] and (top_logprob[11] == -math.inf).all()
    assert sorted(top_token[13, :4].tolist()) == [0, 1, 2, 3] and top_token[13, 4] == 4
    assert top_logprob[13, 4] == -math.inf and top_logprob[13, :4].isfinite().all()
    for r in (15, 17):
        assert logprob[r] == 0 and entropy[r] == 0 and not stats[r].any()
        assert (top_token[r] == -1).all() and not top_logprob[r].any()
    odd = [7, 9, 11, 13, 15, 17]
    keep = torch.ones(rows, dtype=torch.bool)
    keep[odd] = False
    clean, at = x.clone(), tokens.clone()
    clean[odd], at[odd] = 0, 0
    again = [t.cpu() for t in csa.token_logprobs(clean.cuda(), at.cuda(), top)]
    for got, want in zip((logprob, entropy, stats, top_logprob, top_token), again):
        assert torch.equal(got[keep], want[keep])
    g = torch.ones(rows, device="cuda")
    dx = torch.full_like(x, 3.0).cuda()
    csa.token_logprobs_backward(dx, x.cuda(), tokens.cuda(), stats.cuda(), entropy.cuda(), g)
    assert csa.get_status() == _lib.CSA_ERR_INDEX
    assert not dx[[11, 15, 17]].any() and dx[7].isnan().any() and dx[9].isnan().any()
    assert dx[keep.cuda()].isfinite().all()


def test_repeated_alternatives_and_the_token_among_them():
    """Weights of one element named several times add up."""
    x = torch.randn((2, 5000), generator=torch.Generator().manual_seed(3))
    tokens = torch.tensor([11, 4999], dtype=torch.int32)
    top_token = torch.tensor([[11, 7, 11], [3, 3, 3]], dtype=torch.int32)
    d_top = torch.tensor([[0.5, 2.0, -0.25], [1.0, -3.0, 0.5]])
    d = torch.tensor([1.5, -0.5])
    want, bound = ref.backward(x, tokens, 1.0, d, None, d_top, top_token)
    f = csa.token_logprobs(x.cuda(), tokens.cuda())
    dx = torch.empty_like(x).cuda()
    csa.token_logprobs_backward(dx, x.cuda(), tokens.cuda(), f[2], f[1], d.cuda(), None, d_top.cuda(),
                                top_token.cuda())
    close(dx, want, bound, "repeated")


def test_gradient_is_the_difference_quotient():
    g = torch.Generator().manual_seed(5)
    x = torch.randn((3, 900), generator=g) * 2
    tokens = torch.tensor([4, 899, 0], dtype=torch.int32)
    a, b = torch.randn((3,), generator=g), torch.randn((3,), generator=g)

    def value(y):  # in 64 bits, per row
        lp = torch.log_softmax(y.double(), 1)
        return a.double() * lp.gather(1, tokens.long()[:, None])[:, 0] - b.double() * (lp.exp() * lp).sum(1)

    f = csa.token_logprobs(x.cuda(), tokens.cuda())
    dx = torch.empty_like(x).cuda()
    csa.token_logprobs_backward(dx, x.cuda(), tokens.cuda(), f[2], f[1], a.cuda(), b.cuda())
    for j in (0, 4, 33, 899):
        e = torch.zeros_like(x, dtype=torch.float64)
        e[:, j] = 2.0 ** -12
        quotient = (value(x.double() + e) - value(x.double() - e)) * 2.0 ** 11
        # third derivatives of such functions are below 40: 40 / 6 * 2^-24
        assert ((dx[:, j].cpu().double() - quotient).abs() < 2.0 ** -20).all()


def test_out_of_range_tokens_are_reported():
    x = torch.randn((3, 100), device="cuda")
    f = csa.token_logprobs(x, torch.tensor([5, 100, 7], dtype=torch.int32, device="cuda"), 2)
    assert csa.get_status() == csa.CSA_ERR_INDEX
    assert f[0][1] == 0 and f[1][1] == 0 and f[4][1].tolist() == [-1, -1] and f[0][0] < 0
    dx = torch.full_like(x, 3)
    d = torch.ones((3,), device="cuda")
    bad = torch.tensor([[1, 2], [0, 0], [1, 1000]], dtype=torch.int32, device="cuda")
    csa.token_logprobs_backward(dx, x, torch.tensor([5, 100, 7], dtype=torch.int32, device="cuda"), f[2],
                                f[1], d, d, torch.ones((3, 2), device="cuda"), bad)
    assert csa.get_status() == csa.CSA_ERR_INDEX
    assert (dx[1] == 0).all() and dx.isfinite().all()


def test_streams_graph_and_sm_limit():
    g = torch.Generator().manual_seed(9)
    x = (torch.randn((64, 20011), generator=g) * 3).to(torch.bfloat16).cuda()
    tokens = torch.randint(0, 20011, (64,), generator=g, dtype=torch.int32).cuda()
    want = csa.token_logprobs(x, tokens, 5)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = csa.token_logprobs(x, tokens, 5, stream=st)
    st.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    out = [torch.empty_like(t) for t in want]
    dx = torch.empty_like(x)
    d = torch.ones((64,), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.token_logprobs_forward(out[0], out[1], out[2], x, tokens, 1.0, out[3], out[4])
        csa.token_logprobs_backward(dx, x, tokens, out[2], out[1], d, d)
    x2 = (torch.randn((64, 20011), generator=g) * 3).to(torch.bfloat16).cuda()
    x.copy_(x2)
    graph.replay()
    want = csa.token_logprobs(x2, tokens, 5)
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    dw = torch.empty_like(x)
    csa.token_logprobs_backward(dw, x2, tokens, want[2], want[1], d, d)
    assert torch.equal(dx, dw)
    csa.set_stream_sm_limit(st, 3)
    try:
        st.wait_stream(torch.cuda.current_stream())
        few = csa.token_logprobs(x2, tokens, 5, stream=st)
        st.synchronize()
    finally:
        csa.set_stream_sm_limit(st, 0)
    ref_want, bound = ref.forward(x2.cpu(), tokens.cpu(), 1.0, 5)
    assert torch.equal(few[4], want[4])
    for i, name in enumerate(("logprob", "entropy", "stats", "top_logprob")):
        close(few[i], ref_want[name], bound[name], name)


@pytest.mark.parametrize("sms", [1, 5])
@pytest.mark.parametrize("rows,vocab,top", [(300, 5000, 4), (3000, 300, 7), (3000, 1900, 0), (40, 30000, 3)])
def test_rows_in_turn_under_a_limit(rows, vocab, top, sms):
    """Few SMs: CTAs, clusters and warps that take several rows, forwards and backwards."""
    g = torch.Generator().manual_seed(rows + sms)
    x = torch.randn((rows, vocab), generator=g) * 3
    tokens = torch.randint(-vocab // 9, vocab, (rows,), generator=g, dtype=torch.int32)
    d = {"d_logprob": torch.randn((rows,), generator=g), "d_entropy": torch.randn((rows,), generator=g)}
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, sms)
    try:
        got = csa.token_logprobs(x.cuda(), tokens.cuda(), top)
        dx = torch.full_like(x, 9.0).cuda()
        csa.token_logprobs_backward(dx, x.cuda(), tokens.cuda(), got[2], got[1],
                                    **{k: v.cuda() for k, v in d.items()})
        assert csa.get_status() == 0
    finally:
        csa.set_stream_sm_limit(stream, 0)
    want, bound = ref.forward(x, tokens, 1.0, top)
    assert torch.equal(got[4].cpu().long(), want["top_token"].long())
    for i, name in enumerate(("logprob", "entropy", "stats", "top_logprob")):
        close(got[i], want[name], bound[name], name)
    wd, bd = ref.backward(x, tokens, 1.0, **d)
    close(dx, wd, bd, "gradient")


def test_past_2_to_the_31():
    """Rows that lie more than 2^31 elements and 2^32 bytes into the logits."""
    rows, V = 45000, 50257
    x = torch.empty((rows, V), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    at = [0, 20000, 42731, 44999]
    x.fill_(-1.5)
    for r in at:
        x[r] = torch.randn((V,), generator=g, device="cuda") * 3
    tokens = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    tokens[at] = torch.tensor([5, 50256, 777, 31000], dtype=torch.int32, device="cuda")
    got = csa.token_logprobs(x, tokens, 3)
    want, bound = ref.forward(x[at].cpu(), tokens[at].cpu(), 1.0, 3)
    assert torch.equal(got[4][at].cpu().long(), want["top_token"])
    close(got[0][at], want["logprob"], bound["logprob"], "logprob")
    d = torch.ones((rows,), device="cuda")
    wd, bd = ref.backward(x[at].cpu(), tokens[at].cpu(), 1.0, d[at].cpu())
    csa.token_logprobs_backward(x, x, tokens, got[2], got[1], d)
    assert csa.get_status() == 0
    close(x[at], wd, bd, "in place", torch.bfloat16)
    left_out = torch.ones((rows,), dtype=torch.bool, device="cuda")
    left_out[at] = False
    assert not x[left_out].any()


def test_from_a_dense_layer():
    """Logits as a dense layer writes them, then the gradient by that layer's input."""
    g = torch.Generator().manual_seed(1)
    X = torch.randn((77, 96), generator=g).to(torch.bfloat16)
    W = (torch.randn((1003, 96), generator=g) * 0.2).to(torch.bfloat16)
    tokens = torch.randint(0, 1003, (77,), generator=g, dtype=torch.int32)
    logits = csa.dense(X.cuda(), W.cuda())
    logprob, entropy, stats, top_logprob, top_token = csa.token_logprobs(logits, tokens.cuda(), 3)
    want, bound = ref.forward(logits.cpu(), tokens, 1.0, 3)
    close(logprob, want["logprob"], bound["logprob"], "logprob")
    close(entropy, want["entropy"], bound["entropy"], "entropy")
    d = torch.full((77,), -1 / 77, device="cuda")
    dlogits = logits.to(torch.bfloat16)
    f = csa.token_logprobs(dlogits, tokens.cuda())
    wd, bd = ref.backward(dlogits.cpu(), tokens, 1.0, d.cpu())
    csa.token_logprobs_backward(dlogits, dlogits, tokens.cuda(), f[2], f[1], d)
    close(dlogits, wd, bd, "dlogits", torch.bfloat16)
    dX = csa.dense(dlogits, W.t().contiguous().cuda())  # dX = dlogits W
    exact = dlogits.cpu().double() @ W.double()
    # sums of 1003 products in fp32
    size = dlogits.cpu().double().abs() @ W.double().abs()
    assert ((dX.cpu().double() - exact).abs() <= 1010 * 2.0 ** -24 * size).all()
