"""cache_attention_forward where codes, scales and pages hold what no row sees, where V's
scales are zero or far apart, and where many small weights add up: both kernels, against the
definition in 64 bits (GPU)."""
import math

import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=[0, 2], ids=["all_sms", "2_sms"])
def sms(request):
    """The whole GPU, where these batches have the kernel for few rows, and two SMs, where
    sequences of many rows take the kernel for prompts."""
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, request.param)
    yield request.param
    torch.cuda.synchronize()
    csa.set_stream_sm_limit(stream, 0)


def attend(b, q, dtype, window=0, sinks=0, scale=None, table=None):
    cache, batch = b.device(csa)
    if table is not None:
        batch.table.copy_(torch.tensor(table, dtype=torch.int32))
    out = torch.full((b.rows, q.shape[1], b.D), 7.0, dtype=dtype, device="cuda")
    csa.cache_attention_forward(out, q.cuda(), cache, batch, scale=scale, window=window, sinks=sinks)
    assert csa.get_status() == 0
    return out.cpu().double()


def check(b, q, got, dtype, window=0, sinks=0, scale=None, what=""):
    want, bound = ref.attention(q, *b.values("k"), *b.values("v"), b.offsets, b.lengths, b.table,
                                window, sinks, scale)
    room = bound * (1 + ref.half_step(dtype)) + want.abs() * ref.half_step(dtype) + \
        (2.0 ** -25 if dtype == torch.float16 else 0.0)
    bad = ~((got - want).abs() <= room)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(),
                           got[bad][:3].tolist(), want[bad][:3].tolist())


HIDDEN = [
    # new, old, Hq, Hkv, D, P, window, sinks
    ([1, 2], [700, 300], 4, 2, 64, 16, 40, 0),
    ([1, 1, 3], [1000, 129, 515], 4, 2, 128, 64, 100, 4),
    ([1, 2], [777, 200], 2, 1, 48, 32, 33, 70),
    ([1], [500], 8, 1, 80, 128, 1, 17),
    ([150, 40], [600, 300], 4, 2, 64, 16, 50, 3),
    ([200, 90], [500, 77], 2, 2, 128, 64, 65, 0),
    ([130], [900], 4, 1, 112, 128, 100, 130),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new,old,Hq,Hkv,D,P,window,sinks", HIDDEN)
def test_what_no_row_sees_does_not_matter(new, old, Hq, Hkv, D, P, window, sinks, fmt):
    """Keys left of every row's window and past the sinks: their codes are NaN, the scales of
    pages that hold nothing else NaN, infinite, negative or zero, those pages' entries no page."""
    dtype = torch.bfloat16
    b = ref.Batch(new, old, Hkv, D, P, fmt, seed=D + P)
    table = [list(row) for row in b.table]
    gone = 0
    for s, (n, L) in enumerate(zip(b.new, b.lengths)):
        to = L - n - window + 1  # the first row's window begins here
        for t in range(sinks, to):
            for name in ("k", "v"):
                b.codes[name].view(torch.uint8)[b.table[s][t // P], :, t % P] = 0x7F
        for i in range(-(-sinks // P), max(to, 0) // P):
            for name, bad in (("k", (math.nan, math.inf, -1.0)), ("v", (math.nan, math.inf, -1.0, 0.0))):
                b.scale[name][b.table[s][i]] = bad[i % len(bad)]
            table[s][i] = (-7, b.pages, 2 ** 31 - 1)[i % 3]
            gone += 1
    assert gone > 0
    q = b.rows_of(Hq, dtype, seed=11)
    for t in (None, table):
        got = attend(b, q, dtype, window, sinks, table=t)
        check(b, q, got, dtype, window, sinks, what="entries" if t else "codes and scales")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new,old,window", [([1, 1], [500, 20], 0), ([150, 33], [70, 200], 0),
                                            ([2, 140], [300, 400], 90)])
def test_blocks_of_scale_zero(new, old, window, fmt):
    """A block whose V has scale 0 is a block of zeros, and its weights count; one whose K has
    scale 0 has scores of 0."""
    dtype = torch.float16
    for P, which in ((16, "v"), (64, "v"), (32, "k"), (32, "kv")):
        b = ref.Batch(new, old, 2, 64, P, fmt, seed=P)
        for i, p in enumerate(sum(([p for p in row if p >= 0] for row in b.table), [])):
            for name in which:
                if (i + (name == "k")) % 2 == 0:
                    b.scale[name][p, i // 2 % 2:] = 0.0
        q = b.rows_of(4, dtype, seed=5)
        check(b, q, attend(b, q, dtype, window, 5), dtype, window, 5, what=(P, which))
    for name in ("v",):
        b.scale[name][:] = 0.0
    assert bool((attend(b, q, dtype, window, 5) == 0).all())


@pytest.mark.parametrize("big", [2.0 ** 27, 2.0 ** 53, 2.0 ** 93])
@pytest.mark.parametrize("small", ["zeros", 2.0 ** -60, 2.0 ** -95])
@pytest.mark.parametrize("new,old,window", [([1], [900], 0), ([1, 2], [15000, 70], 0), ([140], [500], 0),
                                            ([3, 140], [300, 500], 200)])
def test_every_key_counts_in_the_denominator(new, old, window, small, big):
    """Blocks of V far smaller than others (a written block of zeros has scale 2^-100), with
    scores as large: what they weigh does not depend on V."""
    dtype = torch.bfloat16
    for first in range(3):
        b = ref.Batch(new, old, 1, 64, 32, "int8", seed=7 + first)
        for s, L in enumerate(b.lengths):
            blocks = -(-L // 32)
            for i in range(blocks):
                p = b.table[s][i]
                tiny = (i < blocks // 2, i >= blocks // 2, i % 3 == 0)[first]
                b.scale["v"][p, 0] = (2.0 ** -100 if small == "zeros" else small) if tiny else big
                if tiny and small == "zeros":
                    b.codes["v"][p] = torch.where(b.live[p][None, :, None], 0, b.codes["v"][p])
        for q_scale in (0.0, 1.0):
            q = b.rows_of(2, dtype, q_scale, seed=11)
            check(b, q, attend(b, q, dtype, window, 3), dtype, window, 3, what=(first, q_scale))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new", [1, 70])
def test_many_small_weights_add_up(new, fmt):
    """One key of weight 1 whose V is 0, before N = 2^15 keys of weight 2^-27: the output is
    theirs, N 2^-27 v.

    A weight is rounded to fp16: 2^-11 relatively, and 2^-25 absolutely where subnormal, where
    the largest of its row is at least 2^7: 2^-32 of that for each key. The weights' own
    errors are those of ref.attention (scores here are exact: one product of a key)."""
    dtype, D, P = torch.bfloat16, 64, 128
    N = 2 ** 15
    b = ref.Batch([new], [N - new], 1, D, P, fmt, seed=2)
    top = 127 if fmt == "int8" else 448
    pages = b.table[0][: N // P]
    for name in ("k", "v"):
        b.codes[name][:] = torch.zeros_like(b.codes[name].float()).to(b.codes[name].dtype)
        b.scale[name][:] = 2.0 ** -6
    b.codes["k"][pages[0], 0, 0, 0] = top
    b.codes["v"][pages] = (torch.randn((len(pages), 1, P, D), generator=b.g).abs() * 30 + 1).clamp(max=120).round().to(
        b.codes["v"].dtype)
    b.codes["v"][pages[0], 0, 0] = torch.zeros(D).to(b.codes["v"].dtype)
    q = torch.zeros((new, 1, D), dtype=dtype)
    q[:, 0, 0] = 1.0
    scale = 27 * math.log(2) / (top * 2.0 ** -6)
    got = attend(b, q, dtype, scale=scale)
    want, _ = ref.attention(q, *b.values("k"), *b.values("v"), b.offsets, b.lengths, b.table, scale=scale)
    v = b.values("v")
    vmax = float((v[0] * v[1][..., None, None]).max())
    # exponents up to 32 in size: their roundings are worth 2^-18; sums of N terms
    d = 2.0 ** -16 + 2.0 ** -18 + N * 2.0 ** -24
    room = want * (2 * d + 2.0 ** -11 + ref.half_step(dtype)) * 1.01 + N * 2.0 ** -32 * vmax
    assert bool((want > 4 * N * 2.0 ** -32 * vmax).all())
    bad = ~((got - want).abs() <= room)
    assert not bad.any(), (int(bad.sum()), got[bad][:3].tolist(), want[bad][:3].tolist())
