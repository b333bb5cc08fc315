"""cache_attention_forward on unusual scales of blocks: both kernels, against the definition
in 64 bits (GPU)."""
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
