"""cache_attention_forward on batches of other shapes: many sequences, prompts beside single
tokens, more query heads than a block of rows holds; against the definition in 64 bits (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref

pytestmark = pytest.mark.gpu


def attend(b, q, dtype, window=0, sinks=0, max_new=None):
    cache, batch = b.device(csa)
    if max_new is not None:
        batch = csa.KvBatch(batch.offsets, batch.lengths, batch.table, rows=b.rows, max_new=max_new)
    out = torch.full((b.rows, q.shape[1], b.D), 7.0, dtype=dtype, device="cuda")
    csa.cache_attention_forward(out, q.cuda(), cache, batch, window=window, sinks=sinks)
    return out


def check(b, q, out, dtype, window=0, sinks=0, what=""):
    want, bound = ref.attention(q, *b.values("k"), *b.values("v"), b.offsets, b.lengths, b.table,
                                window, sinks)
    n = b.offsets[-1]
    got = out.cpu().double()
    room = bound * (1 + ref.half_step(dtype)) + want.abs() * ref.half_step(dtype) + \
        (2.0 ** -25 if dtype == torch.float16 else 0.0)
    bad = ~((got - want).abs() <= room)[:n]
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist())
    assert bool((got[n:] == 7.0).all()), f"{what}: rows of no sequence"


@pytest.fixture(params=[0, 2], ids=["all_sms", "2_sms"])
def sms(request):
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, request.param)
    yield request.param
    torch.cuda.synchronize()
    csa.set_stream_sm_limit(stream, 0)


@pytest.mark.parametrize("S,window", [(530, 0), (600, 20), (1100, 0)])
def test_many_sequences(S, window, sms):
    """More sequences than a CTA has threads: several to a thread in both work lists."""
    new = [(0, 1, 1, 2, 1)[i % 5] for i in range(S)]
    old = [(i * 37) % 90 for i in range(S)]
    for i, n in ((3, 70), (S // 2, 40), (S - 2, 150), (S - 1, 1)):
        new[i] = n
    b = ref.Batch(new, old, 1, 32, 16, "int8", seed=S, extra_rows=1)
    q = b.rows_of(2, torch.bfloat16, seed=1)
    out = attend(b, q, torch.bfloat16, window, 3)
    assert csa.get_status() == 0
    check(b, q, out, torch.bfloat16, window, 3)


@pytest.mark.parametrize("G", [12, 32])
@pytest.mark.parametrize("new,old,P,D", [([1, 1], [200, 31], 16, 64), ([2, 1, 5], [100, 0, 40], 64, 128),
                                         ([30, 11], [50, 130], 32, 80)])
def test_many_query_heads_of_a_kv_head(G, new, old, P, D, sms):
    """A token's query heads over one and over several blocks of rows."""
    b = ref.Batch(new, old, 2, D, P, "e4m3", seed=G + P)
    q = b.rows_of(2 * G, torch.float16, seed=2)
    out = attend(b, q, torch.float16)
    assert csa.get_status() == 0
    check(b, q, out, torch.float16)


def withheld(b, q, dtype):
    """The status of a call whose kernel for prompts, where it has work, misses its codes."""
    csa.set_wait_limit_ns(20_000_000)  # 20 ms
    try:
        csa.debug_inject(True)
        out = attend(b, q, dtype)
        return csa.get_status(), out
    finally:
        csa.set_wait_limit_ns(0)
        csa.debug_inject(False)


def test_short_prompt_among_single_tokens():
    """One request of 40 new tokens beside 63 single ones is not work for the kernel for
    prompts (3 blocks of 16 rows and 8 heads on 152 SMs): withholding that kernel's codes
    changes nothing."""
    b = ref.Batch([1] * 20 + [40] + [1] * 43, [(i * 91) % 300 for i in range(64)], 8, 64, 32, "int8", seed=4)
    q = b.rows_of(8, torch.bfloat16, seed=3)
    status, out = withheld(b, q, torch.bfloat16)
    assert status == 0
    check(b, q, out, torch.bfloat16)


def test_long_prompt_among_single_tokens():
    """700 new tokens beside 60 single ones are (44 blocks and 8 heads): same rule, other side."""
    b = ref.Batch([1] * 30 + [700] + [1] * 30, [(i * 91) % 300 for i in range(61)], 8, 64, 32, "int8", seed=5)
    q = b.rows_of(8, torch.bfloat16, seed=3)
    status, _ = withheld(b, q, torch.bfloat16)
    assert status == csa.CSA_ERR_TIMEOUT
    out = attend(b, q, torch.bfloat16)
    assert csa.get_status() == 0
    check(b, q, out, torch.bfloat16)


def test_single_tokens_under_a_large_max_new(sms):
    """max_new far above what any sequence has: the same bits."""
    b = ref.Batch([1] * 50, [(i * 53) % 400 for i in range(50)], 4, 64, 16, "e4m3", seed=6)
    q = b.rows_of(8, torch.bfloat16, seed=3)
    out = attend(b, q, torch.bfloat16)
    assert torch.equal(out, attend(b, q, torch.bfloat16, max_new=5000))
    assert csa.get_status() == 0
    check(b, q, out, torch.bfloat16)
