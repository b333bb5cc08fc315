"""Lengths and offsets that change while calls are under way, which the calls do not allow: what
they compute is undefined, but they write nothing outside their rows, end, and leave the next
call as it should be (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sms", [0, 2])
@pytest.mark.parametrize("S", [5, 700])
def test_arrays_that_change_under_calls(S, sms):
    """Two valid states of a batch (prompts there and here) written in turn from another stream
    while 100 calls run; then a quiet call against the definition."""
    D, H = 32, 2
    new = [1] * S
    new[0], new[S // 2], new[-1] = 150, 40, 33
    other = new[::-1]
    old = [(i * 37) % 60 for i in range(S)]
    b = ref.Batch([max(x) for x in zip(new, other)], old, 1, D, 16, "int8", seed=S)
    states = []
    for n in (new, other):
        off = [sum(n[:i]) for i in range(S + 1)]
        states.append([torch.tensor(t, dtype=torch.int32, device="cuda")
                       for t in (off, [a + c for a, c in zip(n, old)])])
    rows = sum(new)
    cache, _ = b.device(csa)
    off, lengths = (t.clone() for t in states[0])
    table = torch.tensor(b.table, dtype=torch.int32, device="cuda")
    batch = csa.KvBatch(off, lengths, table, rows=rows, max_new=150)
    q = b.rows_of(H, torch.bfloat16)[:rows].contiguous()
    qd = q.cuda()
    big = torch.full((rows + 2000, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[1000: 1000 + rows]
    need = csa.cache_attention_workspace_size(cache, batch, H)
    ws = torch.full((need + 2 ** 16,), 85, dtype=torch.uint8, device="cuda")
    calls, writer = torch.cuda.Stream(), torch.cuda.Stream()
    csa.set_stream_sm_limit(calls, sms)
    torch.cuda.synchronize()
    try:
        for i in range(100):
            csa.cache_attention_forward(out, qd, cache, batch, workspace=ws[:need], stream=calls)
            with torch.cuda.stream(writer):
                for k in range(6):
                    for to, state in zip((off, lengths), states[k % 2]):
                        to.copy_(state)
        torch.cuda.synchronize()
        assert csa.get_status(calls) in (0, csa.CSA_ERR_INDEX)
        assert bool((big[:1000] == 7.0).all()) and bool((big[1000 + rows:] == 7.0).all())
        assert bool((ws[need:] == 85).all())
        for to, state in zip((off, lengths), states[0]):
            to.copy_(state)
        torch.cuda.synchronize()
        csa.cache_attention_forward(out, qd, cache, batch, workspace=ws[:need], stream=calls)
        assert csa.get_status(calls) == 0
    finally:
        csa.set_stream_sm_limit(calls, 0)
    want, bound = ref.attention(q, *b.values("k"), *b.values("v"), states[0][0].tolist(),
                                states[0][1].tolist(), b.table)
    err = (out.cpu().double() - want).abs()
    assert bool((err <= bound * 1.01 + want.abs() * 2.0 ** -8).all())
