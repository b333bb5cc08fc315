"""The rotary, cache and cache-attention calls past 2^31 bytes and elements: a cache whose pages
and rows whose tokens and heads lie that far apart give the bits of compact ones (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa

pytestmark = pytest.mark.gpu

Hq, Hkv, D, P = 4, 4, 128, 128
APART = 2 ** 30 + 64  # elements: three rows reach past 2^31 of them


@pytest.fixture(params=[0, 2], ids=["all_sms", "2_sms"])
def sms(request):
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, request.param)
    yield request.param
    torch.cuda.synchronize()
    csa.set_stream_sm_limit(stream, 0)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_pages_far_into_a_large_cache(dtype, sms):
    """Two sequences on the last pages of 2.2 GB of codes and on the first ones of a small cache."""
    pages = 2 ** 31 // (Hkv * P * D) + 40
    new, old = [150, 1], [90, 300]
    rows = sum(new)
    g = torch.Generator().manual_seed(1)
    first = torch.randn((sum(old), 2, Hkv, D), generator=g).to(torch.bfloat16).cuda()
    x = torch.randn((rows, 3, Hq, D), generator=g).to(torch.bfloat16).cuda()
    results = []
    for count, at in ((8, 0), (pages, pages - 8)):
        cache = csa.KvCache.empty(count, Hkv, P, D, dtype)
        table = at + torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
        csa.kv_cache_write(cache, csa.KvBatch(ints(0, old[0], sum(old)), ints(*old), table, rows=sum(old)),
                           first[:, 0], first[:, 1])
        batch = csa.KvBatch(ints(0, new[0], rows), ints(*(a + b for a, b in zip(new, old))), table, rows=rows)
        csa.kv_cache_write(cache, batch, x[:, 1], x[:, 2])
        out = csa.cache_attention(x[:, 0], cache, batch)
        k, v = (torch.empty((rows, Hkv, D), device="cuda") for _ in range(2))
        csa.kv_cache_read(k, v, cache, batch)
        assert csa.get_status() == 0
        results.append((out, k, v, cache.k[at: at + 8].clone(), cache.v[at: at + 8].clone()))
        del cache
    for a, b in list(zip(*results))[:3]:
        assert torch.equal(a, b)
    # the codes of tokens 0 .. length - 1 of each sequence
    for i in (3, 4):
        for s in range(2):
            n = new[s] + old[s]
            a, b = (r[i].view(torch.uint8)[4 * s: 4 * s + 4].transpose(1, 2).reshape(-1, Hkv, D)[:n]
                    for r in results)
            assert torch.equal(a, b)


def far_rows(compact, apart, buffer, offset):
    """`compact` [n, heads, D] in `buffer` with its tokens (or heads) APART elements apart."""
    n, heads, size = compact.shape
    strides = (APART, size, 1) if apart == "tokens" else (size, APART, 1)
    view = buffer.as_strided((n, heads, size), strides, offset)
    view.copy_(compact)
    return view


@pytest.mark.parametrize("apart", ["tokens", "heads"])
def test_rows_far_apart(apart, sms):
    """Three tokens (or heads) 2^30 elements apart: Q, K, V and the outputs."""
    n, heads = (3, 2) if apart == "tokens" else (70, 3)
    buffer = torch.empty(2 * APART + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(2)
    compact = [torch.randn((n, heads, D), generator=g).to(torch.bfloat16).cuda() for _ in range(3)]
    far = [far_rows(c, apart, buffer, 2 ** 15 * i) for i, c in enumerate(compact)]
    table = csa.RotaryTable(D)
    results = []
    for q, k, v in (compact, far):
        out = torch.empty_like(compact[0])
        if q is far[0]:
            out = far_rows(out, apart, buffer, 2 ** 17)
            back = [far_rows(compact[0], apart, buffer, 2 ** 18 + 2 ** 15 * i) for i in range(2)]
            turned = far_rows(compact[0], apart, buffer, 2 ** 19)
        else:
            back = [torch.empty_like(out) for _ in range(2)]
            turned = torch.empty_like(out)
        csa.rotary_forward(turned, q, table, start=7)
        csa.rotary_forward(k, k, table, start=7)
        cache = csa.KvCache.empty(2, heads, P, D)
        batch = csa.KvBatch(ints(0, n), ints(n + 5), ints(1, 0).view(1, 2), rows=n)
        csa.kv_cache_write(cache, csa.KvBatch(ints(0, 5), ints(5), ints(1, 0).view(1, 2), rows=5),
                           *(torch.full((5, heads, D), 0.5, dtype=torch.bfloat16, device="cuda"),) * 2)
        csa.kv_cache_write(cache, batch, k, v)
        csa.cache_attention_forward(out, turned, cache, batch)
        csa.kv_cache_read(*back, cache, batch)
        assert csa.get_status() == 0
        results.append([t.clone(memory_format=torch.contiguous_format) for t in (turned, k, out, *back)])
    for a, b in zip(*results):
        assert torch.equal(a, b)
