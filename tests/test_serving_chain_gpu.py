"""From one dense layer to the next: packed QKV of a dense layer (fp32, rounded to the cache's
type by the caller), rotary positions, the cache, attention over it, the next dense layer; direct
and replayed from a graph (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref

pytestmark = pytest.mark.gpu

Hq, Hkv, D, P, WIDTH, I = 4, 2, 64, 32, 8, 192


def layer(X, W, Wo, table, cache, batch, pos, out):
    """Rows X [rows, I] through the layer: (packed QKV after its rotation, the result)."""
    qkv = csa.dense(X, W).to(X.dtype)
    x = qkv.view(-1, Hq + 2 * Hkv, D)
    qk = x[:, : Hq + Hkv]
    csa.rotary_forward(qk, qk, table, pos)
    csa.kv_cache_write(cache, batch, x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:])
    csa.cache_attention_forward(out, x[:, :Hq], cache, batch)
    return x, csa.dense(out.view(-1, Hq * D), Wo)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_dense_to_dense(fmt):
    """A prompt of 150 tokens and three single ones. QKV: fp32 sums of I exact products, then one
    rounding. The attention against the definition on the codes the GPU wrote. The result:
    fp32 sums of Hq * D exact products."""
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(4)
    W, Wo = (torch.randn(s, generator=g).mul(s[1] ** -0.5).to(dt) for s in
             (((Hq + 2 * Hkv) * D, I), (48, Hq * D)))
    Wd, Wod, table = W.cuda(), Wo.cuda(), csa.RotaryTable(D)
    f = ref.frequencies(D)
    cache = csa.KvCache.empty(WIDTH, Hkv, P, D, torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
    pages = list(range(WIDTH))[::-1]
    at = 0
    for n in (150, 1, 1, 1):
        X = torch.randn((n, I), generator=g).to(dt)
        pos = torch.arange(at, at + n)
        at += n
        batch = csa.KvBatch(*(torch.tensor(t, dtype=torch.int32, device="cuda")
                              for t in ([0, n], [at], [pages])), rows=n)
        out = torch.empty((n, Hq, D), dtype=dt, device="cuda")
        x, y = layer(X.cuda(), Wd, Wod, table, cache, batch, pos.to(torch.int32).cuda(), out)
        assert csa.get_status() == 0
        # Q, K, V: a sum off by I 2^-24 of its terms' size moves a rotated pair by as much of
        # both its elements; two roundings to bf16 and the rotation's own error
        X64, W64 = X.double(), W.double()
        exact = (X64 @ W64.T).view(n, -1, D)
        size = (X64.abs() @ W64.abs().T).view(n, -1, D) * (I * 2.0 ** -24) + exact.abs() * 2.0 ** -8
        want, pair = ref.rotary(exact[:, : Hq + Hkv], pos, f)
        _, moved = ref.rotary(size[:, : Hq + Hkv], pos, f)
        got = x.cpu().double()
        room = moved + pair * 2.0 ** -20
        room += (want.abs() + room) * 2.0 ** -8
        assert bool(((got[:, : Hq + Hkv] - want).abs() <= room).all())
        assert bool(((got[:, Hq + Hkv:] - exact[:, Hq + Hkv:]).abs() <= size[:, Hq + Hkv:] * 1.01).all())
        held = []
        for name in ("k", "v"):
            c = getattr(cache, name).float().double().cpu()
            live = (torch.arange(WIDTH * P) < at).view(WIDTH, P)
            order = torch.empty(WIDTH, dtype=torch.long)
            order[torch.tensor(pages)] = torch.arange(WIDTH)
            held += [torch.where(live[order][:, None, :, None], c, 0.0), getattr(cache, name + "_scale").double().cpu()]
        att, bound = ref.attention(x[:, :Hq].cpu(), *held, [0, n], [at], [pages])
        o = out.cpu().double()
        assert bool(((o - att).abs() <= bound * 1.01 + att.abs() * 2.0 ** -8).all())
        flat, Wo64 = o.view(n, -1), Wo.double()
        assert bool(((y.cpu().double() - flat @ Wo64.T).abs()
                     <= Hq * D * 2.0 ** -24 * (flat.abs() @ Wo64.abs().T)).all())


def test_replayed_chain_equals_direct_calls():
    """Single-token steps of two sequences through the layer from one graph: the direct calls' bits."""
    S = 2
    g = torch.Generator().manual_seed(5)
    W, Wo = (torch.randn(s, generator=g).mul(s[1] ** -0.5).to(torch.bfloat16).cuda() for s in
             (((Hq + 2 * Hkv) * D, I), (48, Hq * D)))
    table = csa.RotaryTable(D)
    Xs = [torch.randn((S, I), generator=g).to(torch.bfloat16).cuda() for _ in range(40)]
    runs = []
    for graphed in (False, True):
        cache = csa.KvCache.empty(S * WIDTH, Hkv, P, D)
        pages = torch.arange(S * WIDTH, dtype=torch.int32, device="cuda").view(S, WIDTH)
        lengths = torch.zeros(S, dtype=torch.int32, device="cuda")
        batch = csa.KvBatch(torch.arange(S + 1, dtype=torch.int32, device="cuda"), lengths, pages, rows=S, max_new=1)
        X, pos = torch.zeros_like(Xs[0]), torch.zeros(S, dtype=torch.int32, device="cuda")
        out = torch.empty((S, Hq, D), dtype=torch.bfloat16, device="cuda")

        def step():
            pos.copy_(lengths)
            lengths.add_(1)
            return layer(X, W, Wo, table, cache, batch, pos, out)[1]

        graph = torch.cuda.CUDAGraph()
        if graphed:
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                y = step()
        got = []
        for x in Xs:
            X.copy_(x)
            if graphed:
                graph.replay()
            else:
                y = step()
            got.append(y.clone())
        assert csa.get_status() == 0
        runs.append(torch.stack(got))
    assert torch.equal(*runs)
