"""The calls together, as a model's layer makes them: packed QKV from the dense layer's
output, rotary positions, the cache, attention over it, and the output as the next dense
layer's X; prompts in chunks and then single tokens, direct and captured into a graph (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref

pytestmark = pytest.mark.gpu

Hq, Hkv, D, P, WIDTH = 4, 2, 64, 32, 6


def step(qkv, table, cache, batch, pos, out):
    """One layer's attention: rows [rows, (Hq + 2 Hkv) * D], rotated in place."""
    x = qkv.view(-1, Hq + 2 * Hkv, D)
    qk = x[:, : Hq + Hkv]
    csa.rotary_forward(qk, qk, table, pos)
    csa.kv_cache_write(cache, batch, x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:])
    csa.cache_attention_forward(out, x[:, :Hq], cache, batch)


def reference(qkv, pos, f, mem):
    """The same in 64 bits on one sequence; `mem`: its cache ({name: (codes, scale)})."""
    x = qkv.view(-1, Hq + 2 * Hkv, D)
    rot, _ = ref.rotary(x[:, : Hq + Hkv], pos, f)
    rot = rot.to(qkv.dtype)
    n, L = len(pos), int(pos[-1]) + 1
    for name, rows in (("k", rot[:, Hq:]), ("v", x[:, Hq + Hkv:])):
        ref.write(*mem[name], rows, [0, n], [L], [list(range(WIDTH))], mem["fmt"])
    return ref.attention(rot[:, :Hq], *mem["k"], *mem["v"], [0, n], [L], [list(range(WIDTH))])


@pytest.fixture(params=[0, 2], ids=["all_sms", "2_sms"])
def sms(request):
    """The whole GPU (few rows for it: one kernel) or two SMs (prompts take the other)."""
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, request.param)
    yield request.param
    torch.cuda.synchronize()
    csa.set_stream_sm_limit(stream, 0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_prompt_chunks_then_tokens(fmt, sms):
    """Bits of K that round the other way on the GPU move a code by one step at most, so the
    room is that of the derived bound, the output's half step, and of one code in 128 keys;
    the two paths' outputs over the whole run differ by 2^-6 of the values' size at most."""
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(1)
    table, f = csa.RotaryTable(D), ref.frequencies(D)
    S = 2
    cache = csa.KvCache.empty(S * WIDTH, Hkv, P, D,
                              torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
    pages = torch.arange(S * WIDTH, dtype=torch.int32).view(S, WIDTH)
    mem = [{"fmt": fmt, **{n: (torch.zeros((WIDTH, Hkv, P, D), dtype=torch.float64),
                               torch.zeros((WIDTH, Hkv), dtype=torch.float64)) for n in "kv"}}
           for _ in range(S)]
    length = [0, 0]
    for chunk in ([70, 33], [40, 1], [1, 1], [1, 1], [3, 2]):
        rows = sum(chunk)
        qkv = torch.randn((rows, (Hq + 2 * Hkv) * D), generator=g).to(dt)
        pos = torch.cat([length[s] + torch.arange(chunk[s]) for s in range(S)])
        length = [a + b for a, b in zip(length, chunk)]
        off = torch.tensor([0, chunk[0], rows], dtype=torch.int32, device="cuda")
        batch = csa.KvBatch(off, torch.tensor(length, dtype=torch.int32, device="cuda"),
                            pages.cuda(), rows=rows, max_new=max(chunk))
        out = torch.empty((rows, Hq, D), dtype=dt, device="cuda")
        step(qkv.cuda(), table, cache, batch, pos.to(torch.int32).cuda(), out)
        assert csa.get_status() == 0
        at = 0
        for s in range(S):
            want, bound = reference(qkv[at: at + chunk[s]], pos[at: at + chunk[s]], f, mem[s])
            got = out[at: at + chunk[s]].cpu().double()
            vmax = float((mem[s]["v"][0] * mem[s]["v"][1][..., None, None]).abs().max())
            assert bool(((got - want).abs() <= bound + want.abs() * 2.0 ** -8 + vmax * 2.0 ** -6).all())
            at += chunk[s]
    # the next layer takes the output as it is
    W = torch.randn((24, Hq * D), generator=g).to(dt)
    y = csa.dense(out.view(rows, Hq * D), W.cuda())
    want = out.view(rows, Hq * D).cpu().double() @ W.double().T
    # fp32 sums of 256 exact products
    room = 256 * 2.0 ** -24 * (out.view(rows, Hq * D).cpu().double().abs() @ W.double().abs().T)
    assert bool(((y.cpu().double() - want).abs() <= room).all())


def test_captured_step_equals_direct_steps():
    """Eight single-token steps replayed from one graph, the lengths and positions advanced
    in place, against the same steps called directly: same bits."""
    dt, S = torch.float16, 3
    table = csa.RotaryTable(D)
    g = torch.Generator().manual_seed(2)
    xs = [torch.randn((S, (Hq + 2 * Hkv) * D), generator=g).to(dt).cuda() for _ in range(8)]
    pages = torch.randperm(S * WIDTH, generator=g).to(torch.int32).view(S, WIDTH).cuda()
    start = torch.tensor([0, 31, 100], dtype=torch.int32, device="cuda")
    fill = torch.randn((131, Hkv, D), generator=g).to(dt).cuda()

    def fresh():
        cache = csa.KvCache.empty(S * WIDTH, Hkv, P, D)
        off = torch.tensor([0, 0, 31, 131], dtype=torch.int32, device="cuda")
        csa.kv_cache_write(cache, csa.KvBatch(off, start, pages, rows=131), fill, fill)
        lengths = start.clone()
        return cache, csa.KvBatch(torch.arange(S + 1, dtype=torch.int32, device="cuda"), lengths,
                                  pages, rows=S, max_new=1)

    def advance(batch, pos):
        pos.copy_(batch.lengths)
        batch.lengths.add_(1)

    cache, batch = fresh()
    pos, out = torch.empty_like(start), torch.empty((S, Hq, D), dtype=dt, device="cuda")
    want = []
    for x in xs:
        advance(batch, pos)
        step(x.clone(), table, cache, batch, pos, out)
        want.append(out.clone())
    cache2, batch2 = fresh()
    x2 = torch.empty_like(xs[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        advance(batch2, pos)
        step(x2, table, cache2, batch2, pos, out)
    for x, w in zip(xs, want):
        x2.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    n = int(batch.lengths.sum())
    held = []
    for c in (cache, cache2):
        off = torch.tensor([0, 8, 47, n], dtype=torch.int32, device="cuda")
        kv = [torch.empty((n, Hkv, D), device="cuda") for _ in range(2)]
        csa.kv_cache_read(*kv, c, csa.KvBatch(off, batch.lengths, pages, rows=n))
        held.append(kv)
    assert torch.equal(held[0][0], held[1][0]) and torch.equal(held[0][1], held[1][1])
    assert csa.get_status() == 0
