"""cache_attention_forward against the definition in 64 bits, within the bound that
serving_ref.attention derives from its arithmetic plus one rounding to the type (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=[0, 2], ids=["all_sms", "2_sms"])
def sms(request):
    """Every test on the whole GPU, where a short batch has a kernel for few rows, and held
    to two SMs, where sequences of many rows take the kernel for prompts and every worker
    has many units."""
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, request.param)
    yield request.param
    torch.cuda.synchronize()
    csa.set_stream_sm_limit(stream, 0)


def run(b: ref.Batch, Hq, dtype, window=0, sinks=0, scale=None, q=None, q_scale=1.0):
    q = b.rows_of(Hq, dtype, q_scale, seed=11) if q is None else q
    cache, batch = b.device(csa)
    out = torch.full((b.rows, Hq, b.D), 7.0, dtype=dtype, device="cuda")
    csa.cache_attention_forward(out, q.cuda(), cache, batch, scale=scale, window=window, sinks=sinks)
    assert csa.get_status() == 0
    return q, out


def check(b, q, out, dtype, window=0, sinks=0, scale=None, what="", skip=None,
          hidden=None):
    kc, ks = b.values("k")
    vc, vs = b.values("v")
    want, bound = ref.attention(q, kc, ks, vc, vs, b.offsets, b.lengths, b.table, window, sinks, scale,
                                hidden)
    n = b.offsets[-1]
    got = out.cpu().double()
    err = (got[:n] - want[:n]).abs()
    room = bound[:n] * (1 + ref.half_step(dtype)) + want[:n].abs() * ref.half_step(dtype) + \
        (2.0 ** -25 if dtype == torch.float16 else 0.0)
    bad = ~(err <= room)
    if skip is not None:
        bad &= ~skip[:n, :, None]
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(),
                           float((err / room)[bad].max()))
    assert bool((got[n:] == 7.0).all()), f"{what}: rows of no sequence"


CASES = [
    # new, old, Hq, Hkv, D, P, window, sinks
    ([1], [0], 1, 1, 16, 16, 0, 0),
    ([1], [776], 12, 12, 64, 64, 0, 0),
    ([1, 1, 1, 1, 1], [0, 1, 62, 63, 64], 4, 2, 64, 32, 0, 0),
    ([1, 2, 5], [1000, 17, 0], 8, 1, 128, 16, 0, 0),
    ([3, 1, 0, 9], [130, 4, 10, 0], 6, 2, 80, 64, 0, 0),
    ([1] * 40, list(range(0, 400, 10)), 3, 3, 48, 32, 0, 0),
    ([1, 1, 2], [500, 3, 90], 8, 2, 128, 32, 64, 4),
    ([1, 4], [700, 300], 7, 1, 64, 128, 33, 0),
    ([2, 1], [300, 64], 4, 4, 112, 16, 1, 0),
    ([1, 1], [400, 200], 2, 2, 64, 64, 100, 130),
    ([6, 1], [300, 900], 4, 2, 128, 64, 2 ** 31 - 1, 5),
    ([40, 7], [30, 100], 4, 2, 64, 16, 0, 0),
    ([70, 130, 1], [0, 65, 500], 4, 1, 128, 64, 0, 0),
    ([150, 33], [70, 200], 2, 2, 64, 32, 40, 3),
    ([129], [0], 3, 3, 32, 128, 0, 0),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new,old,Hq,Hkv,D,P,window,sinks", CASES)
def test_against_definition(new, old, Hq, Hkv, D, P, window, sinks, dtype, fmt):
    b = ref.Batch(new, old, Hkv, D, P, fmt, seed=len(new) + D, extra_rows=2)
    q, out = run(b, Hq, dtype, window, sinks)
    check(b, q, out, dtype, window, sinks)


@pytest.mark.parametrize("n", [1, 200])
def test_rows_that_see_nothing(n):
    """Length zero, and rows before a sequence's beginning: zeros."""
    b = ref.Batch([n, 3], [0, 5], 2, 64, 16, "e4m3", seed=1)
    cache, _ = b.device(csa)
    off, length, table = b.ints()
    q = b.rows_of(4, torch.bfloat16)
    for short in (0, n // 2):
        length[0] = short
        out = torch.full((b.rows, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        csa.cache_attention_forward(out, q.cuda(), cache,
                                    csa.KvBatch(off, length, table, rows=b.rows))
        assert csa.get_status() == 0
        assert bool((out[: n - short] == 0).all())
        b.lengths[0] = short
        kc, ks = b.values("k")
        vc, vs = b.values("v")
        want, bound = ref.attention(q, kc, ks, vc, vs, b.offsets, b.lengths, b.table)
        err = (out.cpu().double() - want).abs()
        assert bool((err <= bound * 1.01 + want.abs() * 2.0 ** -8).all())


@pytest.mark.parametrize("new,old", [([1, 1], [3000, 50]), ([200], [300])])
@pytest.mark.parametrize("kind", ["large", "huge_bf16", "tiny_bf16", "zero"])
def test_extreme_queries(kind, new, old):
    """Scores that saturate the softmax, queries outside fp16's range in bf16, zeros."""
    b = ref.Batch(new, old, 2, 64, 64, "int8", seed=3)
    q = b.rows_of(4, torch.bfloat16)
    scale = None
    if kind == "large":
        q = q * 8
    elif kind == "huge_bf16":
        q, scale = (q.float() * 2.0 ** 100).to(torch.bfloat16), 2.0 ** -103
    elif kind == "tiny_bf16":
        q, scale = (q.float() * 2.0 ** -90).to(torch.bfloat16), 2.0 ** 87
    else:
        q = q * 0
    q, out = run(b, 4, torch.bfloat16, scale=scale, q=q)
    check(b, q, out, torch.bfloat16, scale=scale, what=kind)


def test_infinite_and_nan_queries_stay_in_their_rows():
    b = ref.Batch([4, 150], [100, 20], 1, 64, 32, "int8", seed=5)
    q = b.rows_of(3, torch.float16)
    bad = q.clone()
    bad[1, 2, 7] = float("nan")
    bad[20, 0, 3] = float("inf")
    _, out = run(b, 3, torch.float16, q=bad)
    hit = torch.zeros((b.rows, 3), dtype=torch.bool)
    hit[1, 2] = hit[20, 0] = True
    check(b, q, out, torch.float16, what="others", skip=hit)
    assert bool(out.cpu()[hit].isnan().any(-1).all())


def test_blocks_of_very_different_scales():
    """Scales from 2^-60 to 2^20 within one sequence: each block counts with its own."""
    for new, old in (([1], [400]), ([160], [300])):
        b = ref.Batch(new, old, 1, 64, 16, "e4m3", seed=6)
        n = -(-b.lengths[0] // 16)
        for i, p in enumerate(b.table[0][:n]):
            b.scale["v"][p, 0] = 2.0 ** ((i * 37) % 81 - 60)
            b.scale["k"][p, 0] = 2.0 ** (-(i % 5) - 4)
        q, out = run(b, 2, torch.bfloat16)
        check(b, q, out, torch.bfloat16)


def test_strided_queries_and_outputs():
    """Q inside a packed QKV row, the output head-major: same bits as contiguous tensors."""
    for new, old in (([1, 5], [77, 200]), ([140, 3], [10, 60])):
        b = ref.Batch(new, old, 2, 64, 16, "int8", seed=7)
        packed = torch.randn((b.rows, 8, 64), generator=b.g).to(torch.bfloat16).cuda()
        cache, batch = b.device(csa)
        want = torch.empty((b.rows, 4, 64), dtype=torch.bfloat16, device="cuda")
        csa.cache_attention_forward(want, packed[:, :4].contiguous(), cache, batch)
        out = torch.zeros((4, b.rows, 64), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        csa.cache_attention_forward(out, packed[:, :4], cache, batch)
        assert torch.equal(out, want)


def test_page_order_and_shared_pages():
    """The same tokens on other pages give the same bits, and two sequences may share full
    pages of a common prefix."""
    b = ref.Batch([1, 1], [150, 150], 2, 64, 32, "int8", seed=9)
    b.table[1][:3] = b.table[0][:3]
    q = b.rows_of(4, torch.bfloat16)
    q, out = run(b, 4, torch.bfloat16, q=q)
    check(b, q, out, torch.bfloat16)
    perm = torch.randperm(b.pages, generator=b.g)
    back = torch.argsort(perm)
    for d in (b.codes, b.scale):
        for name in d:
            d[name] = d[name].view(torch.uint8)[perm].view(d[name].dtype) if d is b.codes else d[name][perm]
    b.table = [[int(back[p]) if p >= 0 else p for p in row] for row in b.table]
    _, again = run(b, 4, torch.bfloat16, q=q)
    assert torch.equal(out, again)


@pytest.mark.parametrize("new,old", [([1, 2], [900, 100]), ([200, 1], [100, 500])])
def test_repeatable_limited_and_captured(new, old, sms):
    """Same bits call after call; an SM limit changes no more than the sums' order; a
    captured call follows its inputs and lengths."""
    b = ref.Batch(new, old, 2, 128, 64, "int8", seed=10)
    q, first = run(b, 4, torch.bfloat16)
    _, second = run(b, 4, torch.bfloat16)
    assert torch.equal(first, second)
    cache, batch = b.device(csa)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(first)
    csa.set_stream_sm_limit(st, 5)
    try:
        with torch.cuda.stream(st):
            qd = q.cuda()
            csa.cache_attention_forward(out, qd, cache, batch)
    finally:
        csa.set_stream_sm_limit(st, 0)
    torch.cuda.synchronize()
    check(b, q, out, torch.bfloat16, what="limited")
    ws = torch.empty(csa.cache_attention_workspace_size(cache, batch, 4), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    graph = torch.cuda.CUDAGraph()
    csa.set_stream_sm_limit(st, sms)
    try:
        with torch.cuda.graph(graph, stream=st):
            csa.cache_attention_forward(out, qd, cache, batch, workspace=ws)
    finally:
        csa.set_stream_sm_limit(st, 0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    batch.lengths.sub_(37)
    b.lengths = [n - 37 for n in b.lengths]
    graph.replay()
    torch.cuda.synchronize()
    check(b, q, out, torch.bfloat16, what="shorter")


@pytest.mark.parametrize("new,old", [([1, 4, 2], [300, 50, 0]), ([150, 30], [70, 200])])
def test_in_place(new, old):
    """The output over Q itself, inside a packed row: the same bits, its neighbours untouched."""
    b = ref.Batch(new, old, 2, 64, 32, "e4m3", seed=15, extra_rows=1)
    q, want = run(b, 4, torch.float16)
    cache, batch = b.device(csa)
    packed = torch.full((b.rows, 8, 64), 7.0, dtype=torch.float16, device="cuda")
    packed[:, 2:6] = q.cuda()
    n = b.offsets[-1]
    csa.cache_attention_forward(packed[:, 2:6], packed[:, 2:6], cache, batch)
    assert csa.get_status() == 0
    assert torch.equal(packed[:n, 2:6], want[:n])
    assert torch.equal(packed[n:, 2:6].cpu(), q[n:])
    assert bool((packed[:, :2] == 7.0).all()) and bool((packed[:, 6:] == 7.0).all())


@pytest.mark.parametrize("new,old,window", [([1] * 70, [1] * 69 + [2000], 0), ([1] * 9, [128 * i for i in range(9)], 0),
                                            ([1, 1, 2], [5000, 3, 40], 200), ([1], [20000], 0)])
def test_units_shared_by_many_groups(new, old, window):
    """Runs that end at a unit's first tile, inside it and after it; one-tile units in a row."""
    b = ref.Batch(new, old, 3, 64, 64, "int8", seed=16)
    q, out = run(b, 3, torch.bfloat16, window, 4)
    check(b, q, out, torch.bfloat16, window, 4)


def test_withheld_codes_time_out_and_recover():
    """The prompt kernel's bounded waits: codes that never arrive end in a status."""
    b = ref.Batch([300, 260], [40, 500], 2, 64, 32, "int8", seed=17)
    q = b.rows_of(8, torch.bfloat16).cuda()
    cache, batch = b.device(csa)
    out = torch.empty_like(q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    csa.set_stream_sm_limit(st, 2)
    assert csa.get_status() == 0
    csa.set_wait_limit_ns(20_000_000)  # 20 ms
    try:
        with torch.cuda.stream(st):
            csa.debug_inject(True)
            csa.cache_attention_forward(out, q, cache, batch)
            assert csa.get_status(st) == csa.CSA_ERR_TIMEOUT
            assert csa.get_status(st) == 0
            csa.set_wait_limit_ns(0)
            csa.cache_attention_forward(out, q, cache, batch)
            assert csa.get_status(st) == 0
    finally:
        csa.set_wait_limit_ns(0)
        csa.debug_inject(False)
        csa.set_stream_sm_limit(st, 0)
    check(b, q.cpu(), out, torch.bfloat16, what="after the timeout")


def test_workspace_that_is_too_small_or_absent():
    b = ref.Batch([1], [5], 1, 64, 16, "int8")
    cache, batch = b.device(csa)
    q = b.rows_of(2, torch.bfloat16).cuda()
    out = torch.full_like(q, 3.0)
    need = csa.cache_attention_workspace_size(cache, batch, 2)
    with pytest.raises(csa.CsaError) as e:
        csa.cache_attention_forward(out, q, cache, batch,
                                    workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.code == csa.CSA_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())


def test_bad_pages_are_masked_and_reported():
    """A block whose page number is out of range is left out of the sums (checked by the
    kernel), and the status says so."""
    for new, old in (([1, 1], [100, 100]), ([150, 1], [100, 100])):
        b = ref.Batch(new, old, 2, 64, 32, "int8", seed=12)
        q = b.rows_of(2, torch.bfloat16)
        cache, _ = b.device(csa)
        off, length, table = b.ints()
        table[0, 1] = b.pages
        out = torch.empty((b.rows, 2, 64), dtype=torch.bfloat16, device="cuda")
        csa.cache_attention_forward(out, q.cuda(), cache, csa.KvBatch(off, length, table, rows=b.rows))
        assert csa.get_status() == csa.CSA_ERR_INDEX
        gone = torch.zeros(b.lengths[0], dtype=torch.bool)
        gone[32:64] = True
        check(b, q, out, torch.bfloat16, hidden={0: gone})


def test_two_streams_at_once():
    """Two calls side by side with workspaces of their own."""
    bs = [ref.Batch([1, 1], [600 + i, 40], 2, 64, 64, "int8", seed=20 + i) for i in range(2)]
    ready, outs = [], []
    for b in bs:
        cache, batch = b.device(csa)
        q = b.rows_of(4, torch.float16, seed=11)
        ready.append((b, q, q.cuda(), cache, batch, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for b, q, qd, cache, batch, st in ready:
        out = torch.full((b.rows, 4, 64), 7.0, dtype=torch.float16, device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        csa.cache_attention_forward(out, qd, cache, batch, stream=st)
        outs.append(out)
    torch.cuda.synchronize()
    for (b, q, *_), out in zip(ready, outs):
        check(b, q, out, torch.float16)
