"""cache_attention_shared_forward against the definition in 64 bits, within the bound that
serving_ref.attention derives from its arithmetic plus one rounding to the type (GPU)."""
import pytest
import torch

import causal_attention_score_gb300 as csa
import shared_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=[(0, csa.SHARED_ALWAYS), (2, csa.SHARED_ALWAYS), (0, csa.SHARED_AUTO)],
                ids=["all_sms", "2_sms", "where_it_pays"])
def sms(request):
    """On the whole GPU, where the shared part is cut into many pieces, and held to two SMs, where
    every worker has many units; and as short a shared part as here is left to the sequences."""
    stream = torch.cuda.current_stream()
    csa.set_stream_sm_limit(stream, request.param[0])
    csa.set_shared_part(request.param[1])
    yield request.param
    torch.cuda.synchronize()
    csa.set_shared_part(csa.SHARED_AUTO)
    csa.set_stream_sm_limit(stream, 0)


def run(b, Hq, dtype, scale=None, q=None, **kw):
    q = b.rows_of(Hq, dtype, seed=11) if q is None else q
    cache, batch = b.device(csa)
    out = torch.full((b.rows, Hq, b.D), 7.0, dtype=dtype, device="cuda")
    csa.cache_attention_shared_forward(out, q.cuda(), cache, batch, *b.lists(), scale=scale, **kw)
    assert csa.get_status() == 0
    return q, out


def check(b, q, out, scale=None, what=""):
    want, room = ref.room(b, q, scale, out.dtype)
    n = b.offsets[-1]
    got = out.cpu().double()
    err = (got[:n] - want[:n]).abs()
    bad = ~(err <= room[:n])
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), float((err / room[:n])[bad].max()))
    assert bool((got[n:] == 7.0).all()), f"{what}: rows of no sequence"


CASES = [
    # new, old, groups (from, to, shared), Hq, Hkv, D, P
    ([1], [0], [(0, 1, 16)], 1, 1, 16, 16),
    ([1, 1, 1], [0, 5, 40], [(0, 3, 320)], 2, 2, 64, 64),                      # rows of 8
    ([1, 1, 1, 1], [3, 90, 1, 17], [(0, 4, 1040)], 12, 12, 64, 16),
    ([1, 2, 1, 3, 1], [0, 1, 2, 33, 100], [(0, 5, 224)], 6, 2, 80, 32),        # rows of 16
    ([1] * 6, [0, 10, 20, 30, 40, 300], [(0, 2, 128), (2, 6, 640)], 8, 2, 128, 128),
    ([1] * 9, list(range(9)), [(0, 9, 208)], 8, 2, 64, 16),                    # tcgen05: 36 rows, a tile's tail
    ([2, 1, 3, 1, 4], [0, 9, 300, 64, 1], [(0, 5, 576)], 16, 2, 128, 64),
    ([1] * 40, [(7 * i) % 50 for i in range(40)], [(0, 40, 1504)], 8, 1, 112, 32),  # 320 rows: two blocks
    ([1, 1, 1, 1, 1, 1], [0, 1, 2, 3, 4, 5], [(1, 3, 96), (3, 3, 64), (3, 5, 0)], 2, 2, 48, 32),  # some alone
    ([0, 1, 0, 2, 0], [0, 4, 0, 3, 9], [(0, 5, 160)], 4, 2, 32, 32),           # the first without rows
    ([30, 70, 1, 12], [0, 3, 50, 0], [(0, 4, 384)], 4, 2, 64, 64),             # prompts behind it
    ([25, 140], [0, 0], [(0, 1, 128), (1, 2, 256)], 3, 1, 96, 128),
    ([1] * 34, [60] * 34, [(0, 17, 480), (17, 34, 32)], 4, 2, 64, 16),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new,old,groups,Hq,Hkv,D,P", CASES)
def test_against_definition(new, old, groups, Hq, Hkv, D, P, dtype, fmt):
    b = ref.SharedBatch(new, old, groups, Hkv, D, P, fmt, seed=len(new) + D, extra_rows=2)
    q, out = run(b, Hq, dtype)
    check(b, q, out)
    # with all tables written out, cache_attention_forward's result
    cache, batch = b.device_whole(csa)
    whole = torch.full_like(out, 7.0)
    csa.cache_attention_forward(whole, q.cuda(), cache, batch)
    check(b, q, whole, what="cache_attention_forward")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("kind", ["large", "huge_bf16", "tiny_bf16", "zero", "negative_scale"])
def test_extreme_queries(kind, many):
    b = ref.SharedBatch([1] * (12 if many else 3), [i * 20 for i in range(12 if many else 3)],
                        [(0, 12 if many else 3, 448)], 2, 64, 64, "int8", seed=3)
    q, scale = b.rows_of(8, torch.bfloat16), None
    if kind == "large":
        q = q * 8
    elif kind == "huge_bf16":
        q, scale = (q.float() * 2.0 ** 100).to(torch.bfloat16), 2.0 ** -103
    elif kind == "tiny_bf16":
        q, scale = (q.float() * 2.0 ** -90).to(torch.bfloat16), 2.0 ** 87
    elif kind == "zero":
        q = q * 0
    else:
        scale = -0.3
    q, out = run(b, 8, torch.bfloat16, scale=scale, q=q)
    check(b, q, out, scale, kind)


@pytest.mark.parametrize("many", [False, True])
def test_a_row_without_numbers_spoils_itself_only(many):
    n = 12 if many else 3
    b = ref.SharedBatch([1] * n, [5] * n, [(0, n, 256)], 2, 64, 32, "e4m3", seed=4)
    q = b.rows_of(8, torch.bfloat16)
    good, out = run(b, 8, torch.bfloat16, q=q)
    spoiled = q.clone()
    spoiled[1, 3, 7] = float("nan")
    spoiled[2, 0, 0] = float("inf")
    _, got = run(b, 8, torch.bfloat16, q=spoiled)
    keep = torch.ones((n, 8), dtype=torch.bool)
    keep[1, 3] = keep[2, 0] = False
    assert torch.equal(got.cpu()[keep], out.cpu()[keep])
    assert not got.cpu()[1, 3].isfinite().any()


@pytest.mark.parametrize("many", [False, True])
def test_scales_of_v_far_apart(many):
    """Blocks of V far below and above others', and of scale 0, shared and own: every key counts."""
    n = 12 if many else 3
    b = ref.SharedBatch([1] * n, [40] * n, [(0, n, 320)], 2, 64, 32, "int8", seed=5)
    for i, s in enumerate((2.0 ** 34, 0.0, 2.0 ** -60, 2.0 ** -100)):
        b.scale["v"][b.table[0][2 * i]] = s
        b.scale["v"][b.table[1][10]] = 2.0 ** 40
        b.scale["v"][b.table[2][10]] = 0.0
    q, out = run(b, 8, torch.bfloat16)
    check(b, q, out)


def test_in_place_and_strides():
    b = ref.SharedBatch([1, 2, 1] * 5, [4] * 15, [(0, 15, 192)], 2, 64, 64, "int8", seed=6)
    q, want = run(b, 8, torch.bfloat16)
    cache, batch = b.device(csa)
    x = q.cuda()
    csa.cache_attention_shared_forward(x, x, cache, batch, *b.lists())
    assert torch.equal(x[: b.offsets[-1]], want[: b.offsets[-1]])
    packed = torch.zeros((b.rows, 3, 8, 64), dtype=torch.bfloat16, device="cuda")  # slices side by side
    packed[:, 0] = q.cuda()
    csa.cache_attention_shared_forward(packed[:, 2], packed[:, 0], cache, batch, *b.lists())
    assert torch.equal(packed[:, 2][: b.offsets[-1]], want[: b.offsets[-1]]) and bool((packed[:, 1] == 0).all())
    heads_first = torch.full((8, b.rows, 64), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    csa.cache_attention_shared_forward(heads_first, q.cuda(), cache, batch, *b.lists())
    assert torch.equal(heads_first[: b.offsets[-1]], want[: b.offsets[-1]])
    assert torch.equal(csa.cache_attention_shared(q.cuda(), cache, batch, *b.lists())[: b.offsets[-1]],
                       want[: b.offsets[-1]])
    assert csa.get_status() == 0


@pytest.mark.parametrize("many", [False, True])
def test_entries_that_break_the_rules(many):
    """What they name is left as it was and reported; the rest is computed."""
    n = 14 if many else 4
    b = ref.SharedBatch([1] * n, [3] * n, [(0, n // 2, 128), (n // 2, n, 64)], 2, 64, 32, "int8", seed=7)
    q = b.rows_of(8, torch.bfloat16)
    cache, batch = b.device(csa)
    groups, shared = b.lists()
    want, room = ref.room(b, q)
    ws = torch.empty(csa.cache_attention_shared_workspace_size(cache, batch, 8, 2), dtype=torch.uint8, device="cuda")

    def left(rows):  # rows that were left as they were; the others are right
        out = torch.full((n, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        csa.cache_attention_shared_forward(out, q.cuda(), cache, batch, groups, shared, workspace=ws)
        assert csa.get_status() == csa.CSA_ERR_INDEX
        got = out.cpu().double()
        for s in range(n):
            if s in rows:
                assert bool((got[s] == 7.0).all()), s
            else:
                assert bool(((got[s] - want[s]).abs() <= room[s]).all()), s

    first, second, every = range(n // 2), range(n // 2, n), range(n)
    for bad in (-32, 16, 33, 2 ** 30, -2 ** 31, 96 * 32):
        keep = int(shared[1])
        shared[1] = bad
        left(second)
        shared[1] = keep
    for at, bad in ((0, -1), (2, n + 1), (1, 2 ** 31 - 1), (1, -5)):
        keep = int(groups[at])
        groups[at] = bad
        left(every)
        groups[at] = keep
    keep = int(batch.lengths[1])
    batch.lengths[1] = 100  # a row among the shared tokens
    left([1])
    batch.lengths[1] = -3
    left([1])
    batch.lengths[1] = keep
    keep = batch.offsets.clone()
    batch.offsets[2] = 2 ** 30
    left([1, 2])
    batch.offsets.copy_(keep)
    # a shared page out of range is left out of its sums, and reported
    page = int(batch.table[0, 1])
    batch.table[0, 1] = 10 ** 6
    out = torch.full((n, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    csa.cache_attention_shared_forward(out, q.cuda(), cache, batch, groups, shared, workspace=ws)
    assert csa.get_status() == csa.CSA_ERR_INDEX
    assert bool(out.isfinite().all()) and not bool((out == 7.0).any())
    got = out.cpu().double()
    assert bool(((got[n // 2:] - want[n // 2:]).abs() <= room[n // 2:]).all())
    batch.table[0, 1] = page


def test_batches_that_overlap_rows_stay_within_the_workspace():
    """Offsets whose sequences, each for itself in order, name rows twice over: what is computed is not
    said, but nothing is written outside."""
    n = 6
    b = ref.SharedBatch([5] * n, [3] * n, [(0, 2, 64), (2, 4, 64), (4, 6, 64)], 2, 64, 32, "int8", seed=8)
    cache, batch = b.device(csa)
    q = b.rows_of(8, torch.bfloat16).cuda()
    need = csa.cache_attention_shared_workspace_size(cache, batch, 8, 3)
    ws = torch.full((need + 4096,), 85, dtype=torch.uint8, device="cuda")
    big = torch.full((b.rows + 200, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    batch.offsets.copy_(torch.tensor([0, 29, 1, 30, 2, 30, 30], dtype=torch.int32))
    batch.lengths.fill_(96)
    batch2 = csa.KvBatch(batch.offsets, batch.lengths, batch.table, rows=30, max_new=30)
    csa.cache_attention_shared_forward(big[100:130], q, cache, batch2, *b.lists(), workspace=ws[:need])
    assert csa.get_status() == csa.CSA_ERR_INDEX
    assert bool((big[:100] == 7.0).all()) and bool((big[130:] == 7.0).all()) and bool((ws[need:] == 85).all())


def test_captured_with_growing_sequences_and_a_dirty_workspace():
    b = ref.SharedBatch([1] * 20, [(i * 13) % 60 for i in range(20)], [(0, 8, 512), (8, 20, 96)], 2, 64, 32, "int8",
                        seed=9, width_extra=3)
    cache, batch = b.device(csa)
    groups, shared = b.lists()
    q = b.rows_of(8, torch.bfloat16)
    x, out = q.cuda(), torch.full((20, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(csa.cache_attention_shared_workspace_size(cache, batch, 8, 2), dtype=torch.uint8, device="cuda")
    csa.cache_attention_shared_forward(out, x, cache, batch, groups, shared, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.cache_attention_shared_forward(out, x, cache, batch, groups, shared, workspace=ws)
    for step in range(3):
        ws.fill_(255)
        out.fill_(7.0)
        graph.replay()
        assert csa.get_status() == 0
        check(b, q, out, what=step)
        # the sequences lose a token (what they hold stays), the groups' bounds move
        for s in range(20):
            if b.lengths[s] > b.shared[0 if s < 8 else 1] + 1:
                b.lengths[s] -= 1
        batch.lengths.copy_(torch.tensor(b.lengths, dtype=torch.int32))


def test_two_streams():
    made = [ref.SharedBatch([1] * 18, [i + 5 * k for i in range(18)], [(0, 18, 320)], 2, 64, 64, "int8", seed=20 + k)
            for k in range(2)]
    streams = [torch.cuda.Stream() for _ in made]
    args = [(b.device(csa), b.lists(), b.rows_of(8, torch.bfloat16)) for b in made]
    outs = [torch.full((18, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in made]
    qs = [q.cuda() for _, _, q in args]
    torch.cuda.synchronize()
    for _ in range(5):
        for ((cache, batch), lists, _), st, out, q in zip(args, streams, outs, qs):
            csa.cache_attention_shared_forward(out, q, cache, batch, *lists, stream=st)
    torch.cuda.synchronize()
    assert csa.get_status() == 0
    for b, (_, _, q), out in zip(made, args, outs):
        check(b, q, out)


def test_a_wait_that_runs_out_is_reported(sms):
    b = ref.SharedBatch([1] * 12, [5] * 12, [(0, 12, 320)], 2, 64, 64, "int8", seed=10)
    q, good = run(b, 8, torch.bfloat16)
    cache, batch = b.device(csa)
    out = torch.zeros_like(good)
    try:
        csa.set_wait_limit_ns(3_000_000)
        csa.debug_inject(True)
        csa.cache_attention_shared_forward(out, q.cuda(), cache, batch, *b.lists())
        # (a shared part left to the sequences has no such wait)
        assert csa.get_status() == (csa.CSA_ERR_TIMEOUT if sms[1] == csa.SHARED_ALWAYS else 0)
    finally:
        csa.set_wait_limit_ns(0)
        csa.debug_inject(False)
    csa.cache_attention_shared_forward(out, q.cuda(), cache, batch, *b.lists())
    assert csa.get_status() == 0 and torch.equal(out, good)


def test_one_sm(sms):
    b = ref.SharedBatch([1, 2, 1, 40], [7, 90, 0, 3], [(0, 3, 160), (3, 4, 64)], 2, 64, 32, "int8", seed=13)
    q = b.rows_of(8, torch.bfloat16)
    cache, batch = b.device(csa)
    st = torch.cuda.Stream()
    csa.set_stream_sm_limit(st, 1)
    try:
        out = torch.full((b.rows, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        x = q.cuda()
        torch.cuda.synchronize()
        csa.cache_attention_shared_forward(out, x, cache, batch, *b.lists(), stream=st)
        assert csa.get_status(st) == 0
    finally:
        csa.set_stream_sm_limit(st, 0)
    check(b, q, out)


def test_same_bits_every_time():
    b = ref.SharedBatch([1] * 30, [(i * 17) % 90 for i in range(30)], [(0, 30, 1600)], 2, 64, 32, "int8", seed=12)
    _, want = run(b, 8, torch.bfloat16)
    for _ in range(5):
        _, got = run(b, 8, torch.bfloat16)
        assert torch.equal(got, want)


@pytest.mark.parametrize("S,G", [(1300, 60), (270, 100), (200, 3)])
def test_many_sequences_and_groups(sms, S, G):
    """More than the plan's threads take at once, or keep to themselves."""
    bounds = [S * g // G for g in range(G + 1)]
    groups = [(bounds[g], bounds[g + 1], 16 * (g % 4)) for g in range(G)]
    b = ref.SharedBatch([1] * S, [i % 3 for i in range(S)], groups, 1, 16, 16, "int8", seed=14)
    q, out = run(b, 2, torch.bfloat16)
    check(b, q, out)


@pytest.mark.parametrize("many", [False, True])
def test_long_shared_parts(many, sms):
    """Long enough to be worked out apart of itself, against cache_attention_forward's result. Each of
    the two is off by serving_ref.attention's bound, (2 d + 2^-11) sum p|v| + N 2^-25 max|v| with
    d = (D + 8) 2^-24 max sum |q||k| scale + 2^-16 + N 2^-24, and a rounding to bf16; sum p|v| is the
    latter call's over |v|, which is off by its own rounding and bound (less than a tenth)."""
    n, heads = (40, 4) if many else (4, 2)
    b = ref.SharedBatch([1] * n, [(i * 11) % 70 for i in range(n)], [(0, n, 20000 // 64 * 64)], 4, 64, 64, "int8", seed=15)
    q, out = run(b, 4 * heads, torch.bfloat16)
    cache, batch = b.device_whole(csa)
    whole, spread = torch.full_like(out, 7.0), torch.full_like(out, 7.0)
    csa.cache_attention_forward(whole, q.cuda(), cache, batch)
    positive = csa.KvCache(cache.k, cache.v.clamp(min=-127).abs(), cache.k_scale, cache.v_scale)
    csa.cache_attention_forward(spread, q.cuda(), positive, batch)
    assert csa.get_status() == 0
    N = max(b.lengths)
    (kc, ks), (vc, vs) = b.values("k"), b.values("v")
    live = b.live.any(1)
    k = (kc.abs() * ks[..., None, None])[live].cuda()       # [pages, Hkv, P, D]
    x = q.double().abs().cuda().view(n, 4, heads, 64)
    A = max(float(torch.einsum("nhgd,hpd->nhgp", x, k[i].double()).max()) for i in range(len(k))) / 8
    d = 72 * 2.0 ** -24 * A + 2.0 ** -16 + N * 2.0 ** -24
    most = float((vc.abs() * vs[..., None, None])[live].max())
    one = (2 * d + 2.0 ** -11) * 1.1 * spread.double() + N * 2.0 ** -25 * most
    room = 2 * one * (1 + 2.0 ** -8) + 2.0 ** -8 * (out.double().abs() + whole.double().abs())
    assert bool(((out.double() - whole.double()).abs() <= room).all())


def test_workspace_that_is_too_small_or_misplaced():
    b = ref.SharedBatch([1], [5], [(0, 1, 32)], 1, 64, 16, "int8")
    cache, batch = b.device(csa)
    q = b.rows_of(2, torch.bfloat16).cuda()
    need = csa.cache_attention_shared_workspace_size(cache, batch, 2, 1)
    for ws, code in ((torch.empty(need - 1, dtype=torch.uint8, device="cuda"), csa.CSA_ERR_WORKSPACE),
                     (torch.empty(need + 16, dtype=torch.uint8, device="cuda")[4:], csa.CSA_ERR_ALIGN)):
        with pytest.raises(csa.CsaError) as e:
            csa.cache_attention_shared_forward(torch.empty_like(q), q, cache, batch, *b.lists(), workspace=ws)
        assert e.value.code == code
    with pytest.raises(ValueError, match="groups"):
        csa.cache_attention_shared_forward(torch.empty_like(q), q, cache, batch, b.lists()[1], b.lists()[1])
