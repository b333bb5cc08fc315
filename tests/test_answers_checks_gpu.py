"""The checking build (-DCSA_DEBUG) on attention with shared beginnings: no check of units, parts,
ring places and TMEM columns fails, and the bits are the release library's; and lists and lengths
that change while such calls and those on a cache's books are under way (GPU)."""
import ctypes

import pytest
import torch

import causal_attention_score_gb300 as csa
import shared_ref as ref
from causal_attention_score_gb300 import _lib, build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checking():
    lib = ctypes.CDLL(build_lib.build(debug=True))
    for name, (res, args) in _lib.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


@pytest.mark.parametrize("sms", [0, 2])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new,old,groups,Hq,Hkv,D,P", [
    ([1], [0], [(0, 1, 16)], 1, 1, 16, 16),
    ([1, 1, 1, 1], [3, 90, 1, 17], [(0, 4, 1040)], 12, 12, 64, 16),
    ([1, 2, 1, 3, 1], [0, 1, 2, 33, 100], [(0, 5, 224)], 6, 2, 80, 32),
    ([1] * 9, list(range(9)), [(0, 4, 208), (4, 9, 608)], 24, 2, 64, 16),
    ([2, 1, 3, 1, 4], [0, 9, 300, 64, 1], [(0, 5, 576)], 16, 2, 128, 64),
    ([1] * 66, [(7 * i) % 50 for i in range(66)], [(0, 66, 1536)], 8, 2, 128, 128),
    ([150, 400, 3], [0, 0, 70], [(0, 3, 320)], 4, 2, 64, 64),
])
def test_no_check_fails(checking, monkeypatch, new, old, groups, Hq, Hkv, D, P, fmt, sms):
    b = ref.SharedBatch(new, old, groups, Hkv, D, P, fmt, seed=D + P)
    q = b.rows_of(Hq, torch.float16, seed=3).cuda()

    def call():
        stream = torch.cuda.current_stream()
        csa.set_stream_sm_limit(stream, sms)
        csa.set_shared_part(csa.SHARED_ALWAYS)
        try:
            cache, batch = b.device(csa)
            out = torch.zeros_like(q)
            csa.cache_attention_shared_forward(out, q, cache, batch, *b.lists())
            assert csa.get_status() == 0, "a device check failed"
            return out
        finally:
            csa.set_shared_part(csa.SHARED_AUTO)
            csa.set_stream_sm_limit(stream, 0)

    want = call()
    with monkeypatch.context() as m:
        m.setattr(_lib, "_lib", checking)
        got = call()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("sms", [0, 2])
def test_arrays_that_change_under_shared_calls(sms):
    """Two valid states of a batch and its groups written in turn from another stream while 60 calls
    run, which the calls do not allow: what they compute is undefined, but they write nothing outside
    their rows and workspace, end, and leave the next call as it should be."""
    S = 40
    new = [1] * S
    new[3], new[20], new[-1] = 60, 9, 33
    other = new[::-1]
    groups = [(0, 12, 128), (12, 30, 64), (30, 40, 96)]
    b = ref.SharedBatch([max(x) for x in zip(new, other)], [(i * 37) % 60 for i in range(S)], groups, 2, 32, 32, "int8")
    whole = b.device_whole(csa)[1].table
    states = []
    for n, bounds, shared in ((new, [0, 12, 30, 40], [128, 64, 96]), (other, [2, 25, 25, 31], [64, 0, 64])):
        off = [sum(n[:i]) for i in range(S + 1)]
        length = [b.lengths[i] - b.new[i] + n[i] for i in range(S)]
        states.append([torch.tensor(t, dtype=torch.int32, device="cuda") for t in (off, length, bounds, shared)])
    rows = sum(new)
    cache, _ = b.device(csa)
    arrays = [t.clone() for t in states[0]]
    off, lengths, bounds, shared = arrays
    batch = csa.KvBatch(off, lengths, whole, rows=rows, max_new=60)
    q = b.rows_of(8, torch.bfloat16)[:rows].contiguous().cuda()
    big = torch.full((rows + 2000, 8, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[1000: 1000 + rows]
    need = csa.cache_attention_shared_workspace_size(cache, batch, 8, 3)
    ws = torch.full((need + 2 ** 16,), 85, dtype=torch.uint8, device="cuda")
    calls, writer = torch.cuda.Stream(), torch.cuda.Stream()
    csa.set_stream_sm_limit(calls, sms)
    csa.set_shared_part(csa.SHARED_ALWAYS)
    torch.cuda.synchronize()
    try:
        quiet = torch.zeros_like(out)
        csa.cache_attention_shared_forward(quiet, q, cache, batch, bounds, shared, workspace=ws[:need], stream=calls)
        assert csa.get_status(calls) == 0
        for i in range(60):
            csa.cache_attention_shared_forward(out, q, cache, batch, bounds, shared, workspace=ws[:need], stream=calls)
            with torch.cuda.stream(writer):
                for k in range(6):
                    for to, state in zip(arrays, states[k % 2]):
                        to.copy_(state)
        torch.cuda.synchronize()
        assert csa.get_status(calls) in (0, csa.CSA_ERR_INDEX)
        assert bool((big[:1000] == 7.0).all()) and bool((big[1000 + rows:] == 7.0).all())
        assert bool((ws[need:] == 85).all())
        for to, state in zip(arrays, states[0]):
            to.copy_(state)
        torch.cuda.synchronize()
        csa.cache_attention_shared_forward(out, q, cache, batch, bounds, shared, workspace=ws[:need], stream=calls)
        assert csa.get_status(calls) == 0
        assert torch.equal(out, quiet)
    finally:
        csa.set_shared_part(csa.SHARED_AUTO)
        csa.set_stream_sm_limit(calls, 0)


def test_books_that_change_under_calls():
    """refs, lengths and lists written from another stream while calls on the books run: nothing
    outside them and the cache is written, and the calls end."""
    pages, S, width = 300, 30, 12
    held = torch.full((3 * 4096 + pages + S + S * width,), 77, dtype=torch.int32, device="cuda")
    refs, lengths = held[4096: 4096 + pages], held[8192 + pages: 8192 + pages + S]
    table = held[-4096 - S * width: -4096].view(S, width)
    guard = torch.ones_like(held, dtype=torch.bool)
    for t in (refs, lengths, table):
        at = (t.data_ptr() - held.data_ptr()) // 4
        guard[at: at + t.numel()] = False
    for t in (refs, lengths, table):
        t.zero_()
    pool = torch.full((2, pages + 2, 2, 16, 32), 5, dtype=torch.int8, device="cuda")
    scales = torch.zeros((2, pages, 2), device="cuda")
    cache = csa.KvCache(pool[0, 1:-1], pool[1, 1:-1], scales[0], scales[1])
    books = csa.KvPages(refs, lengths, table, 16)
    csa.kv_pages_extend(books, torch.arange(10, dtype=torch.int32, device="cuda"),
                        torch.arange(10, 110, 10, dtype=torch.int32, device="cuda"))
    first = [t.clone() for t in (refs, lengths, table)]
    lists = torch.arange(S, dtype=torch.int32, device="cuda")
    parents, children, more = lists[:8].clone(), lists[12:20].clone(), torch.full((8,), 17, dtype=torch.int32, device="cuda")
    moves, used = torch.zeros((pages,), dtype=torch.int32, device="cuda"), torch.zeros((1,), dtype=torch.int32, device="cuda")
    need = csa.kv_pages_workspace_size(books, 8)
    ws = torch.full((need + 4096,), 85, dtype=torch.uint8, device="cuda")
    writer = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(40):
        csa.kv_cache_fork(cache, books, parents, children, workspace=ws[:need])
        csa.kv_pages_extend(books, children, more, workspace=ws[:need])
        csa.kv_pages_free(books, children)
        csa.kv_cache_compact(cache, books, moves, used, workspace=ws[:need])
        with torch.cuda.stream(writer):
            for t, s in zip((refs, lengths, table), first):
                t.copy_(s)
            parents.random_(0, S)
            children.random_(0, S)
            table.random_(-5, pages + 5)
            lengths.random_(0, width * 16)
            refs.random_(0, 3)
    torch.cuda.synchronize()
    assert csa.get_status() in (0, csa.CSA_ERR_INDEX, csa.CSA_ERR_PAGES)
    assert bool((held[guard] == 77).all()) and bool((ws[need:] == 85).all())
    assert bool((pool[:, 0] == 5).all()) and bool((pool[:, -1] == 5).all())
