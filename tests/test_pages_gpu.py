"""kv_pages_extend, kv_cache_fork, kv_pages_free, kv_cache_copy and kv_cache_compact against
books kept one entry at a time (GPU). Everything is whole numbers: equal, or wrong."""
import random

import pytest
import torch

import causal_attention_score_gb300 as csa
from pages_ref import INDEX, PAGES, Books

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def made(pages, heads, P, D, sequences, width, dtype=torch.int8, seed=0):
    """A cache of random bytes with empty books, and the books kept beside it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = csa.KvCache.empty(pages, heads, P, D, dtype)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda").to(torch.uint8))
    for t in (cache.k_scale, cache.v_scale):
        t.copy_(torch.rand(t.shape, generator=g, device="cuda"))
    books = csa.KvPages.empty(cache, sequences, width)
    pools = (cache.k, cache.v, cache.k_scale, cache.v_scale)
    return cache, books, pools, Books(books.refs, books.lengths, books.table, P, pools)


@pytest.mark.parametrize("pages,heads,P,D,sequences,width,dtype", [
    (40, 1, 16, 16, 12, 6, torch.int8),
    (300, 3, 32, 48, 40, 20, torch.float8_e4m3fn),
    (1500, 2, 64, 128, 150, 24, torch.int8),      # two chunks of the free pages' list
    (90, 5, 128, 112, 20, 7, torch.float8_e4m3fn),
])
def test_any_order_of_calls(pages, heads, P, D, sequences, width, dtype):
    cache, books, pools, want = made(pages, heads, P, D, sequences, width, dtype)
    rng = random.Random(pages)
    for turn in range(40):
        empty = [s for s in range(sequences) if want.lengths[s] == 0]
        live = [s for s in range(sequences) if want.lengths[s] > 0]
        what = rng.choice(("extend", "extend", "fork", "fork", "free", "compact"))
        if what == "extend":
            at = rng.sample(range(sequences), rng.randint(1, sequences))
            more = [min(rng.choice((0, 1, 1, 5, P, 3 * P + 2)), width * P - want.lengths[s]) for s in at]
            status = want.extend(at, more)
            csa.kv_pages_extend(books, ints(at), ints(more))
        elif what == "fork" and empty and live:
            children = rng.sample(empty, rng.randint(1, len(empty)))
            parents = [rng.choice(live) for _ in children]
            tokens = None
            if rng.random() < 0.5:
                tokens = [rng.choice((0, want.lengths[p] // P * P, rng.randint(0, want.lengths[p]))) for p in parents]
            status = want.fork(parents, children, tokens)
            csa.kv_cache_fork(cache, books, ints(parents), ints(children), None if tokens is None else ints(tokens))
        elif what == "free" and live:
            at = rng.sample(live, rng.randint(1, max(1, len(live) // 2)))
            status = want.free(at)
            csa.kv_pages_free(books, ints(at))
        else:
            moves, n = want.compact()
            got, used, status = ints([7] * pages), ints([-5]), set()
            csa.kv_cache_compact(cache, books, got, used)
            assert got.tolist() == moves and used.item() == n
        assert csa.get_status() in (status or {0}), (turn, what)
        want.check(books, pools)
        # shared pages are whole: a page of several sequences is never a last one written in part
        assert all(r >= 0 for r in want.refs)


def test_refused_entries():
    """Places that are none, named twice, of wrong lengths or without pages are left as they were."""
    cache, books, pools, want = made(6, 2, 16, 32, 6, 4)

    def both(name, *lists, status):
        expected = getattr(want, name)(*lists)
        assert expected == status
        args = [None if v is None else ints(v) for v in lists]
        {"extend": lambda: csa.kv_pages_extend(books, *args), "free": lambda: csa.kv_pages_free(books, *args),
         "fork": lambda: csa.kv_cache_fork(cache, books, *args)}[name]()
        assert csa.get_status() in (status or {0})
        want.check(books, pools)

    both("extend", [0, 1], [20, 3], status=set())
    both("extend", [-1, 6, 2 ** 31 - 1, 1], [1, 1, 1, 1], status={INDEX})
    both("extend", [1, 1, 0], [1, 40, -1], status={INDEX})
    both("extend", [1], [64], status={INDEX})              # past the table's width
    both("extend", [1], [2 ** 31 - 1], status={INDEX})
    both("extend", [2, 3], [60, 1], status={PAGES})        # 3 pages are free, 4 and then 1 wanted
    both("extend", [2, 3], [16, 0], status=set())
    both("fork", [0, 0], [4, 4], None, status={INDEX})     # the same place twice
    both("fork", [0, 9, -1, 4], [5, 3, 3, 3], None, status={INDEX})
    both("fork", [1], [1], None, status={INDEX})
    both("fork", [0], [2], None, status={INDEX})           # a place with a sequence
    both("fork", [1], [3], [99], status={INDEX})
    both("fork", [1], [3], [-1], status={INDEX})
    both("free", [4, 4, 17, -3], status={INDEX})
    both("free", [3], status=set())                        # nothing there
    both("fork", [3], [4], None, status=set())             # of nothing
    both("extend", [3], [16], status=set())                # the last page
    both("fork", [1, 2], [4, 3], None, status={PAGES, INDEX})
    books.lengths[5] = -7
    want.lengths[5] = -7
    both("free", [5], status={INDEX})
    both("extend", [5], [1], status={INDEX})
    books.lengths[5] = 65
    want.lengths[5] = 65
    both("free", [5], status={INDEX})
    both("fork", [5], [4], [1], status={INDEX})


def test_pages_out_of_range():
    """Table entries that name no page are skipped and reported."""
    cache, books, pools, want = made(8, 1, 16, 16, 3, 4)
    csa.kv_pages_extend(books, ints([0]), ints([40]))
    want.extend([0], [40])
    for page in (-1, 8, 2 ** 31 - 1):
        for block in (0, 2):
            books.table[0, block] = page
            keep, want.table[0][block] = want.table[0][block], page
            csa.kv_cache_fork(cache, books, ints([0]), ints([1]))
            assert want.fork([0], [1]) == {INDEX} and csa.get_status() == csa.CSA_ERR_INDEX
            want.check(books, pools)
            csa.kv_pages_free(books, ints([1]))
            status = want.free([1])
            assert csa.get_status() in (status or {0})
            want.check(books, pools)
            books.table[0, block] = keep
            want.table[0][block] = keep
    books.table[0, 1] = 9
    want.table[0][1] = 9
    moves, n = want.compact()
    got, used = ints([0] * 8), ints([0])
    csa.kv_cache_compact(cache, books, got, used)
    assert csa.get_status() == csa.CSA_ERR_INDEX and got.tolist() == moves and used.item() == n
    want.check(books, pools)
    # a page counted fewer times than it is named: reported, never below 0
    books.table[0, 1] = 0
    books.refs.zero_()
    csa.kv_pages_free(books, ints([0]))
    assert csa.get_status() == csa.CSA_ERR_INDEX and books.refs.tolist() == [0] * 8


def test_copy_between_caches():
    a, _, pa, _ = made(20, 3, 32, 80, 1, 1, torch.float8_e4m3fn, seed=1)
    b, _, pb, _ = made(9, 3, 32, 80, 1, 1, torch.float8_e4m3fn, seed=2)
    before = [t.clone() for t in pb]
    to, frm = [8, 0, 3, 5], [19, 0, 7, 7]
    csa.kv_cache_copy(b, a, ints(to), ints(frm))
    assert csa.get_status() == 0
    for got, was, source in zip(pb, before, pa):
        for t, f in zip(to, frm):
            was.view(torch.uint8)[t] = source.view(torch.uint8)[f]
        assert torch.equal(got.view(torch.uint8), was.view(torch.uint8))
    csa.kv_cache_copy(b, a, ints([1, 9, -1, 2]), ints([20, 3, 4, -1]))  # none of them a pair of pages
    assert csa.get_status() == csa.CSA_ERR_INDEX
    for got, was in zip(pb, before):
        assert torch.equal(got.view(torch.uint8), was.view(torch.uint8))
    csa.kv_cache_copy(a, a, ints([1, 2]), ints([5, 5]))                 # within one cache
    assert csa.get_status() == 0
    for t in pa:
        assert torch.equal(t.view(torch.uint8)[1], t.view(torch.uint8)[5])
        assert torch.equal(t.view(torch.uint8)[2], t.view(torch.uint8)[5])


def test_large_pages_are_copied_whole():
    """More than one job a page, the last of them short."""
    cache, books, pools, want = made(24, 40, 128, 80, 8, 3)
    csa.kv_pages_extend(books, ints(range(8)), ints([300] * 8))
    want.extend(range(8), [300] * 8)
    csa.kv_pages_free(books, ints([0, 2, 5]))
    want.free([0, 2, 5])
    csa.kv_cache_fork(cache, books, ints([1, 7]), ints([0, 2]))
    want.fork([1, 7], [0, 2])
    want.check(books, pools)
    csa.kv_pages_free(books, ints([1]))
    want.free([1])
    got, used = ints([0] * 24), ints([0])
    csa.kv_cache_compact(cache, books, got, used)
    moves, n = want.compact()
    assert csa.get_status() == 0 and got.tolist() == moves and used.item() == n
    want.check(books, pools)


def test_pages_past_2_to_the_32():
    """Pages whose codes begin more than 2^32 bytes into the cache."""
    cache = csa.KvCache.empty(34000, 8, 128, 128)  # 131072 bytes a page, 4.5 GB each of K and V
    for t in (cache.k, cache.v):
        t[0], t[33999], t[33000] = 1, 3, 4
    cache.k_scale.fill_(0.5)
    refs = torch.zeros((34000,), dtype=torch.int32, device="cuda")
    refs[33000] = refs[33999] = 1
    table = torch.tensor([[33000, 33999], [0, 0], [0, 0]], dtype=torch.int32, device="cuda")
    books = csa.KvPages(refs, ints([200, 0, 0]), table, 128)
    refs[:33990] += 1
    refs[33000] -= 1
    csa.kv_cache_fork(cache, books, ints([0]), ints([1]))  # its last page: 33990
    assert csa.get_status() == 0 and books.table[1].tolist() == [33000, 33990]
    assert bool((cache.k[33990, :, :72] == 3).all()) and bool((cache.v[33990, :, :72] == 3).all())
    csa.kv_cache_copy(cache, cache, ints([33998]), ints([33000]))
    assert bool((cache.k[33998] == 4).all()) and bool((cache.v[33998] == 4).all())
    refs[:100] = 0
    moves, used = ints([0] * 34000), ints([0])
    csa.kv_cache_compact(cache, books, moves, used)
    assert csa.get_status() == 0 and used.item() == 33892
    end = moves[33999].item()
    assert end == 99 and bool((cache.k[end] == 3).all()) and books.table[0].tolist() == [33000, 99]
    assert bool((cache.v[books.table[1, 1].item(), :, :72] == 3).all())


@pytest.mark.parametrize("pages", [1, 31, 33, 1024, 1025, 1024 * 1024 + 3, 2500000])
def test_number_of_pages(pages):
    """Free pages are found at any number of pages, wherever they are."""
    cache = csa.KvCache.empty(pages, 1, 16, 16)
    g = torch.Generator().manual_seed(pages)
    taken = torch.rand((pages,), generator=g) < 0.9
    taken[-1] = False
    refs = torch.where(taken, 2, 0).to(torch.int32)
    free = torch.nonzero(refs == 0)[:, 0].tolist()
    want = min(len(free), 3000)
    books = csa.KvPages(refs.cuda(), ints([0, 0, 0]), torch.full((3, 3000), -1, dtype=torch.int32, device="cuda"), 16)
    first = want // 2
    csa.kv_pages_extend(books, ints([2, 0]), ints([first * 16, (want - first) * 16]))
    assert csa.get_status() == 0
    assert books.table[2, :first].tolist() == free[:first]
    assert books.table[0, :want - first].tolist() == free[first:want]
    assert books.lengths.tolist() == [(want - first) * 16, 0, first * 16]
    refs[free[:want]] = 1
    assert torch.equal(books.refs.cpu(), refs)
    moves, used = torch.empty((pages,), dtype=torch.int32, device="cuda"), ints([0])
    csa.kv_cache_compact(cache, books, moves, used)
    assert csa.get_status() == 0
    live = torch.nonzero(refs > 0)[:, 0]
    n = live.numel()
    expect = torch.full((pages,), -1, dtype=torch.int32)
    expect[live] = live.to(torch.int32)
    expect[live[live >= n]] = torch.nonzero(refs[:n] == 0)[:, 0].to(torch.int32)
    assert used.item() == n and torch.equal(moves.cpu(), expect)
    assert torch.equal(books.refs.cpu() > 0, torch.arange(pages) < n)
    assert books.table[2, :first].tolist() == expect[free[:first]].tolist()


@pytest.mark.parametrize("pages,n", [(3000, 513), (40000, 700), (40000, 3), (33000, 1500)])
def test_many_entries(pages, n):
    """Entries in several rounds of the planning CTA, pages in many chunks."""
    cache = csa.KvCache.empty(pages, 1, 16, 16)
    books = csa.KvPages.empty(cache, n + 5, 8)
    want = Books(books.refs, books.lengths, books.table, 16)
    rng = random.Random(n)
    for _ in range(3):
        at = rng.sample(range(n + 5), n)
        more = [rng.choice((0, 1, 16, 30)) for _ in at]
        status = want.extend(at, more)
        csa.kv_pages_extend(books, ints(at), ints(more))
        assert csa.get_status() in (status or {0})
        want.check(books)
        gone = rng.sample(range(n + 5), n // 3)
        csa.kv_pages_free(books, ints(gone))
        want.free(gone)
    moves, used = ints([0] * pages), ints([0])
    csa.kv_cache_compact(cache, books, moves, used)
    m, u = want.compact()
    assert csa.get_status() == 0 and moves.tolist() == m and used.item() == u
    want.check(books)


def test_length_past_31_bits():
    """A table with room for more tokens than a length can say: the entry is left out."""
    width = 2 ** 24 + 2
    refs, table = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.zeros((2, width), dtype=torch.int32, device="cuda")
    lengths = ints([2 ** 31 - 100, 0])
    books = csa.KvPages(refs, lengths, table, 128)
    csa.kv_pages_extend(books, ints([0, 1]), ints([200, 130]))
    assert csa.get_status() == INDEX
    assert lengths.tolist() == [2 ** 31 - 100, 130] and refs.tolist() == [1, 1] + [0] * 6
    csa.kv_pages_extend(books, ints([0]), ints([99]))
    assert csa.get_status() == 0 and lengths.tolist() == [2 ** 31 - 1, 130]
    assert not table[0].any() and table[1, :3].tolist() == [0, 1, 0]


def test_captured_and_on_other_streams():
    """A turn (end, fork, extend, compact) captured once and replayed from other books; two caches on
    two streams with workspaces of their own."""
    cache, books, pools, _ = made(200, 2, 16, 32, 30, 10, seed=3)
    csa.kv_pages_extend(books, ints(range(10)), ints(range(20, 120, 10)))
    ws = torch.empty(csa.kv_pages_workspace_size(books, 30), dtype=torch.uint8, device="cuda")
    ended, parents, children = ints([1, 3]), ints([0, 0, 2, 4]), ints([11, 12, 13, 14])
    grow, more = ints([0, 11, 12, 5]), ints([1, 1, 1, 17])
    moves, used = ints([0] * 200), ints([0])
    saved = [t.clone() for t in (books.refs, books.lengths, books.table, *pools)]

    def turn(c, b, m, u, w, stream=None):
        csa.kv_pages_free(b, ended, stream=stream)
        csa.kv_cache_fork(c, b, parents, children, workspace=w, stream=stream)
        csa.kv_pages_extend(b, grow, more, workspace=w, stream=stream)
        csa.kv_cache_compact(c, b, m, u, workspace=w, stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn(cache, books, moves, used, ws)
    for t, s in zip((books.refs, books.lengths, books.table, *pools), saved):
        t.view(torch.uint8).copy_(s.view(torch.uint8))
    want = Books(books.refs, books.lengths, books.table, 16, pools)
    for _ in range(2):
        ws.random_()  # nothing is kept there from one call to the next
        graph.replay()
        torch.cuda.synchronize()
        want.free([1, 3])
        want.fork(parents.tolist(), children.tolist())
        want.extend(grow.tolist(), more.tolist())
        m, n = want.compact()
        want.check(books, pools)
        assert moves.tolist() == m and used.item() == n
        # the next turn begins with the children gone
        csa.kv_pages_free(books, children)
        want.free(children.tolist())
    csa.get_status()
    two = [made(200, 2, 16, 32, 30, 10, seed=s) for s in (5, 6)]
    streams = [torch.cuda.Stream() for _ in two]
    outs = [(ints([0] * 200), ints([0])) for _ in two]
    torch.cuda.synchronize()
    for (c, b, p, _), st, (m, u) in zip(two, streams, outs):
        csa.kv_pages_extend(b, ints(range(10)), ints(range(20, 120, 10)), stream=st)
        turn(c, b, m, u, None, stream=st)
    torch.cuda.synchronize()
    assert csa.get_status() == 0
    for (c, b, p, w), (m, u) in zip(two, outs):
        w.extend(range(10), range(20, 120, 10))
        w.free([1, 3])
        w.fork(parents.tolist(), children.tolist())
        w.extend(grow.tolist(), more.tolist())
        mv, n = w.compact()
        w.check(b, p)
        assert m.tolist() == mv and u.item() == n
