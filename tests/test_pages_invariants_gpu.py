"""What holds of a cache's books after any call (GPU): a page is counted as often as live table entries
name it, and a last page written in part is its sequence's alone."""
import random

import pytest
import torch

import causal_attention_score_gb300 as csa
from test_pages_gpu import ints, made

pytestmark = pytest.mark.gpu


def check(books, P):
    refs, lengths, table = books.refs.tolist(), books.lengths.tolist(), books.table.tolist()
    named = [0] * len(refs)
    for s, length in enumerate(lengths):
        assert 0 <= length <= len(table[s]) * P
        for b in range(-(-length // P)):
            named[table[s][b]] += 1
    assert named == refs
    for s, length in enumerate(lengths):
        if length % P:
            assert refs[table[s][length // P]] == 1, (s, length)


@pytest.mark.parametrize("pages,P,sequences,width,seed", [(60, 16, 14, 8, 0), (60, 16, 14, 8, 1), (400, 64, 60, 12, 2),
                                                          (2100, 32, 200, 30, 3)])
def test_counts_and_last_pages(pages, P, sequences, width, seed):
    cache, books, _, _ = made(pages, 2, P, 32, sequences, width, seed=seed)
    rng = random.Random(seed)
    forked = 0
    for turn in range(60):
        lengths = books.lengths.tolist()
        empty = [s for s in range(sequences) if lengths[s] == 0]
        live = [s for s in range(sequences) if lengths[s] > 0]
        what = rng.choice(("extend", "extend", "fork", "fork", "free", "compact"))
        if what == "fork" and empty and live:
            children = rng.sample(empty, rng.randint(1, len(empty)))
            parents = [rng.choice(live) for _ in children]
            tokens = [rng.choice((lengths[p], rng.randint(0, lengths[p]))) for p in parents]
            csa.kv_cache_fork(cache, books, ints(parents), ints(children), ints(tokens))
            forked += len(children)
        elif what == "free" and live:
            csa.kv_pages_free(books, ints(rng.sample(live, rng.randint(1, max(1, len(live) // 2)))))
        elif what == "compact":
            csa.kv_cache_compact(cache, books, ints([0] * pages), ints([0]))
        else:
            at = rng.sample(range(sequences), rng.randint(1, sequences))
            more = [min(rng.choice((1, 5, P, 2 * P + 3)), width * P - lengths[s]) for s in at]
            csa.kv_pages_extend(books, ints(at), ints(more))
        assert csa.get_status() in (0, csa.CSA_ERR_PAGES), (turn, what)
        check(books, P)
    assert forked > sequences // 2
