"""Answers sampled from prompts, as a server does it: room for prompts, their keys and values
written, prompts forked into answers, tokens appended, attention that reads the shared part once,
logits from a dense layer, their tokens' log probabilities and gradients, answers that end, the
cache compacted, and the next step over it (GPU)."""
import math

import pytest
import torch

import causal_attention_score_gb300 as csa
import logprobs_ref
import serving_ref as ref
from pages_ref import Books

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


class Server:
    Hq, Hkv, D, P, VOCAB = 8, 2, 64, 32, 1111

    def __init__(self, fmt, sequences=14, width=24, pages=200):
        dt = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
        self.cache = csa.KvCache.empty(pages, self.Hkv, self.P, self.D, dt)
        self.pages = csa.KvPages.empty(self.cache, sequences, width)
        self.books = Books(self.pages.refs, self.pages.lengths, self.pages.table, self.P)
        self.rotary = csa.RotaryTable(self.D)
        self.g = torch.Generator().manual_seed(7)
        self.S = sequences
        self.W = (torch.randn((self.VOCAB, self.Hq * self.D), generator=self.g) * 0.1).to(torch.bfloat16).cuda()

    def step(self, new, groups=None):
        """new[s] more tokens of each sequence: K and V written, attention over them. (out, rows' q)"""
        at = [s for s in range(self.S) if new[s]]
        csa.kv_pages_extend(self.pages, ints(at), ints(new[s] for s in at))
        assert self.books.extend(at, [new[s] for s in at]) == set()
        rows = sum(new)
        x = torch.randn((rows, self.Hq + 2 * self.Hkv, self.D), generator=self.g).to(torch.bfloat16).cuda()
        first = [self.books.lengths[s] - new[s] for s in range(self.S)]
        positions = ints(p for s in range(self.S) for p in range(first[s], first[s] + new[s]))
        qk = x[:, : self.Hq + self.Hkv]
        csa.rotary_forward(qk, qk, self.rotary, positions)
        self.offsets = [sum(new[:s]) for s in range(self.S + 1)]
        batch = csa.KvBatch(ints(self.offsets), self.pages.lengths, self.pages.table, rows=rows, max_new=max(new))
        csa.kv_cache_write(self.cache, batch, x[:, self.Hq: self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:])
        q = x[:, : self.Hq]
        if groups:
            out = csa.cache_attention_shared(q, self.cache, batch, *(ints(v) for v in groups))
        else:
            out = csa.cache_attention(q, self.cache, batch)
        assert csa.get_status() == 0
        self.books.check(self.pages)
        self.batch = batch
        return out, q

    def expected(self, q):
        """Attention in 64 bits over what the cache holds."""
        held = []
        for t, s in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            # (slots that nothing was written to may hold anything)
            held += [torch.nan_to_num(t.cpu().float()).double(), torch.nan_to_num(s.cpu().double(), 0, 0, 0)]
        return ref.attention(q.cpu(), *held, self.offsets, self.books.lengths, self.books.table)

    def close(self, out, q, what):
        want, bound = self.expected(q)
        err = (out.cpu().double() - want).abs()
        assert bool((err <= bound * 1.01 + want.abs() * 2.0 ** -8).all()), what


@pytest.mark.parametrize("mode", [csa.SHARED_ALWAYS, csa.SHARED_AUTO])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_answers(fmt, mode):
    csa.set_shared_part(mode)
    try:
        _answers(Server(fmt))
    finally:
        csa.set_shared_part(csa.SHARED_AUTO)


def _answers(s):
    # two prompts, at places 0 and 5
    new = [0] * s.S
    new[0], new[5] = 200, 75
    out, q = s.step(new)
    s.close(out, q, "prompts")
    # four answers to the first, eight to the second; both prompts stay as the groups' first ones
    parents, children = [0] * 4 + [5] * 8, [1, 2, 3, 4] + [6, 7, 8, 9, 10, 11, 12, 13]
    csa.kv_cache_fork(s.cache, s.pages, ints(parents), ints(children))
    assert s.books.fork(parents, children) == set()
    s.books.check(s.pages)
    assert max(s.books.refs) == 9
    shared = [s.books.lengths[0] // s.P * s.P, s.books.lengths[5] // s.P * s.P]
    groups = ([0, 5, s.S], shared)
    for token in range(3):
        new = [0 if i in (0, 5) else 1 for i in range(s.S)]
        out, q = s.step(new, groups)
        s.close(out, q, f"token {token}")
    # the same rows, each sequence reading its prompt for itself
    whole = csa.cache_attention(q, s.cache, s.batch)
    s.close(whole, q, "unshared")
    # the answers' tokens scored
    rows = out.shape[0]
    tokens = torch.randint(0, s.VOCAB, (rows,), generator=s.g, dtype=torch.int32)
    logits = csa.dense(out.reshape(rows, -1), s.W)
    logprob, entropy, stats, top_logprob, top_token = csa.token_logprobs(logits, tokens.cuda(), 5, 1 / 0.7)
    want, bound = logprobs_ref.forward(logits.cpu(), tokens, 1 / 0.7, 5)
    assert torch.equal(top_token.cpu().long(), want["top_token"])
    for got, name in ((logprob, "logprob"), (entropy, "entropy"), (top_logprob, "top_logprob")):
        assert bool(((got.cpu().double() - want[name]).abs() <= bound[name] + want[name].abs() * 2.0 ** -24).all()), name
    # and the gradient of an advantage's weight on each, through the dense layer
    weight = torch.linspace(-1, 1, rows)
    dlogits = torch.empty_like(logits)
    csa.token_logprobs_backward(dlogits, logits, tokens.cuda(), stats, entropy, weight.cuda(),
                                torch.full((rows,), 0.01, device="cuda"), scale=1 / 0.7)
    wd, bd = logprobs_ref.backward(logits.cpu(), tokens, 1 / 0.7, weight, torch.full((rows,), 0.01))
    assert bool(((dlogits.cpu().double() - wd).abs() <= bd + wd.abs() * 2.0 ** -24).all())
    # answers end, the cache is compacted, what is left answers on
    csa.kv_pages_free(s.pages, ints([2, 3, 7, 8, 9]))
    s.books.free([2, 3, 7, 8, 9])
    moves, used = ints([0] * 200), ints([0])
    csa.kv_cache_compact(s.cache, s.pages, moves, used)
    m, n = s.books.compact()
    assert moves.tolist() == m and used.item() == n
    s.books.check(s.pages)
    new = [0 if i in (0, 5, 2, 3, 7, 8, 9) else 1 for i in range(s.S)]
    out, q = s.step(new, groups)
    s.close(out, q, "after compacting")
    # the prompts end last: their shared pages stay with the answers
    csa.kv_pages_free(s.pages, ints([0, 5]))
    s.books.free([0, 5])
    new = [0 if i in (0, 5, 2, 3, 7, 8, 9) else 1 for i in range(s.S)]
    out, q = s.step(new, ([1, 5, s.S], [0, 0]))
    s.close(out, q, "after the prompts")
    left = [i for i in range(s.S) if s.books.lengths[i]]
    csa.kv_pages_free(s.pages, ints(left))
    s.books.free(left)
    assert not any(s.books.refs)
    s.books.check(s.pages)
