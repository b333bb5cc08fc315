"""The books of a cache kept one entry at a time (plain Python), and small caches to keep."""
from __future__ import annotations

import torch

OK, INDEX, PAGES = 0, -12, -13


class Books:
    """refs, lengths, table as lists; codes and scales as CPU tensors: the calls' definitions.
    Every call returns the statuses that it may report."""

    def __init__(self, refs, lengths, table, page_tokens, pools=()):
        self.refs, self.lengths = refs.tolist(), lengths.tolist()
        self.table, self.P = table.tolist(), page_tokens
        self.pools = [t.cpu().clone() for t in pools]  # [pages, ...]; codes [pages, heads, P, D]

    def blocks(self, t):
        return -(-t // self.P)

    def free_pages(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def _fits(self, t):
        return 0 <= t <= len(self.table[0]) * self.P

    def extend(self, sequences, more):
        free, taken, seen, bad = self.free_pages(), 0, set(), set()
        for s, m in zip(sequences, more):
            if not 0 <= s < len(self.lengths) or s in seen:
                bad.add(INDEX)
                continue
            seen.add(s)
            have = self.lengths[s]
            if m < 0 or not self._fits(have) or not self._fits(have + m):
                bad.add(INDEX)
                continue
            want = self.blocks(have + m) - self.blocks(have)
            if want and taken + want > len(free):
                bad.add(PAGES)
                taken += want
                continue
            for i in range(want):
                page = free[taken + i]
                self.table[s][self.blocks(have) + i] = page
                self.refs[page] = 1
            taken += want
            self.lengths[s] = have + m
        return bad

    def fork(self, parents, children, tokens=None):
        free, taken, seen, bad = self.free_pages(), 0, set(), set()
        before = list(self.lengths)
        for i, (p, c) in enumerate(zip(parents, children)):
            if not 0 <= c < len(before) or c in seen:
                bad.add(INDEX)
                continue
            seen.add(c)
            if not 0 <= p < len(before) or p == c:
                bad.add(INDEX)
                continue
            t = before[p] if tokens is None else tokens[i]
            if not self._fits(before[p]) or not 0 <= t <= before[p] or before[c] != 0:
                bad.add(INDEX)
                continue
            whole, part = divmod(t, self.P)
            if part:
                taken += 1
                if taken > len(free):
                    bad.add(PAGES)
                    continue
            for b in range(whole):
                page = self.table[p][b]
                self.table[c][b] = page
                if 0 <= page < len(self.refs):
                    self.refs[page] += 1
                else:
                    bad.add(INDEX)
            if part:
                to, source = free[taken - 1], self.table[p][whole]
                self.table[c][whole] = to
                self.refs[to] = 1
                if not 0 <= source < len(self.refs):
                    bad.add(INDEX)
                else:
                    for x in self.pools:
                        if x.dim() == 4:
                            x[to, :, :part] = x[source, :, :part]
                        else:
                            x[to] = x[source]
            self.lengths[c] = t
        return bad

    def free(self, sequences):
        bad = set()
        for s in sequences:
            if not 0 <= s < len(self.lengths) or not self._fits(self.lengths[s]):
                bad.add(INDEX)
                continue
            for b in range(self.blocks(self.lengths[s])):
                page = self.table[s][b]
                if 0 <= page < len(self.refs) and self.refs[page] > 0:
                    self.refs[page] -= 1
                else:
                    bad.add(INDEX)
            self.lengths[s] = 0
        return bad

    def compact(self):
        n = sum(r != 0 for r in self.refs)
        holes = iter([i for i in range(n) if self.refs[i] == 0])
        moves = [-1 if r == 0 else i if i < n else next(holes) for i, r in enumerate(self.refs)]
        for i in range(n, len(self.refs)):
            if moves[i] >= 0:
                for x in self.pools:
                    x[moves[i]] = x[i]
                self.refs[moves[i]], self.refs[i] = self.refs[i], 0
        for s, t in enumerate(self.lengths):
            if self._fits(t):
                for b in range(self.blocks(t)):
                    page = self.table[s][b]
                    if 0 <= page < len(moves) and moves[page] >= 0:
                        self.table[s][b] = moves[page]
        return moves, n

    def check(self, pages, pools=()):
        """Raises where the device's books or pools differ."""
        assert pages.refs.tolist() == self.refs
        assert pages.lengths.tolist() == self.lengths
        assert pages.table.tolist() == self.table
        for got, want in zip(pools, self.pools):
            assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))
