"""Batches whose sequences share long beginnings, on the host and as device tensors."""
from __future__ import annotations

import torch

import serving_ref as ref


class SharedBatch(ref.Batch):
    """groups: [(first sequence, end, shared tokens)] next to each other, in order. ``old`` are a
    sequence's tokens of its own before this call. On the host every member's table row begins with
    the pages of its group's first one; on the device the others' entries for them name no page."""

    def __init__(self, new, old, groups, Hkv, D, P, fmt, seed=0, **more):
        shared = [0] * len(new)
        for a, z, t in groups:
            for s in range(a, z):
                shared[s] = t
        super().__init__(new, [x + t for x, t in zip(old, shared)], Hkv, D, P, fmt, seed, **more)
        self.device_table = [list(r) for r in self.table]
        for a, z, t in groups:
            for s in range(a + 1, z):
                self.table[s][: t // P] = self.table[a][: t // P]
                self.device_table[s][: t // P] = [-9] * (t // P)
        self.bounds = [a for a, _, _ in groups] + [groups[-1][1]]
        self.shared = [t for _, _, t in groups]

    def ints(self, device="cuda"):
        return tuple(torch.tensor(x, dtype=torch.int32, device=device)
                     for x in (self.offsets, self.lengths, self.device_table))

    def lists(self):
        return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (self.bounds, self.shared))

    def device_whole(self, csa):
        """(KvCache, KvBatch) with every table row written out."""
        cache, batch = self.device(csa)
        table = torch.tensor(self.table, dtype=torch.int32, device="cuda")
        return cache, csa.KvBatch(batch.offsets, batch.lengths, table, rows=self.rows, max_new=max(1, max(self.new)))


def room(b, q, scale=None, dtype=torch.bfloat16):
    """(definition in 64 bits, room for the result): the bound of serving_ref.attention, whose
    2^-16 covers the joining's two exponentials and products (3 of 2^-22 relatively), and one
    rounding to the type."""
    want, bound = ref.attention(q, *b.values("k"), *b.values("v"), b.offsets, b.lengths, b.table, scale=scale)
    return want, (bound * (1 + ref.half_step(dtype)) + want.abs() * ref.half_step(dtype)
                  + (2.0 ** -25 if dtype == torch.float16 else 0.0))
