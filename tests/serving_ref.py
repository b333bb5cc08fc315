"""References of the rotary, cache and cache-attention calls in 64 bits (torch on the CPU),
and small batches to run them on."""
from __future__ import annotations

import math

import torch

FLOOR = 2.0 ** -100


# ------------------------------------------------------------------------------ rotary --

def frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_length=0.0, slow=1.0,
                fast=32.0):
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = []
    for i in range(rot_dim // 2):
        w = base ** (-2.0 * i / rot_dim)
        if scaling == "linear":
            w /= factor
        if scaling == "by_parts":
            r = original_length * w / (2 * math.pi)
            g = min(1.0, max(0.0, (r - slow) / (fast - slow)))
            w = w * (g + (1 - g) / factor)
        f.append(w)
    return torch.tensor(f, dtype=torch.float64)


def rotary(x, positions, f, interleaved=False, backward=False, amplitude=1.0):
    """x [tokens, heads, size] of any type, in 64 bits; (result, |x0| + |x1| of each pair)."""
    y = x.double().clone()
    rd = 2 * len(f)
    angle = positions.double()[:, None] * f * (-1 if backward else 1)
    c, s = amplitude * torch.cos(angle)[:, None], amplitude * torch.sin(angle)[:, None]
    i0, i1 = ((slice(0, rd, 2), slice(1, rd, 2)) if interleaved
              else (slice(0, rd // 2), slice(rd // 2, rd)))
    a, b = y[..., i0].clone(), y[..., i1].clone()
    size = torch.zeros_like(y)
    size[..., i0] = size[..., i1] = abs(amplitude) * (a.abs() + b.abs())
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    return y, size


# ------------------------------------------------------------------------------- cache --

def scale_of(m: float, fmt: str) -> float:
    """The scale of a block whose largest magnitude is m, by search from the definition."""
    if m == 0.0:
        return FLOOR
    if fmt == "e4m3":
        e = math.frexp(m / 448)[1] - 2
        while 448 * 2.0 ** e < m:
            e += 1
        return max(2.0 ** e, FLOOR)
    want = m / 127
    unit = 2.0 ** (math.frexp(want)[1] - 8)
    n = math.floor(want / unit) - 1
    while 127 * n * unit < m:
        n += 1
    return max(n * unit, FLOOR)


def code_values(y, fmt):
    """y (in units of the scale, 64 bits) rounded to the codes' values."""
    y = torch.nan_to_num(y, nan=0.0, posinf=1e300, neginf=-1e300)
    if fmt == "int8":
        return y.round().clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6, max=448))) - 3)
    return ((y.clamp(-1e30, 1e30) / step).round() * step).clamp(-448, 448)


def write(codes, scale, x, offsets, lengths, table, fmt):
    """kv_cache_write on 64-bit copies of one pool's code values and scales, in place."""
    P = codes.shape[2]
    for s in range(len(lengths)):
        n, L = offsets[s + 1] - offsets[s], lengths[s]
        first = L - n
        for b in range(max(first, 0) // P, -(-L // P)):
            lo, hi = max(first, b * P, 0), min(L, b * P + P)
            if lo >= hi:
                continue
            page = table[s][b]
            for h in range(codes.shape[1]):
                rows = x[offsets[s] + lo - first: offsets[s] + hi - first, h].double()
                fin = rows[torch.isfinite(rows)].abs()
                sc = scale_of(float(fin.max()) if fin.numel() else 0.0, fmt)
                old = lo - b * P
                if old > 0:
                    was = float(scale[page, h])
                    sc = max(sc, was)
                    if sc > was:
                        codes[page, h, :old] = code_values(codes[page, h, :old] * was / sc, fmt)
                codes[page, h, old: hi - b * P] = code_values(rows / sc, fmt)
                scale[page, h] = sc


# --------------------------------------------------------------------------- attention --

def visible(p, length, window, sinks):
    """Mask over keys 0 .. length - 1 of a row at position p."""
    t = torch.arange(length)
    see = t <= p
    if window:
        see &= (p - t < window) | (t < sinks)
    return see


def attention(q, kc, ks, vc, vs, offsets, lengths, table, window=0, sinks=0, scale=None,
              hidden=None):
    """Per row and head, in 64 bits: (out, bound on its error before the last rounding).
    ``hidden``: {sequence: mask of keys that no row of it sees}.

    The bound follows the kernel's arithmetic. A score of products |q||k| summing to A is
    off by at most (D + 8) 2^-24 A; the exponent's other roundings (arguments below 64 in
    the base-2 domain: 3 of 64 * 2^-24) and the approximate exponentials add 2^-16
    relatively; a weight so off by a factor 1 + d moves the quotient by at most
    2 d sum p|v|. Weights rounded to fp16 are off by 2^-11 relatively, or 2^-25 of the
    largest where subnormal, which over N keys is N 2^-25 max|v|. Sums of N terms in fp32:
    N 2^-24 relatively."""
    rows, Hq, D = q.shape
    Hkv, P = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros((rows, Hq, D), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for s in range(len(lengths)):
        n, L = offsets[s + 1] - offsets[s], lengths[s]
        if n == 0 or L == 0:
            continue
        pages = [table[s][b] for b in range(-(-L // P))]
        k = (kc[pages] * ks[pages][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :L]
        v = (vc[pages] * vs[pages][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :L]
        for j in range(n):
            p = L - n + j
            if p < 0:
                continue
            see = visible(p, L, window, sinks)
            if hidden and s in hidden:
                see &= ~hidden[s]
            for h in range(Hq):
                x = q[offsets[s] + j, h].double()
                kk, vv = k[h // G][see], v[h // G][see]
                w = torch.softmax(kk @ x * scale, 0)
                A = float((kk.abs() @ x.abs()).max() * abs(scale))
                d = (D + 8) * 2.0 ** -24 * A + 2.0 ** -16 + len(w) * 2.0 ** -24
                out[offsets[s] + j, h] = w @ vv
                bound[offsets[s] + j, h] = ((2 * d + 2.0 ** -11) * (w @ vv.abs())
                                            + len(w) * 2.0 ** -25 * vv.abs().max())
    return out, bound


class Batch:
    """A ragged batch over a shuffled paged cache, on the host and as device tensors.

    new, old: tokens of each sequence in this call and before it. Unused table entries and
    all slots that hold no token have contents that must not matter."""

    def __init__(self, new, old, Hkv, D, P, fmt, seed=0, spare=2, extra_rows=0, width_extra=1):
        g = torch.Generator().manual_seed(seed)
        self.new, self.old, self.fmt, self.P, self.Hkv, self.D = new, old, fmt, P, Hkv, D
        self.lengths = [a + b for a, b in zip(new, old)]
        self.offsets = [sum(new[:i]) for i in range(len(new) + 1)]
        self.rows = self.offsets[-1] + extra_rows
        used = [-(-L // P) for L in self.lengths]
        self.pages = sum(used) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(1, max(used)) + width_extra
        self.table, at = [], 0
        for u in used:
            self.table.append(order[at: at + u] + [-7] * (width - u))
            at += u
        self.g = g
        shape = (self.pages, Hkv, P, D)
        self.codes, self.scale = {}, {}
        for name in ("k", "v"):
            x = torch.randn(shape, generator=g)
            c = (x * 32).round().clamp(-127, 127).to(torch.int8) if fmt == "int8" else \
                (x * 96).clamp(-448, 448).to(torch.float8_e4m3fn)
            live = torch.zeros((self.pages, P), dtype=torch.bool)
            for s, L in enumerate(self.lengths):
                for b in range(used[s]):
                    live[self.table[s][b], : max(0, min(P, L - b * P))] = True
            self.live = live
            junk = -128 if fmt == "int8" else 0x7F  # e4m3's NaN
            raw = c.view(torch.uint8)
            raw.masked_fill_(~live[:, None, :, None].expand(shape), junk & 0xFF)
            self.codes[name] = c
            sc = torch.exp2(torch.randn(shape[:2], generator=g) * 1.5 - 5)
            sc = sc.to(torch.bfloat16).float() if fmt == "int8" else torch.exp2(sc.log2().round())
            sc[~live.any(1)] = float("nan")  # pages that hold nothing
            self.scale[name] = sc

    def values(self, name):
        """64-bit code values (0 in slots that hold no token) and scales."""
        c = self.codes[name].float().double()
        return (torch.where(self.live[:, None, :, None], c, 0.0),
                self.scale[name].double())

    def rows_of(self, heads, dtype, scale=1.0, seed=1):
        g = torch.Generator().manual_seed(seed)
        return (torch.randn((self.rows, heads, self.D), generator=g) * scale).to(dtype)

    def ints(self, device="cuda"):
        return tuple(torch.tensor(x, dtype=torch.int32, device=device)
                     for x in (self.offsets, self.lengths, self.table))

    def device(self, csa):
        """(KvCache, KvBatch) on the GPU."""
        cache = csa.KvCache(*(t.cuda() for t in (self.codes["k"], self.codes["v"],
                                                  self.scale["k"], self.scale["v"])))
        return cache, csa.KvBatch(*self.ints(), rows=self.rows, max_new=max(1, max(self.new)))


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2
