"""Cases and plain forms of the serving operators: rotary positions, a paged cache of 8-bit keys
and values (written and read back), and attention over that cache.

``run`` is one pass of an operator. With ``own`` false it is computed by elementary torch
operations in 32 bits (64 for the angles); with ``own`` true by the library's entry points.
``exact`` gives the same outputs from the definitions in 64 bits.

Layouts: x [tokens, heads, D]; cache codes [pages, heads, P, D] with one fp32 scale for each
page and head; ``offsets`` [S + 1] are each sequence's rows among the new tokens, ``lengths`` [S]
its length including them, ``table`` [S, max_pages] its pages.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
FLOOR = 2.0 ** -100


# ------------------------------------------------------------------------------- cases --

def listed():
    return [
        # Q and K of a GPT-2-small training batch (8 x 1024 tokens, 12 heads of 64)
        {"name": "rotary_train", "op": "rotary", "tokens": 8192, "period": 1024, "heads": 24, "D": 64, "rd": 64,
         "interleaved": False, "dtype": "bf16", "backward": False, "scaling": "none", "far": 0},
        # gradients of the long-context shape (2 x 4096 tokens, 16 heads of 128), half of each
        # head rotated, positions far beyond the trained length
        {"name": "rotary_grad_far", "op": "rotary", "tokens": 8192, "period": 0, "heads": 32, "D": 128, "rd": 64,
         "interleaved": True, "dtype": "fp32", "backward": True, "scaling": "by_parts", "far": 900000},
        # one decoding step of 48 sequences
        {"name": "rotary_step", "op": "rotary", "tokens": 48, "period": 0, "heads": 32, "D": 128, "rd": 128,
         "interleaved": False, "dtype": "fp16", "backward": False, "scaling": "ntk", "far": 30000},
        # ragged prompts quantised into the cache and read back
        {"name": "cache_prompts", "op": "cache", "S": 8, "new_lo": 900, "new_hi": 6000, "old_hi": 200, "Hkv": 16, "D": 128,
         "P": 64, "codes": "int8", "dtype": "bf16", "read": "all"},
        # one token appended to each of 256 sequences, its block read back
        {"name": "cache_step", "op": "cache", "S": 256, "new_lo": 1, "new_hi": 1, "old_hi": 1500, "Hkv": 8, "D": 128,
         "P": 32, "codes": "e4m3", "dtype": "bf16", "read": "blocks"},
        # a few tokens of a few sequences (drafted tokens being checked)
        {"name": "cache_drafts", "op": "cache", "S": 5, "new_lo": 1, "new_hi": 7, "old_hi": 333, "Hkv": 12, "D": 64,
         "P": 16, "codes": "int8", "dtype": "fp16", "read": "blocks"},
        # one token of one sequence: latency
        {"name": "attend_one", "op": "attend", "S": 1, "new_lo": 1, "new_hi": 1, "old_lo": 776, "old_hi": 776, "Hq": 12, "Hkv": 12,
         "D": 64, "P": 64, "codes": "int8", "dtype": "bf16", "window": 0, "sinks": 0},
        # decoding a ragged batch, every head with its own keys
        {"name": "attend_step", "op": "attend", "S": 64, "new_lo": 1, "new_hi": 1, "old_lo": 300, "old_hi": 8191, "Hq": 16, "Hkv": 16,
         "D": 128, "P": 64, "codes": "int8", "dtype": "bf16", "window": 0, "sinks": 0},
        # decoding with grouped heads, a sliding window and a few first tokens kept
        {"name": "attend_window", "op": "attend", "S": 48, "new_lo": 1, "new_hi": 3, "old_lo": 100, "old_hi": 15000, "Hq": 32, "Hkv": 8,
         "D": 128, "P": 32, "codes": "e4m3", "dtype": "fp16", "window": 4096, "sinks": 4},
        # whole prompts of the long-context shape (2 x 4096 tokens, 16 heads of 128)
        {"name": "attend_prompts", "op": "attend", "S": 2, "new_lo": 4096, "new_hi": 4096, "old_lo": 0, "old_hi": 0, "Hq": 16, "Hkv": 16,
         "D": 128, "P": 64, "codes": "int8", "dtype": "bf16", "window": 0, "sinks": 0},
        # chunks of longer prompts over what the cache already holds, grouped heads
        {"name": "attend_chunks", "op": "attend", "S": 5, "new_lo": 200, "new_hi": 777, "old_lo": 50, "old_hi": 9000, "Hq": 32, "Hkv": 4,
         "D": 64, "P": 128, "codes": "e4m3", "dtype": "bf16", "window": 0, "sinks": 0},
        # a whole decoding step: rotate Q and K, write K and V, attend
        {"name": "step", "op": "step", "S": 32, "new_lo": 1, "new_hi": 1, "old_lo": 60, "old_hi": 2000, "Hq": 16, "Hkv": 16,
         "D": 128, "P": 64, "codes": "int8", "dtype": "bf16", "window": 0, "sinks": 0},
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, evenly over their logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rotary", "cache", "attend", "attend", "step"))
    if op == "rotary":
        D = 16 * rng.randint(2, 8)
        heads = rng.randint(2, 40)
        period = rng.choice((0, 0, spread(rng, 7, 3000)))
        return {"op": "rotary", "tokens": spread(rng, 1, max(1, 30_000_000 // (heads * D))), "period": period, "heads": heads, "D": D,
                "rd": rng.choice((D, D, D // 2, 8 * rng.randint(1, D // 8))), "interleaved": rng.random() < 0.5,
                "dtype": rng.choice(("bf16", "fp16", "fp32")), "backward": rng.random() < 0.5,
                "scaling": rng.choice(("none", "linear", "ntk", "by_parts")), "far": rng.choice((0, spread(rng, 1000, 1_000_000)))}
    case = {"op": op, "D": rng.choice((64, 128, 16 * rng.randint(2, 8))), "P": rng.choice((16, 32, 64, 128)),
            "codes": rng.choice(("int8", "e4m3")), "dtype": rng.choice(("bf16", "fp16"))}
    if op == "cache":
        case |= {"Hkv": rng.randint(1, 16), "old_hi": spread(rng, 1, 3000), "read": "blocks"}
        if rng.random() < 0.5:  # decoding steps
            return case | {"S": spread(rng, 1, 256), "new_lo": 1, "new_hi": rng.randint(1, 6)}
        hi = spread(rng, 40, 6000)
        return case | {"S": rng.randint(1, 8), "new_lo": rng.randint(1, hi), "new_hi": hi, "read": rng.choice(("all", "blocks"))}
    kv, group = rng.randint(1, 16), rng.choice((1, 1, 2, 3, 4, 7, 8))
    while kv * group > 40:
        kv = max(1, kv // 2)
    case |= {"Hkv": kv, "Hq": kv * group, "window": 0, "sinks": 0}
    if rng.random() < 0.4:
        case |= {"window": spread(rng, 16, 5000), "sinks": rng.choice((0, 1, 4, 70))}
    if op == "step" or rng.random() < 0.6:  # decoding steps
        hi = spread(rng, 30, 12000)
        return case | {"S": spread(rng, 1, max(1, min(96, 500_000 // hi))), "new_lo": 1, "new_hi": 1 if op == "step" else rng.randint(1, 5),
                       "old_lo": rng.randint(1, hi), "old_hi": hi}
    new, old = spread(rng, 20, 3500), spread(rng, 1, 4000)
    most = max(1, int(2 * 16 * 4096 * 2048 / (case["Hq"] * new * (old + new))))
    return case | {"S": rng.randint(1, min(6, most)), "new_lo": rng.randint(1, new), "new_hi": new, "old_lo": rng.randint(0, old), "old_hi": old}


def ragged(n, lo, hi, step):
    """n whole numbers between lo and hi, most of them nearer to lo, the largest hi."""
    got = [lo + int((hi - lo) * ((i * step) % 1.0) ** 1.5) for i in range(n)]
    return got[:-1] + [hi]


def sizes(case):
    """(new tokens, older tokens) of each sequence, by the case alone."""
    return (ragged(case["S"], case["new_lo"], case["new_hi"], 0.618034),
            ragged(case["S"], case.get("old_lo", 0), case["old_hi"], 0.754878))


def visible(case):
    """For each sequence (keys that its rows see between them, pairs of row and key)."""
    got = []
    w, k = case["window"], case["sinks"]
    for n, old in zip(*sizes(case)):
        if not w:
            got.append((old + n, n * old + n * (n + 1) // 2))
            continue
        pairs = 0
        for p in range(old, old + n):
            first = max(0, p + 1 - w)
            pairs += p + 1 - first + min(k, first)
        first = max(0, old + 1 - w)
        got.append((old + n - first + min(k, first), pairs))
    return got


def work(case):
    if case["op"] == "rotary":
        n = case["tokens"] * case["heads"] * case["D"]
        return {"bytes": 2.0 * n * SIZE[case["dtype"]], "flops": 3.0 * case["tokens"] * case["heads"] * case["rd"]}
    e, D, Hkv, P = SIZE[case["dtype"]], case["D"], case["Hkv"], case["P"]
    new, old = sizes(case)
    if case["op"] == "cache":
        rows = sum(new)
        back = sum(o + n for n, o in zip(new, old)) if case["read"] == "all" else sum(o % P + n for n, o in zip(new, old))
        return {"bytes": 2.0 * Hkv * D * (rows * (e + 1) + back * (1 + e)), "flops": 2.0 * Hkv * D * (2 * rows + back)}
    rows, Hq = sum(new), case["Hq"]
    seen = visible(case)
    nbytes = 2.0 * rows * Hq * D * e + sum(s * 2.0 * D * Hkv + -(-s // P) * 8.0 * Hkv for s, _ in seen)
    flops = sum(4.0 * D * Hq * p for _, p in seen)
    if case["op"] == "step":
        nbytes += 2.0 * rows * (Hq + Hkv) * D * e + 2.0 * rows * Hkv * D * (e + 1)
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------------------ inputs --

def scaling_of(case):
    """The arguments of a rotary table: those of a model stretched to eight times its length."""
    return {"none": {}, "linear": {"factor": 8.0}, "ntk": {"factor": 8.0},
            "by_parts": {"factor": 8.0, "original_length": 4096.0, "slow": 1.0, "fast": 32.0, "amplitude": 0.1 * math.log(8.0) + 1.0}}[case["scaling"]]


def prepare_rotary(case, g):
    n, H, D = case["tokens"], case["heads"], case["D"]
    x = torch.randn((n, H, D), generator=g, device="cuda").to(DTYPES[case["dtype"]])
    positions = None
    if not case["period"]:
        positions = (torch.randint(0, 4096, (n,), generator=g, device="cuda") + case["far"]).to(torch.int32)
    s = {"x": x, "positions": positions, "out": torch.empty_like(x)}
    if own:
        import causal_attention_score_gb300 as csa
        s["rotary"] = csa.RotaryTable(case["rd"], base=10000.0, scaling=case["scaling"], device="cuda", **scaling_of(case))
    return s


def codes_of(case, shape, g):
    """What a written cache holds: codes of normal values."""
    x = torch.randn(shape, generator=g, device="cuda")
    if case["codes"] == "int8":
        return x.mul_(32).round_().clamp_(-127, 127).to(torch.int8)
    return x.mul_(96).clamp_(-448, 448).to(torch.float8_e4m3fn)


def scales_of(case, shape, g):
    """Scales of such blocks: of 8 significant bits (int8) or powers of two (e4m3)."""
    s = torch.exp2(torch.randn(shape, generator=g, device="cuda") * 0.5 - 5)
    return s.to(torch.bfloat16).float() if case["codes"] == "int8" else torch.exp2(torch.round(torch.log2(s)) - 2)


def prepare_cache(case, g):
    new, old = sizes(case)
    S, H, P, D = case["S"], case["Hkv"], case["P"], case["D"]
    total = [a + b for a, b in zip(new, old)]
    most = max(-(-t // P) for t in total)
    used = [-(-t // P) for t in total]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.zeros((S, most), dtype=torch.int32), 0
    place = torch.zeros((S, most), dtype=torch.int64)
    for i, u in enumerate(used):
        place[i, :u] = torch.arange(at, at + u)
        at += u
    table = torch.where((torch.arange(most)[None, :] < torch.tensor(used)[:, None]).cuda(), order[place.cuda()], 0).to(torch.int32)
    s = {"table": table,
         "offsets": torch.tensor([0] + [sum(new[: i + 1]) for i in range(S)], dtype=torch.int32).cuda(),
         "lengths": torch.tensor(total, dtype=torch.int32).cuda(), "spare": order[-1].long(), "rows": sum(new), "max_new": max(new)}
    for name in ("k", "v"):
        s[name] = codes_of(case, (pages, H, P, D), g)
        s[name + "_scale"] = scales_of(case, (pages, H), g)
    # slots that no token has been written to hold what was there before: here the codes of no number
    blank = -128 if case["codes"] == "int8" else 0x7F
    have = torch.tensor(total if case["op"] == "attend" else old).cuda()
    free = torch.arange(most * P, device="cuda")[None, :] >= have[:, None]
    i, t = torch.nonzero(free & (torch.arange(most * P, device="cuda")[None, :] < torch.tensor(used).cuda()[:, None] * P), as_tuple=True)
    for name in ("k", "v"):
        s[name].view(torch.uint8)[table[i, t // P].long(), :, t % P] = blank & 0xFF
    if own:
        import causal_attention_score_gb300 as csa
        s["cache"] = csa.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = csa.KvBatch(s["offsets"], s["lengths"], table, rows=s["rows"], max_new=s["max_new"])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rotary":
        return {"case": case, **prepare_rotary(case, g)}
    s = {"case": case, **prepare_cache(case, g)}
    dt, rows, D = DTYPES[case["dtype"]], s["rows"], case["D"]
    if case["op"] in ("cache", "step"):
        for name in ("k_new", "v_new"):
            # tokens differ in size, so blocks that are written to in part do get larger
            x = torch.randn((rows, case["Hkv"], D), generator=g, device="cuda")
            s[name] = (x * torch.exp2(torch.randn((rows, case["Hkv"], 1), generator=g, device="cuda") * 0.5)).to(dt)
    if case["op"] == "cache":
        new, old = sizes(case)
        back = [n + (o if case["read"] == "all" else o % case["P"]) for n, o in zip(new, old)]
        s["back_offsets"] = torch.tensor([0] + [sum(back[: i + 1]) for i in range(case["S"])], dtype=torch.int32).cuda()
        s["back_rows"], s["max_back"] = sum(back), max(back)
        s["k_back"] = torch.empty((s["back_rows"], case["Hkv"], D), dtype=dt, device="cuda")
        s["v_back"] = torch.empty_like(s["k_back"])
        if own:
            import causal_attention_score_gb300 as csa
            s["back"] = csa.KvBatch(s["back_offsets"], s["lengths"], s["table"], rows=s["back_rows"], max_new=s["max_back"])
        return s
    s["q"] = torch.randn((rows, case["Hq"], D), generator=g, device="cuda").to(dt)
    s["out"] = torch.empty_like(s["q"])
    if case["op"] == "step":
        s["positions"] = s["lengths"] - 1
        s["q_rot"], s["k_rot"] = torch.empty_like(s["q"]), torch.empty_like(s["k_new"])
        if own:
            import causal_attention_score_gb300 as csa
            s["rotary"] = csa.RotaryTable(D, base=10000.0, device="cuda")
    if own:
        import causal_attention_score_gb300 as csa
        s["workspace"] = torch.empty(csa.cache_attention_workspace_size(s["cache"], s["batch"], case["Hq"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------- plain forms --

def frequencies(rd, scaling, factor=1.0, original_length=0.0, slow=1.0, fast=32.0, amplitude=1.0, base=10000.0):
    i = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    if scaling == "ntk" and rd > 2:
        base = base * factor ** (rd / (rd - 2))
    f = torch.exp(-2 * i / rd * math.log(base))
    if scaling == "linear":
        f = f / factor
    if scaling == "by_parts":
        keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f


def plain_rotary(x, positions, f, interleaved, backward, amplitude):
    rd = 2 * f.numel()
    angle = positions.double()[:, None] * f
    cos, sin = (amplitude * torch.cos(angle)).float()[:, None], (amplitude * torch.sin(angle)).float()[:, None]
    if backward:
        sin = -sin
    y = x.float().clone()
    a, b = (y[..., 0:rd:2], y[..., 1:rd:2]) if interleaved else (y[..., : rd // 2], y[..., rd // 2: rd])
    u, w = a * cos - b * sin, b * cos + a * sin
    a.copy_(u)
    b.copy_(w)
    return y.to(x.dtype)


def plain_scale(amax, codes):
    """The scale of a block by its largest magnitude, exact in fp32."""
    if codes == "int8":
        s = ((amax / 127).view(torch.int32) & -65536).view(torch.float32)
        s = torch.where(s * 127 < amax, (s.view(torch.int32) + 65536).view(torch.float32), s)
    else:
        m, e = torch.frexp(amax)  # amax = m 2^e with 0.5 <= m < 1, and 448 = 0.875 * 2^9
        s = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).int()), torch.zeros_like(amax))
    return s.clamp(min=FLOOR)


def plain_codes(y, codes):
    """Values in units of the scale, as codes (NaN: 0)."""
    if codes == "int8":
        return torch.round(y).nan_to_num(0.0, 127.0, -127.0).clamp(-127, 127).to(torch.int8)
    return y.nan_to_num(0.0, 448.0, -448.0).clamp(-448, 448).to(torch.float8_e4m3fn)


def plain_write(pool, scale, x, case, s):
    """The new rows of x into one pool, block by block."""
    S, P, H, D = case["S"], case["P"], case["Hkv"], case["D"]
    n = (s["offsets"][1:] - s["offsets"][:-1]).long()
    start = s["lengths"].long() - n
    first = start // P
    J = (s["max_new"] + 2 * P - 2) // P
    pos = (first * P)[:, None] + torch.arange(J * P, device="cuda")
    fresh = ((pos >= start[:, None]) & (pos < s["lengths"].long()[:, None])).view(S, J, P)
    older = (pos < start[:, None]).view(S, J, P)
    row = (s["offsets"][:-1].long()[:, None] + pos - start[:, None]).clamp(0, s["rows"] - 1)
    y = x[row].float().view(S, J, P, H, D).transpose(2, 3)  # [S, J, H, P, D]
    fm, om = fresh[:, :, None, :, None], older[:, :, None, :, None]
    amax = torch.where(fm & y.isfinite(), y.abs(), 0.0).amax((3, 4))
    touched = fresh.any(2)
    page = s["table"].long().gather(1, (first[:, None] + torch.arange(J, device="cuda")).clamp(max=s["table"].shape[1] - 1))
    page = torch.where(touched, page, s["spare"])  # a page of no sequence, which keeps what it holds
    was = torch.where(older.any(2)[:, :, None], scale[page], 0.0)
    now = torch.maximum(was, plain_scale(amax, case["codes"]))
    held = pool[page]
    grown = plain_codes(torch.where(om, held.float(), 0.0) * was[..., None, None] / now[..., None, None], case["codes"])
    made = plain_codes(torch.where(fm, y, 0.0) / now[..., None, None], case["codes"])
    bits = torch.where(fm, made.view(torch.uint8), torch.where(om, grown.view(torch.uint8), held.view(torch.uint8)))
    pool.view(torch.uint8)[page] = torch.where(touched[:, :, None, None, None], bits, held.view(torch.uint8))
    scale[page] = torch.where(touched[:, :, None], now, scale[page])


def plain_read(pool, scale, offsets, lengths, table, rows, P, dtype):
    """The last tokens of each sequence, as many as it has rows in offsets."""
    r = torch.arange(rows, device="cuda")
    i = torch.searchsorted(offsets[1:].long().contiguous(), r, right=True)
    pos = lengths.long()[i] - offsets[1:].long()[i] + r
    page = table.long()[i, pos // P]
    return (pool[page, :, pos % P].float() * scale[page][..., None]).to(dtype)


def plain_attend(q, case, s):
    """Scores of every row with every key of its sequence, padded to the longest."""
    S, Hq, Hkv, D, P = case["S"], case["Hq"], case["Hkv"], case["D"], case["P"]
    G, most = Hq // Hkv, s["table"].shape[1] * P
    lengths, offsets = s["lengths"].long(), s["offsets"].long()
    n = offsets[1:] - offsets[:-1]
    t = torch.arange(most, device="cuda")
    j = torch.arange(s["max_new"], device="cuda")
    pos = (lengths - n)[:, None] + j  # [S, N]
    see = (t <= pos[..., None]) & (j < n[:, None])[..., None]
    if case["window"]:
        see &= (pos[..., None] - t < case["window"]) | (t < case["sinks"])
    row = (offsets[:-1, None] + j).clamp(max=s["rows"] - 1)
    qs = q[row].float().view(S, -1, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D)
    live = (t < lengths[:, None])[:, None, :, None]

    def values(pool, scale):
        x = pool[s["table"].long()].float() * scale[s["table"].long()][..., None, None]  # [S, pages, Hkv, P, D]
        return torch.where(live, x.transpose(1, 2).reshape(S, Hkv, most, D), 0.0)

    a = (qs @ values(s["k"], s["k_scale"]).transpose(2, 3)).view(S, Hkv, G, -1, most)
    a = a.mul_(1 / math.sqrt(D)).masked_fill_(~see[:, None, None], -math.inf)
    a = a.sub_(a.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = a.sum(-1, keepdim=True)
    o = (a.view(S, Hkv, -1, most) @ values(s["v"], s["v_scale"])).view(S, Hkv, G, -1, D) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, -1, Hq, D)
    i = torch.searchsorted(offsets[1:].contiguous(), torch.arange(s["rows"], device="cuda"), right=True)
    return o[i, torch.arange(s["rows"], device="cuda") - offsets[i]].to(q.dtype)


# --------------------------------------------------------------------------- one pass --

def run(state):
    s, case = state, state["case"]
    if own:
        return run_own(s, case)
    if case["op"] == "rotary":
        f = frequencies(case["rd"], case["scaling"], **scaling_of(case))
        positions = s["positions"] if s["positions"] is not None else torch.arange(case["tokens"], device="cuda") % case["period"] + case["far"]
        return plain_rotary(s["x"], positions, f, case["interleaved"], case["backward"], scaling_of(case).get("amplitude", 1.0))
    if case["op"] == "cache":
        for name in ("k", "v"):
            plain_write(s[name], s[name + "_scale"], s[name + "_new"], case, s)
        back = [plain_read(s[name], s[name + "_scale"], s["back_offsets"], s["lengths"], s["table"], s["back_rows"], case["P"], s["k_back"].dtype)
                for name in ("k", "v")]
        return {"k": back[0], "v": back[1], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if case["op"] == "attend":
        return plain_attend(s["q"], case, s)
    f = frequencies(case["D"], "none")
    q = plain_rotary(s["q"], s["positions"], f, False, False, 1.0)
    k = plain_rotary(s["k_new"], s["positions"], f, False, False, 1.0)
    plain_write(s["k"], s["k_scale"], k, case, s)
    plain_write(s["v"], s["v_scale"], s["v_new"], case, s)
    # (K's scales follow from the rotated K, whose last bit may differ)
    return {"out": plain_attend(q, case, s), "q": q, "k": k, "v_scale": s["v_scale"]}


def run_own(s, case):
    import causal_attention_score_gb300 as csa
    if case["op"] == "rotary":
        call = csa.rotary_backward if case["backward"] else csa.rotary_forward
        start = case["far"] if s["positions"] is None else 0
        call(s["out"], s["x"], s["rotary"], s["positions"], start=start, period=case["period"], interleaved=case["interleaved"])
        return s["out"]
    if case["op"] == "cache":
        csa.kv_cache_write(s["cache"], s["batch"], s["k_new"], s["v_new"])
        csa.kv_cache_read(s["k_back"], s["v_back"], s["cache"], s["back"])
        return {"k": s["k_back"], "v": s["v_back"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if case["op"] == "attend":
        csa.cache_attention_forward(s["out"], s["q"], s["cache"], s["batch"], window=case["window"], sinks=case["sinks"], workspace=s["workspace"])
        return s["out"]
    csa.rotary_forward(s["q_rot"], s["q"], s["rotary"], s["positions"])
    csa.rotary_forward(s["k_rot"], s["k_new"], s["rotary"], s["positions"])
    csa.kv_cache_write(s["cache"], s["batch"], s["k_rot"], s["v_new"])
    csa.cache_attention_forward(s["out"], s["q_rot"], s["cache"], s["batch"], window=case["window"], sinks=case["sinks"], workspace=s["workspace"])
    return {"out": s["out"], "q": s["q_rot"], "k": s["k_rot"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------------------- in 64 bits --

def exact_rotary(x, positions, case_rd, scaling, args, interleaved, backward):
    """Each pair as a complex number times a unit one (its conjugate backward)."""
    base, rd = 10000.0, case_rd
    factor = args.get("factor", 1.0)
    f = []
    for i in range(rd // 2):
        w = (base * factor ** (rd / (rd - 2)) if scaling == "ntk" and rd > 2 else base) ** (-2.0 * i / rd)
        if scaling == "linear":
            w /= factor
        if scaling == "by_parts":
            turns = args["original_length"] * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - args["slow"]) / (args["fast"] - args["slow"])))
            w = w * keep + w / factor * (1 - keep)
        f.append(w)
    angle = torch.outer(positions.double(), torch.tensor(f, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.full_like(angle, args.get("amplitude", 1.0)), -angle if backward else angle)[:, None]
    y = x.double()
    head = y[..., :rd].unflatten(-1, (rd // 2, 2)) if interleaved else y[..., :rd].unflatten(-1, (2, rd // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, y[..., rd:]], -1)


def exact_scale(amax, codes):
    if codes == "e4m3":
        e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448) - 1)
        for _ in range(3):
            e = torch.where(448 * torch.exp2(e) < amax, e + 1, e)
        s = torch.exp2(e)
    else:
        want = amax / 127
        unit = torch.exp2(torch.floor(torch.log2(want.clamp(min=1e-300))) - 7)
        s = torch.ceil(want / unit) * unit
    return s.clamp(min=FLOOR)


def exact_round(y, codes):
    if codes == "int8":
        return y.round().clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return ((y / step).round() * step).clamp(-448, 448)


def exact_pools(case, s, k_new):
    """Values of every slot and scales after the write, one sequence and block at a time."""
    got = {}
    new, old = sizes(case)
    P = case["P"]
    table, at = s["table"].cpu(), s["offsets"].cpu()
    for name, x in (("k", k_new), ("v", s["v_new"].double())):
        codes, scale = s[name].double(), s[name + "_scale"].double()
        for i, (n, o) in enumerate(zip(new, old)):
            for j in range(o // P, (o + n - 1) // P + 1):
                a, b = max(o, j * P), min(o + n, j * P + P)
                page = int(table[i, j])
                rows = x[int(at[i]) + a - o: int(at[i]) + b - o].transpose(0, 1)  # [H, tokens, D]
                s1 = exact_scale(rows.abs().amax((1, 2)), case["codes"])
                if a > j * P:
                    s1 = torch.maximum(s1, scale[page])
                    codes[page, :, : a - j * P] = exact_round(codes[page, :, : a - j * P] * (scale[page] / s1)[:, None, None], case["codes"])
                codes[page, :, a - j * P: b - j * P] = exact_round(rows / s1[:, None, None], case["codes"])
                scale[page] = s1
        got[name], got[name + "_scale"] = codes, scale
    return got


def exact_attend(q, pools, case, s):
    new, old = sizes(case)
    P, D, G = case["P"], case["D"], case["Hq"] // case["Hkv"]
    outs, at = [], 0
    for i, (n, o) in enumerate(zip(new, old)):
        L = n + o
        pages = s["table"][i, : -(-L // P)].long()
        k, v = ((pools[x][pages].double() * pools[x + "_scale"][pages].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :L] for x in ("k", "v"))
        row = torch.arange(o, L, device="cuda")[:, None]
        key = torch.arange(L, device="cuda")[None]
        hide = key > row
        if case["window"]:
            hide = hide | ((key <= row - case["window"]) & (key >= case["sinks"]))
        out = torch.empty((n, case["Hq"], D), dtype=torch.float64, device="cuda")
        for h in range(case["Hkv"]):
            a = torch.einsum("nhd,td->hnt", q[at: at + n, h * G: h * G + G].double(), k[h]) / math.sqrt(D)
            a = torch.softmax(a.masked_fill(hide, -math.inf), -1)
            out[:, h * G: h * G + G] = torch.einsum("hnt,td->nhd", a, v[h])
        outs.append(out)
        at += n
    return torch.cat(outs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        positions = s["positions"] if s["positions"] is not None else torch.arange(case["tokens"], device="cuda") % case["period"] + case["far"]
        return exact_rotary(s["x"], positions, case["rd"], case["scaling"], scaling_of(case), case["interleaved"], case["backward"])
    if case["op"] == "attend":
        return exact_attend(s["q"], s, case, s)
    if case["op"] == "step":
        # what the step rounds to its type between the operators is rounded here too
        q, k = (exact_rotary(s[n], s["positions"], case["D"], "none", {}, False, False) for n in ("q", "k_new"))
        pools = exact_pools(case, s, k.to(s["k_new"].dtype).double())
        return {"out": exact_attend(q.to(s["q"].dtype), pools, case, s), "q": q, "k": k, "v_scale": pools["v_scale"]}
    pools = exact_pools(case, s, s["k_new"].double())
    new, old = sizes(case)
    back = {"k": [], "v": []}
    for i, (n, o) in enumerate(zip(new, old)):
        first = 0 if case["read"] == "all" else o - o % case["P"]
        pages = s["table"][i, : -(-(n + o) // case["P"])].long()
        for name in ("k", "v"):
            x = pools[name][pages] * pools[name + "_scale"][pages][..., None, None]  # [pages, H, P, D]
            back[name].append(x.transpose(1, 2).flatten(0, 1)[first: n + o])
    return {"k": torch.cat(back["k"]), "v": torch.cat(back["v"]), "k_scale": pools["k_scale"], "v_scale": pools["v_scale"]}
