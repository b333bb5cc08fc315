"""Cases and plain forms of the operators around answers that share a prompt: the pages of a cache
(forked, extended, freed, copied, compacted), attention for a batch whose sequences share a long
prefix, and the log probabilities of given tokens with entropy, top alternatives and gradient.

``run`` is one pass of an operator. With ``own`` false it is computed by elementary torch operations
in 32 bits; with ``own`` true by the library's entry points. ``exact`` gives the same outputs from
the definitions in 64 bits.

Layouts: logits [rows, vocab]; cache codes [pages, heads, P, D] with one fp32 scale for each page and
head; ``refs`` [pages] how many table entries name a page, ``lengths`` [S], ``table`` [S, width] the
pages of each sequence; ``offsets`` [S + 1] each sequence's rows among the new tokens; ``groups``
[G + 1]: sequences groups[g] .. groups[g + 1] - 1 share their first ``shared[g]`` tokens.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
ENTROPY_WEIGHT, TOP_WEIGHT = 0.01, 0.1


# ------------------------------------------------------------------------------- cases --

def listed():
    return [
        # the last token of one sequence, with the alternatives that an answer's reader asks for: latency
        {"name": "logprobs_one", "op": "logprobs", "rows": 1, "vocab": 50257, "pitch": 50257, "top": 20, "dtype": "bf16", "grad": False,
         "masked": 0.0, "padded": 0.0, "scale": 1.0},
        # a decoding step of 48 sequences at temperature 0.7, a part of the vocabulary forbidden; a dense layer's fp32 result
        {"name": "logprobs_step", "op": "logprobs", "rows": 48, "vocab": 50257, "pitch": 50257, "top": 5, "dtype": "fp32", "grad": False,
         "masked": 0.3, "padded": 0.0, "scale": 1.0 / 0.7},
        # scoring the tokens of a training batch (8 x 1024) with its entropy
        {"name": "logprobs_score", "op": "logprobs", "rows": 8192, "vocab": 50257, "pitch": 50264, "top": 2, "dtype": "fp32", "grad": False,
         "masked": 0.0, "padded": 0.05, "scale": 1.0},
        # log probabilities and entropy of such a batch, and the gradient of a loss made of them
        {"name": "logprobs_train", "op": "logprobs", "rows": 8192, "vocab": 50257, "pitch": 50304, "top": 0, "dtype": "bf16", "grad": True,
         "masked": 0.0, "padded": 0.1, "scale": 1.0},
        # four answers to a short prompt, every head with its own keys: latency
        {"name": "shared_few", "op": "attend", "S": 4, "G": 1, "alone": 0, "shared_lo": 1040, "shared_hi": 1040, "old_lo": 3, "old_hi": 90,
         "new_lo": 1, "new_hi": 1, "Hq": 12, "Hkv": 12, "D": 64, "P": 16, "codes": "e4m3", "dtype": "fp16"},
        # 64 answers sampled from one long prompt, a token of each
        {"name": "shared_answers", "op": "attend", "S": 64, "G": 1, "alone": 0, "shared_lo": 8192, "shared_hi": 8192, "old_lo": 1, "old_hi": 1000,
         "new_lo": 1, "new_hi": 1, "Hq": 32, "Hkv": 8, "D": 128, "P": 64, "codes": "int8", "dtype": "bf16"},
        # a server's batch over four long documents and some requests of their own, drafted tokens being checked
        {"name": "shared_documents", "op": "attend", "S": 200, "G": 4, "alone": 8, "shared_lo": 4096, "shared_hi": 32768, "old_lo": 20, "old_hi": 900,
         "new_lo": 1, "new_hi": 3, "Hq": 32, "Hkv": 8, "D": 128, "P": 32, "codes": "e4m3", "dtype": "bf16"},
        # requests that begin behind one set of instructions
        {"name": "shared_prompts", "op": "attend", "S": 16, "G": 1, "alone": 0, "shared_lo": 6016, "shared_hi": 6016, "old_lo": 0, "old_hi": 0,
         "new_lo": 60, "new_hi": 400, "Hq": 16, "Hkv": 16, "D": 64, "P": 64, "codes": "int8", "dtype": "bf16"},
        # a prompt forked into four answers and the next token's room made, beside three other sequences
        {"name": "fork_few", "op": "fork", "prompts": 1, "answers": 4, "running": 2, "finished": 1, "long": 700, "spare": 24,
         "Hkv": 12, "D": 64, "P": 64, "codes": "int8"},
        # a server's turn: 24 sequences finish, 32 prompts of eight answers each begin, 96 go on
        {"name": "fork_many", "op": "fork", "prompts": 32, "answers": 8, "running": 96, "finished": 24, "long": 2500, "spare": 900,
         "Hkv": 8, "D": 128, "P": 64, "codes": "e4m3"},
        # a small cache put in order, one prompt kept in another
        {"name": "compact_few", "op": "compact", "running": 6, "finished": 2, "kept": 1, "long": 300, "spare": 40, "Hkv": 12, "D": 64, "P": 16, "codes": "int8"},
        # a cache of about a gigabyte after much coming and going, so that its end can be given back
        {"name": "compact_many", "op": "compact", "running": 160, "finished": 60, "kept": 12, "long": 4000, "spare": 2400, "Hkv": 8, "D": 128, "P": 64,
         "codes": "int8"},
    ]


def spread(rng, lo, hi):
    """A whole number between lo and hi, evenly over their logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("logprobs", "logprobs", "attend", "attend", "attend", "fork", "compact"))
    if op == "logprobs":
        vocab = rng.choice((50257, spread(rng, 17, 200_000), spread(rng, 5000, 200_000)))
        grad = rng.random() < 0.5
        return {"op": op, "rows": spread(rng, 1, max(1, min(20_000, 400_000_000 // vocab // (1 + grad)))), "vocab": vocab,
                "pitch": vocab + rng.choice((0, 0, 3, -vocab % 64)), "top": min(vocab, rng.choice((0, 1, 5, 20, 32))),
                "dtype": rng.choice(("bf16", "fp16", "fp32")), "grad": grad, "masked": rng.choice((0.0, 0.0, 0.5)),
                "padded": rng.choice((0.0, 0.2)), "scale": rng.choice((1.0, 1.0 / 0.7, 0.5))}
    if op == "fork":
        kv, D, P = rng.randint(1, 16), 16 * rng.randint(1, 8), rng.choice((16, 32, 64, 128))
        return {"op": op, "prompts": spread(rng, 1, 24), "answers": spread(rng, 1, 10), "running": rng.randint(0, 80), "finished": rng.randint(1, 30),
                "long": spread(rng, 20, 1500), "spare": 300, "Hkv": min(kv, 8), "D": D, "P": P, "codes": rng.choice(("int8", "e4m3"))}
    if op == "compact":
        kv, D, P = rng.randint(1, 8), 16 * rng.randint(1, 8), rng.choice((16, 32, 64, 128))
        running = spread(rng, 1, 120)
        return {"op": op, "running": running, "finished": rng.randint(1, 60), "kept": rng.randint(1, min(running, 9)), "long": spread(rng, 20, 3000),
                "spare": spread(rng, 10, 1200), "Hkv": kv, "D": D, "P": P, "codes": rng.choice(("int8", "e4m3"))}
    kv, group = rng.randint(1, 12), rng.choice((1, 1, 2, 3, 4, 7, 8))
    while kv * group > 32:
        kv = max(1, kv // 2)
    P, S = rng.choice((16, 32, 64, 128)), spread(rng, 1, 120)
    case = {"op": "attend", "D": rng.choice((64, 128, 16 * rng.randint(2, 8))), "P": P, "codes": rng.choice(("int8", "e4m3")),
            "dtype": rng.choice(("bf16", "fp16")), "Hkv": kv, "Hq": kv * group, "S": S, "G": rng.randint(1, max(1, min(6, S // 2))),
            "alone": rng.choice((0, 0, S // 5))}
    if rng.random() < 0.3:  # prompts behind a shared beginning
        new, S = spread(rng, 10, 300), min(S, 12)
        hi = spread(rng, 200, 5000)
        return case | {"S": S, "G": min(case["G"], S), "alone": 0, "new_lo": rng.randint(1, new), "new_hi": new, "old_lo": 0, "old_hi": rng.choice((0, 50)),
                       "shared_lo": spread(rng, 200, hi), "shared_hi": hi}
    old, hi = spread(rng, 2, 800), spread(rng, 200, 16000)
    return case | {"new_lo": 1, "new_hi": rng.choice((1, 1, 4)), "old_lo": rng.randint(1, old), "old_hi": old, "shared_lo": spread(rng, 200, hi), "shared_hi": hi}


def ragged(n, lo, hi, step):
    """n whole numbers between lo and hi, most of them nearer to lo, the largest hi."""
    got = [lo + int((hi - lo) * ((i * step) % 1.0) ** 1.5) for i in range(n)]
    return got[:-1] + [hi] if n else []


def parts(case):
    """An attention case by itself: (new tokens, older tokens of its own, group or -1) of each sequence, shared tokens of
    each group (whole pages), the groups' bounds."""
    S, G, P = case["S"], case["G"], case["P"]
    members = S - case["alone"]
    bounds = [members * g // G for g in range(G + 1)]
    shared = [max(P, t - t % P) for t in ragged(G, case["shared_lo"], case["shared_hi"], 0.381966)]
    group = [next(g for g in range(G) if bounds[g] <= s < bounds[g + 1]) if s < members else -1 for s in range(S)]
    return ragged(S, case["new_lo"], case["new_hi"], 0.618034), ragged(S, case["old_lo"], case["old_hi"], 0.754878), group, shared, bounds


def sequences(case):
    """A case of pages by itself: each sequence's length (0: none yet), as prompts, the running, the finished, answers."""
    prompts, answers = case.get("prompts", 0), case.get("answers", 0)
    n = prompts + case["running"] + case["finished"]
    return ragged(n, max(1, case["long"] // 8), case["long"], 0.618034) + [0] * (prompts * answers)


def work(case):
    if case["op"] == "logprobs":
        n = float(case["rows"]) * case["vocab"]
        return {"bytes": n * SIZE[case["dtype"]] * (2 if case["grad"] else 1), "flops": n * (12 if case["grad"] else 6)}
    D, Hkv, P = case["D"], case["Hkv"], case["P"]
    if case["op"] == "attend":
        new, old, group, shared, _ = parts(case)
        Hq = case["Hq"]
        keys = sum(shared) + sum(n + o for n, o in zip(new, old))
        pairs = sum(n * ((shared[g] if g >= 0 else 0) + o) + n * (n + 1) // 2 for n, o, g in zip(new, old, group))
        return {"bytes": 2.0 * sum(new) * Hq * D * SIZE[case["dtype"]] + 2.0 * keys * Hkv * (D + 4.0 / P), "flops": 4.0 * D * Hq * pairs}
    lengths = sequences(case)
    pages = sum(-(-t // P) for t in lengths) + case["spare"]
    entries = 4.0 * sum(-(-t // P) for t in lengths)
    if case["op"] == "fork":
        # refs read, the prompts' table rows copied, the written part of each prompt's last page
        prompts, answers = case["prompts"], case["answers"]
        tail = sum(2.0 * Hkv * ((t % P) * D + 8) for t in lengths[:prompts] if t % P)
        rows = 4.0 * sum(-(-t // P) for t in lengths[:prompts])
        return {"bytes": 4.0 * pages + (1 + answers) * (tail + rows), "flops": 1.0 * pages}
    # what has to move: pages of running sequences past their number (their places are random: on average that share)
    live = sum(-(-t // P) for t in lengths[: case["running"]])
    kept = sum(-(-t // P) for t in lengths[: case["kept"]])
    moved = live * (pages - live) / pages + kept
    return {"bytes": 4.0 * pages + entries + 2.0 * moved * 2.0 * Hkv * (P * D + 4), "flops": 1.0 * pages}


# ------------------------------------------------------------------------------ inputs --

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


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare_logprobs(case, g):
    rows, V, pitch, dt = case["rows"], case["vocab"], case["pitch"], DTYPES[case["dtype"]]
    held = torch.empty((rows, pitch), dtype=dt, device="cuda")
    logits = held[:, :V]
    tokens = torch.randint(0, V, (rows,), generator=g, device="cuda")
    for i in range(0, rows, 1024):  # logits of a trained model: normal, a few words far ahead, the given one likely
        x = torch.randn((min(1024, rows - i), V), generator=g, device="cuda").mul_(2.5)
        n = x.shape[0]
        x[torch.arange(n, device="cuda"), torch.randint(0, V, (n,), generator=g, device="cuda")] += 9
        if case["masked"]:
            x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < case["masked"], -math.inf)
        t = tokens[i: i + n, None]
        x.scatter_(1, t, x.gather(1, t).clamp(min=-8) + 8)
        logits[i: i + n] = x
    padding = torch.rand((rows,), generator=g, device="cuda") < case["padded"]
    s = {"logits": logits, "tokens": torch.where(padding, -1, tokens).to(torch.int32)}
    if case["grad"]:
        s["d_logprob"] = torch.randn((rows,), generator=g, device="cuda") / rows
        s["d_entropy"] = torch.full((rows,), -ENTROPY_WEIGHT / rows, device="cuda")
        s["d_top"] = torch.randn((rows, case["top"]), generator=g, device="cuda") * (TOP_WEIGHT / rows)
        s["dlogits"] = torch.empty_like(held)[:, :V]
    for name, shape in (("logprob", (rows,)), ("entropy", (rows,)), ("stats", (rows, 2)), ("top_logprob", (rows, case["top"]))):
        s[name] = torch.empty(shape, device="cuda")
    s["top_token"] = torch.empty((rows, case["top"]), dtype=torch.int32, device="cuda")
    return s


def prepare_attend(case, g):
    new, old, group, shared, bounds = parts(case)
    S, H, P, D = case["S"], case["Hkv"], case["P"], case["D"]
    before = [shared[i] if i >= 0 else 0 for i in group]
    total = [b + o + n for b, o, n in zip(before, old, new)]
    width = max(-(-t // P) for t in total)
    pages = sum(b // P for b in shared) + sum(-(-t // P) - b // P for t, b in zip(total, before)) + 2
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    place, at = torch.full((S, width), pages - 1, dtype=torch.int64), 0
    for i, t in enumerate(shared):
        place[bounds[i]: bounds[i + 1], : t // P] = torch.arange(at, at + t // P)
        at += t // P
    for i, (t, b) in enumerate(zip(total, before)):
        n = -(-t // P) - b // P
        place[i, b // P: b // P + n] = torch.arange(at, at + n)
        at += n
    s = {"table": order[place.cuda()].contiguous(), "offsets": ints(0, *np.cumsum(new).tolist()), "lengths": ints(*total), "rows": sum(new),
         "max_new": max(new), "groups": ints(*bounds), "shared": ints(*shared), "total": total, "new": new}
    for name in ("k", "v"):
        s[name] = codes_of(case, (pages, H, P, D), g)
        s[name + "_scale"] = scales_of(case, (pages, H), g)
    s["q"] = torch.randn((s["rows"], case["Hq"], D), generator=g, device="cuda").to(DTYPES[case["dtype"]])
    s["out"] = torch.empty_like(s["q"])
    if own:
        import causal_attention_score_gb300 as csa
        s["cache"] = csa.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = csa.KvBatch(s["offsets"], s["lengths"], s["table"], rows=s["rows"], max_new=s["max_new"])
        size = csa.cache_attention_shared_workspace_size(s["cache"], s["batch"], case["Hq"], case["G"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def prepare_pages(case, g):
    lengths, P, H, D = sequences(case), case["P"], case["Hkv"], case["D"]
    S, prompts, answers = len(lengths), case.get("prompts", 0), case.get("answers", 0)
    used = [-(-t // P) for t in lengths]
    pages = sum(used) + case["spare"] + (prompts * answers * 2 if case["op"] == "fork" else 0)
    width = -(-(max(lengths) + 1) // P)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.full((S, width), -1, dtype=torch.int32), 0
    for i, u in enumerate(used):
        table[i, :u] = order[at: at + u].cpu()
        at += u
    refs = torch.zeros((pages,), dtype=torch.int32, device="cuda")
    refs[order[:at].long()] = 1
    # one buffer of the books, so that each pass begins with them as the server's turn finds them
    s = {"saved": torch.cat([refs, ints(*lengths), table.cuda().flatten()])}
    s["ints"] = s["saved"].clone()
    s["refs"], s["lengths"], s["table"] = s["ints"][:pages], s["ints"][pages: pages + S], s["ints"][pages + S:].view(S, width)
    for name in ("k", "v"):
        s[name] = codes_of(case, (pages, H, P, D), g)
        s[name + "_scale"] = scales_of(case, (pages, H), g)
    running, finished = case["running"], case["finished"]
    s["finished"] = torch.arange(prompts + running, prompts + running + finished, dtype=torch.int32, device="cuda")
    if case["op"] == "fork":
        s["parents"] = torch.arange(prompts, device="cuda").repeat_interleave(answers).to(torch.int32)
        s["children"] = torch.arange(S - prompts * answers, S, dtype=torch.int32, device="cuda")
        s["grow"] = torch.cat([torch.arange(prompts, prompts + running, dtype=torch.int32, device="cuda"), s["children"]])
        s["more"] = torch.ones_like(s["grow"])
    else:
        kept = sum(used[: case["kept"]])
        s["from"], s["to"] = order[:kept].contiguous(), torch.randperm(kept, generator=g, device="cuda").to(torch.int32)
        for name in ("k", "v"):
            s["store_" + name] = torch.zeros((kept, H, P, D), dtype=s[name].dtype, device="cuda")
            s["store_" + name + "_scale"] = torch.zeros((kept, H), device="cuda")
        s["moves"] = torch.empty((pages,), dtype=torch.int32, device="cuda")
        s["in_use"] = torch.empty((1,), dtype=torch.int32, device="cuda")
    if own:
        import causal_attention_score_gb300 as csa
        s["cache"] = csa.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["pages"] = csa.KvPages(s["refs"], s["lengths"], s["table"], page_tokens=P)
        s["workspace"] = torch.empty(csa.kv_pages_workspace_size(s["pages"], S), dtype=torch.uint8, device="cuda")
        if case["op"] == "compact":
            s["store"] = csa.KvCache(s["store_k"], s["store_v"], s["store_k_scale"], s["store_v_scale"])
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"logprobs": prepare_logprobs, "attend": prepare_attend, "fork": prepare_pages, "compact": prepare_pages}[case["op"]]
    return {"case": case, **make(case, g)}


# ------------------------------------------------------------------------- plain forms --

def plain_logprobs(s, case):
    """Log probabilities of the tokens, entropy, the top alternatives, and the gradient of
    sum d_logprob logprob + d_entropy entropy + d_top top_logprob."""
    live = s["tokens"] >= 0
    t = s["tokens"].long().clamp(min=0)[:, None]
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    d = (x - m) * case["scale"]
    e = d.exp()
    total = e.sum(1, keepdim=True)
    log_total = total.log()
    logp = d - log_total
    entropy = log_total - (e * d.clamp(min=-1e30)).sum(1, keepdim=True) / total
    got = {"logprob": torch.where(live, logp.gather(1, t)[:, 0], 0.0), "entropy": torch.where(live, entropy[:, 0], 0.0),
           "stats": torch.where(live[:, None], torch.cat([m, log_total], 1), 0.0)}
    top, column = [], torch.arange(case["vocab"], device="cuda")
    left = torch.ones_like(x, dtype=torch.bool) if case["top"] else None
    for _ in range(case["top"]):  # the largest that is left, of equal ones the first
        most = torch.where(left, x, -math.inf).amax(1, keepdim=True)
        i = torch.where(left & (x == most), column, case["vocab"]).amin(1, keepdim=True)
        left.scatter_(1, i, False)
        top.append(i)
    index = torch.cat(top, 1) if top else t[:, :0]
    got["top_logprob"] = torch.where(live[:, None], logp.gather(1, index), 0.0)
    got["top_token"] = torch.where(live[:, None], index, -1).to(torch.int32)
    if case["grad"]:
        p = e / total
        c = (s["d_logprob"] + s["d_top"].sum(1))[:, None] + s["d_entropy"][:, None] * (logp.clamp(min=-1e30) + entropy)
        dx = -p * c
        dx.scatter_add_(1, t, s["d_logprob"][:, None])
        dx.scatter_add_(1, index, s["d_top"])
        got["dlogits"] = torch.where(live[:, None], dx * case["scale"], 0.0).to(s["logits"].dtype)
    return got


def plain_attend(s, case):
    """Sequence by sequence: scores of its rows with every key that it holds."""
    Hkv, D, P = case["Hkv"], case["D"], case["P"]
    G, outs, at = case["Hq"] // Hkv, [], 0
    for i, (n, L) in enumerate(zip(s["new"], s["total"])):
        pages = s["table"][i, : -(-L // P)].long()
        k, v = ((s[x][pages].float() * s[x + "_scale"][pages][..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :L] for x in ("k", "v"))
        q = s["q"][at: at + n].float().view(n, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, n * G, D)
        a = (q @ k.transpose(1, 2)).view(Hkv, n, G, L).mul_(1 / math.sqrt(D))
        hide = torch.arange(L, device="cuda") > torch.arange(L - n, L, device="cuda")[:, None]
        a = a.masked_fill_(hide[None, :, None], -math.inf)
        a = a.sub_(a.amax(-1, keepdim=True)).exp_()
        o = (a.view(Hkv, n * G, L) @ v).view(Hkv, n, G, D) / a.sum(-1, keepdim=True)
        outs.append(o.permute(1, 0, 2, 3).reshape(n, case["Hq"], D))
        at += n
    return torch.cat(outs).to(s["q"].dtype)


def plain_free(s, ids, P):
    rows = s["table"][ids.long()]
    held = torch.arange(rows.shape[1], device="cuda") < ((s["lengths"][ids.long()] + P - 1) // P)[:, None]
    s["refs"].scatter_add_(0, rows[held].long(), torch.full_like(rows[held], -1))
    s["lengths"][ids.long()] = 0


def plain_extend(s, ids, more, P):
    """Room for more tokens: new pages are the free ones of the lowest numbers, in the order of ids."""
    i, old = ids.long(), s["lengths"][ids.long()]
    b0, b1 = (old + P - 1) // P, (old + more + P - 1) // P
    column = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (column >= b0[:, None]) & (column < b1[:, None])
    free = torch.nonzero(s["refs"] == 0)[:, 0]
    page = free[: int(fresh.sum())].to(torch.int32)
    row, col = torch.nonzero(fresh, as_tuple=True)
    s["table"][i[row], col] = page
    s["refs"][page.long()] = 1
    s["lengths"][i] = old + more


def plain_fork(s, parents, children, P):
    """Children with their parents' tokens: whole pages are shared, the written part of a last one copied."""
    p, c = parents.long(), children.long()
    L = s["lengths"][p]
    column = torch.arange(s["table"].shape[1], device="cuda")
    whole = column < (L // P)[:, None]
    rows = s["table"][p]
    shared = rows[whole].long()
    s["refs"].scatter_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    part = L % P > 0
    free = torch.nonzero(s["refs"] == 0)[:, 0]
    to = free[: int(part.sum())]
    last = (L // P)[part].long()
    source = rows[part, last].long()
    s["table"][c] = torch.where(whole, rows, s["table"][c])
    s["table"][c[part], last] = to.to(torch.int32)
    s["refs"][to] = 1
    s["lengths"][c] = L
    written = (torch.arange(P, device="cuda") < (L % P)[part, None])[:, None, :, None]
    for name in ("k", "v"):
        pool = s[name].view(torch.uint8)
        pool[to] = torch.where(written, pool[source], pool[to])
        s[name + "_scale"][to] = s[name + "_scale"][source]


def plain_compact(s, P):
    """Pages in use past their number move to the free ones below it, both in ascending order."""
    n = int((s["refs"] > 0).sum())
    live = torch.nonzero(s["refs"] > 0)[:, 0]
    source = live[live >= n]
    to = torch.nonzero(s["refs"][:n] == 0)[:, 0]
    for name in ("k", "v", "k_scale", "v_scale"):
        pool = s[name].view(torch.uint8) if name in ("k", "v") else s[name]
        pool[to] = pool[source]
    s["moves"].fill_(-1)
    s["moves"][live] = live.to(torch.int32)
    s["moves"][source] = to.to(torch.int32)
    s["refs"][to] = s["refs"][source]
    s["refs"][source] = 0
    held = torch.arange(s["table"].shape[1], device="cuda") < ((s["lengths"] + P - 1) // P)[:, None]
    s["table"][held] = s["moves"][s["table"][held].long()]
    s["in_use"].fill_(n)


# --------------------------------------------------------------------------- one pass --

def books(s):
    """The cache and its books after a pass, codes as the bytes they are held in."""
    got = {name: s[name] for name in ("refs", "lengths", "table", "k_scale", "v_scale")}
    return got | {name: s[name].view(torch.int8) for name in ("k", "v")}


def run(state):
    s, case = state, state["case"]
    if case["op"] in ("fork", "compact"):
        s["ints"].copy_(s["saved"])
    if own:
        return run_own(s, case)
    if case["op"] == "logprobs":
        return plain_logprobs(s, case)
    if case["op"] == "attend":
        return plain_attend(s, case)
    plain_free(s, s["finished"], case["P"])
    if case["op"] == "fork":
        plain_fork(s, s["parents"], s["children"], case["P"])
        plain_extend(s, s["grow"], s["more"], case["P"])
        return books(s)
    for name in ("k", "v", "k_scale", "v_scale"):
        s["store_" + name][s["to"].long()] = s[name][s["from"].long()]
    plain_compact(s, case["P"])
    return kept(s)


def kept(s):
    store = {"store_" + name: s["store_" + name] if "scale" in name else s["store_" + name].view(torch.int8) for name in ("k", "v", "k_scale", "v_scale")}
    return books(s) | store | {"moves": s["moves"], "in_use": s["in_use"]}


def run_own(s, case):
    import causal_attention_score_gb300 as csa
    if case["op"] == "logprobs":
        csa.token_logprobs_forward(s["logprob"], s["entropy"], s["stats"], s["logits"], s["tokens"], scale=case["scale"],
                                   top_logprob=s["top_logprob"], top_token=s["top_token"])
        got = {name: s[name] for name in ("logprob", "entropy", "stats", "top_logprob", "top_token")}
        if case["grad"]:
            csa.token_logprobs_backward(s["dlogits"], s["logits"], s["tokens"], s["stats"], s["entropy"], d_logprob=s["d_logprob"],
                                        d_entropy=s["d_entropy"], d_top=s["d_top"], top_token=s["top_token"], scale=case["scale"])
            got["dlogits"] = s["dlogits"]
        return got
    if case["op"] == "attend":
        csa.cache_attention_shared_forward(s["out"], s["q"], s["cache"], s["batch"], s["groups"], s["shared"], workspace=s["workspace"])
        return s["out"]
    csa.kv_pages_free(s["pages"], s["finished"])
    if case["op"] == "fork":
        csa.kv_cache_fork(s["cache"], s["pages"], s["parents"], s["children"], workspace=s["workspace"])
        csa.kv_pages_extend(s["pages"], s["grow"], s["more"], workspace=s["workspace"])
        return books(s)
    csa.kv_cache_copy(s["store"], s["cache"], s["to"], s["from"])
    csa.kv_cache_compact(s["cache"], s["pages"], s["moves"], s["in_use"], workspace=s["workspace"])
    return kept(s)


# ------------------------------------------------------------------------- in 64 bits --

def exact_logprobs(s, case):
    """From softmax and its logarithm by their definitions, some rows at a time; the gradient by the chain rule through the
    matrix of derivatives of log p_i by x_j, delta_ij - p_j."""
    got = {name: [] for name in ("logprob", "entropy", "stats", "top_logprob", "top_token")} | ({"dlogits": []} if case["grad"] else {})
    V, K, scale = case["vocab"], case["top"], case["scale"]
    for i in range(0, case["rows"], 512):
        x = s["logits"][i: i + 512].double()
        tokens = s["tokens"][i: i + 512].long()
        n, live = x.shape[0], (tokens >= 0).double()[:, None]
        high = x.max(1, keepdim=True).values
        weight = torch.exp(scale * x - scale * high)
        p = weight / weight.sum(1, keepdim=True)
        log_p = scale * x - scale * high - torch.log(weight.sum(1, keepdim=True))
        surprise = torch.where(p > 0, -p * torch.where(p > 0, log_p, 0.0), 0.0)
        entropy = surprise.sum(1, keepdim=True)
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :K] if K else torch.zeros((n, 0), dtype=torch.long, device="cuda")
        at = tokens.clamp(min=0)[:, None]
        got["logprob"].append(torch.where(live > 0, torch.take_along_dim(log_p, at, 1), 0.0)[:, 0])
        got["entropy"].append((live * entropy)[:, 0])
        got["stats"].append(torch.where(live > 0, torch.cat([high, torch.log(weight.sum(1, keepdim=True))], 1), 0.0))
        got["top_logprob"].append(torch.where(live > 0, torch.take_along_dim(log_p, order, 1), 0.0))
        got["top_token"].append(torch.where(live > 0, order, -1).to(torch.int32))
        if case["grad"]:
            # dL = sum_i w_i d(log p_i) with w: the given token's and the alternatives' weights, and -d_entropy p_i (log p_i + 1)
            w = -s["d_entropy"][i: i + 512].double()[:, None] * torch.where(p > 0, p * (torch.where(p > 0, log_p, 0.0) + 1), 0.0)
            w.scatter_add_(1, at, s["d_logprob"][i: i + 512].double()[:, None])
            w.scatter_add_(1, order, s["d_top"][i: i + 512].double())
            got["dlogits"].append(live * scale * (w - p * w.sum(1, keepdim=True)))
    return {name: torch.cat(x) for name, x in got.items()}


def exact_attend(s, case):
    new, old, group, shared, _ = parts(case)
    P, D, G = case["P"], case["D"], case["Hq"] // case["Hkv"]
    out, at = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for i, (n, o) in enumerate(zip(new, old)):
        L = n + o + (shared[group[i]] if group[i] >= 0 else 0)
        slot = torch.arange(L, device="cuda")
        page = s["table"][i].long()[slot // P]
        for h in range(case["Hkv"]):
            k, v = (s[x][page, h, slot % P].double() * s[x + "_scale"][page, h].double()[:, None] for x in ("k", "v"))
            a = torch.einsum("ngd,td->gnt", s["q"][at: at + n, h * G: h * G + G].double(), k) / math.sqrt(D)
            a = a.masked_fill(slot[None, :] > (L - n + torch.arange(n, device="cuda"))[:, None], -math.inf)
            out[at: at + n, h * G: h * G + G] = torch.einsum("gnt,td->ngd", torch.softmax(a, -1), v)
        at += n
    return out


def exact_pages(s, case):
    """The books kept one entry at a time, on the host; then every page's bytes by where they came from."""
    P = case["P"]
    refs, lengths, table = s["saved"][: s["refs"].numel()].tolist(), sequences(case), s["table"].tolist()
    pages = len(refs)
    came, slots = list(range(pages)), [P] * pages  # the page whose first slots a page now holds, and how many of them

    def lowest():
        return refs.index(0)

    for i in s["finished"].tolist():
        for b in range(-(-lengths[i] // P)):
            refs[table[i][b]] -= 1
        lengths[i] = 0
    got = {}
    if case["op"] == "fork":
        for p, c in zip(s["parents"].tolist(), s["children"].tolist()):
            for b in range(lengths[p] // P):
                table[c][b] = table[p][b]
                refs[table[p][b]] += 1
            if lengths[p] % P:
                to = lowest()
                refs[to], table[c][lengths[p] // P] = 1, to
                came[to], slots[to] = table[p][lengths[p] // P], lengths[p] % P
            lengths[c] = lengths[p]
        for i, more in zip(s["grow"].tolist(), s["more"].tolist()):
            for b in range(-(-lengths[i] // P), -(-(lengths[i] + more) // P)):
                table[i][b] = lowest()
                refs[table[i][b]] = 1
            lengths[i] += more
    else:
        n = sum(r > 0 for r in refs)
        holes, move = (i for i in range(n) if refs[i] == 0), [-1] * pages
        for i in range(pages):
            if refs[i] > 0:
                move[i] = i if i < n else next(holes)
        for i in range(n, pages):
            if refs[i] > 0:
                refs[move[i]], refs[i], came[move[i]] = refs[i], 0, i
        for i, t in enumerate(lengths):
            for b in range(-(-t // P)):
                table[i][b] = move[table[i][b]]
        got = {"moves": torch.tensor(move, dtype=torch.int32), "in_use": torch.tensor([n], dtype=torch.int32)}
        for name in ("k", "v", "k_scale", "v_scale"):
            x = s[name] if "scale" in name else s[name].view(torch.int8)
            store = torch.empty_like(x[: s["to"].numel()])
            store[s["to"].long()] = x[s["from"].long()]
            got["store_" + name] = store.double() if "scale" in name else store
    came, keep = torch.tensor(came, device="cuda"), torch.arange(P, device="cuda") < torch.tensor(slots, device="cuda")[:, None]
    for name in ("k", "v"):
        x = s[name].view(torch.int8)
        got[name] = torch.where(keep[:, None, :, None], x[came], x)
        got[name + "_scale"] = s[name + "_scale"][came].double()
    return got | {"refs": torch.tensor(refs, dtype=torch.int32), "lengths": torch.tensor(lengths, dtype=torch.int32),
                  "table": torch.tensor(table, dtype=torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return exact_logprobs(s, case)
    if case["op"] == "attend":
        return exact_attend(s, case)
    return exact_pages(s, case)
