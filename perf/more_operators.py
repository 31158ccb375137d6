"""More operators of a paged KV cache: their plain forms, their inputs and their work.

Four operators of a decode loop over a paged cache (pools [layer][page][KV head][slot][d]):

* append   norms each query's and key's heads (root mean square, a weight per channel), rotates them by their
           positions, of which a token may have several (time, height, width of an image's patch), and stores k, v
* attend   attention of new rows over their sequences' cached tokens, of which groups of neighbouring sequences share
           a prefix (beams of one prompt, requests behind one instruction) that is read once for the group
* weigh    adds the rows' attention weights to each cached token's accumulated weight, per KV head
* evict    keeps each head's tokens of the largest accumulated weight, the first and the newest ones besides, and moves
           those behind the budget into the places of evicted ones

`own` False computes them in plain torch operations, True calls the framework.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one sequence, normed heads, a single position: latency alone counts
        dict(name="append-norm-1-token", op="append", dtype="bf16", layers=12, batch=1, rows=1, ctx=1024, heads=40,
             kv_heads=8, dim=128, page=16, rotary=128, axes=1, interleaved=False, norm=True, ragged=False),
        # chunks of four prompts with images: normed heads and three position axes, from a fused projection's output
        dict(name="append-norm-axes-chunk", op="append", dtype="bf16", layers=2, batch=4, rows=2048, ctx=4096, heads=40,
             kv_heads=8, dim=128, page=64, rotary=128, axes=3, interleaved=False, norm=True, ragged=True),
        # a few new tokens of 48 sequences, three axes over half of the channels, weights in 32 bits
        dict(name="append-axes-48", op="append", dtype="fp16", layers=2, batch=48, rows=5, ctx=900, heads=64,
             kv_heads=8, dim=64, page=32, rotary=32, axes=3, interleaved=True, norm=True, ragged=True),
        # four beams of one prompt, one new token each: latency counts
        dict(name="attend-prefix-4-beams", op="attend", dtype="fp16", groups=1, per=4, prefix=1000, tail=60, rows=1,
             heads=12, kv_heads=12, dim=64, page=16, tree=False, ragged=False),
        # 64 requests behind one long instruction, one new token each: the bytes of their own tokens count
        dict(name="attend-prefix-64", op="attend", dtype="bf16", groups=1, per=64, prefix=8192, tail=700, rows=1,
             heads=40, kv_heads=8, dim=128, page=64, tree=False, ragged=True),
        # six documents with up to eight requests each, small trees of drafted tokens: the prefix's products count
        dict(name="attend-prefix-groups", op="attend", dtype="bf16", groups=6, per=8, prefix=6000, tail=300, rows=12,
             heads=64, kv_heads=8, dim=64, page=32, tree=True, ragged=True),
        # the weights that one token of one small sequence gives
        dict(name="weigh-1-token", op="weigh", dtype="fp16", batch=1, rows=1, ctx=2048, heads=12, kv_heads=12, dim=64,
             page=16, ragged=False),
        # one token each of 32 long sequences of unequal lengths: the bytes of the keys count
        dict(name="weigh-32", op="weigh", dtype="bf16", batch=32, rows=1, ctx=16384, heads=64, kv_heads=8, dim=64,
             page=64, ragged=True),
        # the last 64 rows of four prompts, whose weights rank the prompts' tokens: the matrix products count
        dict(name="weigh-window-64", op="weigh", dtype="bf16", batch=4, rows=64, ctx=12000, heads=40, kv_heads=8,
             dim=128, page=64, ragged=False),
        # one sequence of a small model comes down to its budget: latency counts
        dict(name="evict-1", op="evict", dtype="fp16", layers=12, batch=1, length=304, high=256, low=256, protect=32,
             first=4, heads=12, kv_heads=12, dim=64, page=16, sorted=True),
        # decoding at the budget: one token of every head of every layer goes, one sequence of four is still below it
        dict(name="evict-decode-8", op="evict", dtype="fp16", layers=64, batch=8, length=2049, high=2048, low=2048,
             protect=128, first=0, heads=40, kv_heads=8, dim=128, page=64, sorted=False),
        # prompts of four sequences come down to one of two budgets
        dict(name="evict-prompt-4", op="evict", dtype="bf16", layers=16, batch=4, length=8192, high=2048, low=1024,
             protect=128, first=64, heads=40, kv_heads=8, dim=128, page=64, sorted=True),
    ]


def _log(rng, low, high):
    """A whole number between low and high, evenly spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


SHAPES = [(12, 12, 64), (40, 8, 128), (64, 8, 64), (16, 16, 128), (7, 1, 64), (20, 4, 128)]


def draw(rng):
    most = max(work(c)["flops"] for c in listed()), max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["append", "attend", "weigh", "evict"])
        heads, kv_heads, dim = rng.choice(SHAPES)
        case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), heads=heads, kv_heads=kv_heads, dim=dim,
                    page=rng.choice([16, 32, 64, 128]))
        if op == "append":
            case.update(layers=rng.randint(1, 12), batch=_log(rng, 1, 64), rows=_log(rng, 1, 2048),
                        ctx=_log(rng, 1, 4096), rotary=rng.choice([dim, dim // 2]), axes=rng.choice([1, 2, 3, 4]),
                        interleaved=rng.random() < 0.3, norm=rng.random() < 0.8, ragged=rng.random() < 0.5)
        elif op == "attend":
            tree = rng.random() < 0.4
            case.update(groups=_log(rng, 1, 8), per=_log(rng, 1, 64), prefix=_log(rng, 16, 16384),
                        tail=_log(rng, 1, 2000), rows=_log(rng, 2, 40) if tree else _log(rng, 1, 64), tree=tree,
                        ragged=rng.random() < 0.6)
        elif op == "weigh":
            case.update(batch=_log(rng, 1, 48), rows=_log(rng, 1, 700), ctx=_log(rng, 1, 16384),
                        ragged=rng.random() < 0.5)
        else:
            length = _log(rng, 2, 16384)
            high = max(1, int(length * rng.uniform(0.1, 1.1)))
            case.update(layers=_log(rng, 1, 64), batch=_log(rng, 1, 16), length=length, high=high,
                        low=max(1, high // rng.choice([1, 2])), protect=_log(rng, 1, max(2, high // 4)),
                        first=rng.choice([0, 1, 4, min(64, high // 2)]), sorted=rng.random() < 0.5)
        w = work(case)
        if w["flops"] <= most[0] and w["bytes"] <= most[1] and _footprint(case) <= 20e9:
            return case


def _footprint(case):
    """Bytes that the plain form holds at most, about."""
    H, d = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        return 6.0 * _tokens(case) * case["layers"] * H * d
    if case["op"] == "evict":
        units = case["layers"] * case["batch"] * H
        return units * case["length"] * (60 + 10 * d)
    if case["op"] == "attend":
        n, g = case["groups"] * case["per"], case["heads"]
        return n * case["rows"] * g * (case["prefix"] + case["tail"]) * 12 + n * (case["prefix"] + case["tail"]) * H * d * 12
    return case["batch"] * (case["ctx"] + case["rows"]) * (case["rows"] * case["heads"] * 12 + H * d * 12)


def _lens(case):
    """Cached tokens and new rows of each sequence: all alike, or unequal (a sequence without new rows among them)."""
    ctx, new = [], []
    if case["op"] == "attend":
        for b, (g, i) in enumerate(_members(case)):
            f = (b * 0.6180339887) % 1.0
            ctx.append(_prefixes(case)[g] + (int(round(case["tail"] * (1 - 0.8 * f))) if case["ragged"] else case["tail"]))
            new.append(max(1, int(round(case["rows"] * (1 - 0.5 * f)))) if case["ragged"] else case["rows"])
        return ctx, new
    for b in range(case["batch"]):
        f = (b * 0.6180339887) % 1.0
        ctx.append(int(round(case["ctx"] * (1 - 0.6 * f))) if case["ragged"] else case["ctx"])
        new.append(max(1, int(round(case["rows"] * (1 - 0.7 * f)))) if case["ragged"] else case["rows"])
    if case["ragged"] and case["batch"] >= 4:
        new[2] = 0
    return ctx, new


def _sizes(case):
    """Sequences of each group: all alike, or unequal (a group of one among them)."""
    if not case["ragged"] or case["groups"] == 1:
        return [case["per"]] * case["groups"]
    n = [max(1, int(round(case["per"] * (1 - 0.6 * ((g * 0.6180339887) % 1.0))))) for g in range(case["groups"])]
    return n[:-1] + [1]


def _prefixes(case):
    return [int(round(case["prefix"] * (1 - 0.4 * ((g * 0.6180339887) % 1.0)))) if case["ragged"] else case["prefix"]
            for g in range(case["groups"])]


def _members(case):
    return [(g, i) for g, n in enumerate(_sizes(case)) for i in range(n)]


def _ancestors(case, b, count):
    """Row i's visible drafted tokens in sequence b's tree, as a whole number of bits: its ancestors and itself."""
    r, bits = random.Random(1000 * case["rows"] + b), []
    for i in range(count):
        p = max(-1, i - 1 - r.randrange(0, 6))
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return bits


def _evicted(case):
    """Length, budget and new length of each sequence."""
    out = []
    for b in range(case["batch"]):
        n = case["length"] if b % 4 != 3 else max(1, case["length"] - 1)
        keep = case["high"] if b % 2 == 0 else case["low"]
        out.append((n, keep, min(n, keep)))
    return out


def _tokens(case):
    if case["op"] == "evict":
        return sum(n for n, _, _ in _evicted(case))
    ctx, new = _lens(case)
    return sum(ctx) + sum(new)


def _sections(case):
    """The axis of each channel pair: two whole shares and the rest in turns, so that all orders occur."""
    half, axes = case["rotary"] // 2, case["axes"]
    return [min(axes - 1, i * axes // half) if i < half // 2 else i % axes for i in range(half)]


def work(case):
    op, Hq, H, d = case["op"], case["heads"], case["kv_heads"], case["dim"]
    if op == "append":
        n = sum(_lens(case)[1])
        moved = n * (2 * (Hq + 2 * H) * d * 2 + 4 * case["axes"]) + case["rotary"] * 4 + (4 * d if case["norm"] else 0)
        return {"bytes": moved, "flops": n * (Hq + H) * ((4 * d if case["norm"] else 0) + 3 * case["rotary"])}
    if op == "attend":
        ctx, new = _lens(case)
        pairs = words = 0
        read = sum(_prefixes(case))
        for b, (g, _) in enumerate(_members(case)):
            t = new[b]
            drafts = sum(x.bit_count() for x in _ancestors(case, b, t)) if case["tree"] else t * (t + 1) // 2
            pairs += ctx[b] * t + drafts
            read += ctx[b] - _prefixes(case)[g] + t
            words += t * 4 * -(-case["rows"] // 32) if case["tree"] else 0
        return {"bytes": read * 4 * H * d + sum(new) * Hq * (4 * d + 4) + words, "flops": 4 * pairs * Hq * d}
    if op == "weigh":
        pairs = read = rows = 0
        for a, t in zip(*_lens(case)):
            pairs += a * t + t * (t + 1) // 2
            read += a + t if t else 0
            rows += t
        return {"bytes": read * H * (2 * d + 8) + rows * Hq * (2 * d + 4) + rows * (4 + 4 * H), "flops": 2 * pairs * Hq * d}
    moved = kept = seen = 0
    for n, keep, N in _evicted(case):
        first, newest = min(case["first"], N), min(case["protect"], n)
        rest = max(0, n - first - newest)
        share = max(0, N - first - newest) / rest if rest else 0.0  # of the others that stay
        behind = n - N
        late = min(newest, behind) if case["sorted"] else newest * behind / n
        moved += min(behind, late + max(0, behind - late) * share) if behind else 0
        kept += N
        seen += n
    units = case["layers"] * H
    return {"bytes": units * (8 * seen + 8 * kept + moved * 8 * d), "flops": units * seen}


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=dt)  # noqa: E731
    state = {"case": case, "op": op}
    L = case.get("layers", 2)
    Hq, H, d, ps = case["heads"], case["kv_heads"], case["dim"], case["page"]
    if op == "evict":
        spans = _evicted(case)
        ctx, new = [n for n, _, _ in spans], [0] * len(spans)
    else:
        ctx, new = _lens(case)
    B = len(ctx)
    blocks = [-(-(a + b) // ps) for a, b in zip(ctx, new)]
    pages = sum(blocks) + 3
    state["k_pages"], state["v_pages"] = randn(L, pages, H, ps, d), randn(L, pages, H, ps, d)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    if op == "attend":
        # a group's sequences name its first one's pages of the prefix; a part-filled last page is each one's own copy
        b = 0
        state["prefixes"], state["sizes"] = _prefixes(case), _sizes(case)
        for P, n in zip(state["prefixes"], state["sizes"]):
            full, fill = P // ps, P % ps
            for i in range(b + 1, b + n):
                table[i, :full] = table[b, :full]
                if fill:
                    for pool in (state["k_pages"], state["v_pages"]):
                        pool[:, table[i, full].long(), :, :fill] = pool[:, table[b, full].long(), :, :fill]
            b += n
        state["group_start"] = ints([sum(state["sizes"][:i]) for i in range(case["groups"] + 1)])
        state["prefix_len"] = ints(state["prefixes"])
    state["table"], state["ctx"] = table, ints(ctx)
    starts = [sum(new[:b]) for b in range(B + 1)]
    state["q_start"], state["live"], state["starts"] = ints(starts), starts[-1], starts
    state["lens"] = (ctx, new)
    n = starts[-1] + (2 if case.get("ragged") else 0)  # a padded batch: rows behind the last sequence
    if op == "append":
        qkv = randn(n, Hq + 2 * H, d) * (0.1 + 8 * torch.rand(n, 1, 1, generator=g, device="cuda").to(dt))
        state["q"], state["k"], state["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        state["q_out"] = torch.zeros(n, Hq, d, device="cuda", dtype=dt)
        state["pos"] = torch.randint(0, 40000, (n, case["axes"]), generator=g, device="cuda", dtype=torch.int32)
        r = case["rotary"]
        state["inv_freq"] = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()
        state["axis"] = ints(_sections(case))
        weight = lambda: 1 + 0.2 * torch.randn(d, generator=g, device="cuda")  # noqa: E731
        wt = torch.float32 if case["axes"] % 2 == 1 and case["interleaved"] else dt
        state["q_norm"], state["k_norm"] = (weight().to(wt), weight().to(wt)) if case["norm"] else (None, None)
    if op in ("attend", "weigh"):
        state["q"] = randn(n, Hq, d)
        state["mask"] = None
    if op == "attend":
        state["out"] = torch.zeros(n, Hq, d, device="cuda", dtype=dt)
        state["lse"] = torch.zeros(n, Hq, device="cuda")
        if case["tree"]:
            words = -(-max(new) // 32)
            rows = [x for b, t in enumerate(new) for x in _ancestors(case, b, t)] + [0] * (n - sum(new))
            cut = [[(x >> 32 * w) & 0xFFFFFFFF for w in range(words)] for x in rows]
            state["mask"] = ints([[w - (1 << 32) if w >> 31 else w for w in x] for x in cut])
    if op == "weigh":
        cap = max(a + t for a, t in zip(ctx, new)) + 5
        state["lse"] = _row_sums(state)
        state["mass"] = torch.rand(B, H, cap, generator=g, device="cuda").pow_(6)
        state["mass_out"] = torch.zeros_like(state["mass"])
        state["pos_map"] = torch.arange(cap, device="cuda", dtype=torch.int32).expand(B, H, cap).contiguous()
        state["positions"] = ints([a + 100 + i for a, t in zip(ctx, new) for i in range(t)] + [0] * (n - sum(new)))
        state["decay"], state["gain"] = 0.9, 0.1 * H / Hq
    if op == "evict":
        cap = max(ctx)
        state["mass"] = torch.rand(L, B, H, cap, generator=g, device="cuda").pow_(6)
        where = torch.arange(cap, device="cuda", dtype=torch.int32).expand(L, B, H, cap)
        if case["sorted"]:
            state["pos_map"] = where.contiguous()
        else:
            # heads that have been at their budget for long: the positions lie in no order, gaps between them
            far = torch.rand(L, B, H, cap, generator=g, device="cuda").argsort(3).to(torch.int32)
            state["pos_map"] = far * 3 + 1
            del far
        state["keep"] = ints([k for _, k, _ in spans])
        state["first"] = ints([case["first"]] * B) if case["first"] else None
        state["mass_out"], state["pos_out"] = torch.zeros_like(state["mass"]), torch.zeros_like(state["pos_map"])
        state["new_len"] = torch.zeros_like(state["ctx"])
        state["spans"] = spans
    if own:
        import confidence_gated_kv_logits_gb300 as pkg
        kv = state["kv"] = pkg.PagedKV(state["k_pages"], state["v_pages"], Hq)
        if op != "evict":
            state["batch"] = kv.batch(state["table"], state["ctx"], state["q_start"], state.get("mask"))
        if op == "attend":
            state["prefix"] = kv.prefix(state["group_start"], state["prefix_len"], n)
    return state


def _keys(s, b, n):
    """Keys of sequence b's first n tokens in layer 1, [KV head, token, d]."""
    at = torch.arange(n, device="cuda")
    ps = s["case"]["page"]
    return s["k_pages"][1, s["table"][b].long()[at // ps], :, at % ps].transpose(0, 1)


def _row_sums(s):
    """ln sum exp of each row's scores: what the attention before gave."""
    case = s["case"]
    Hq, H, d = case["heads"], case["kv_heads"], case["dim"]
    lse = torch.zeros(s["q"].shape[0], Hq, device="cuda")
    for b, (a, t) in enumerate(zip(*s["lens"])):
        if t:
            r = slice(s["starts"][b], s["starts"][b] + t)
            keys = _keys(s, b, a + t).float()
            hidden = torch.ones(t, a + t, dtype=torch.bool, device="cuda").tril_(a).logical_not_()
            for h in range(H):
                q = s["q"][r, h * (Hq // H):(h + 1) * (Hq // H)].float()
                z = (q @ keys[h].T * d ** -0.5).masked_fill_(hidden[:, None], -math.inf)
                lse[r, h * (Hq // H):(h + 1) * (Hq // H)] = torch.logsumexp(z, 2)
    return lse


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return PLAIN[state["op"]](state)


def _run_own(s):
    op, case, kv = s["op"], s["case"], s["kv"]
    if op == "append":
        kv.append(case["layers"] - 1, s["batch"], s["k"], s["v"], q=s["q"], q_out=s["q_out"], positions=s["pos"],
                  inv_freq=s["inv_freq"], interleaved=case["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                  eps=EPS, axis=s["axis"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    if op == "attend":
        kv.attend(1, s["batch"], s["q"], s["out"], lse=s["lse"], prefix=s["prefix"])
        return s["out"], s["lse"]
    if op == "weigh":
        kv.weigh(1, s["batch"], s["q"], s["lse"], s["mass"], s["mass_out"], s["pos_map"], positions=s["positions"],
                 decay=s["decay"], gain=s["gain"])
        return s["mass_out"], s["pos_map"]
    kv.evict(s["table"], s["ctx"], s["mass"], s["pos_map"], s["keep"], s["mass_out"], s["pos_out"], s["new_len"],
             protect=case["protect"], first=s["first"])
    return s["k_pages"], s["v_pages"], s["mass_out"], s["pos_out"], s["new_len"]


def _plain_append(s):
    case, n, r = s["case"], s["live"], s["case"]["rotary"]
    rows = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), rows, right=True)
    place = s["ctx"].long()[seq] + rows - s["q_start"].long()[seq]
    page, slot = s["table"].long()[seq, place // case["page"]], place % case["page"]
    angle = s["pos"][:n].double()[:, s["axis"].long()] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def normed(x, w):
        x = x[:n].float()
        return x if w is None else x * (x.square().mean(2, keepdim=True) + EPS).rsqrt() * w.float()

    def rotated(x):
        y = x.clone()
        even = torch.arange(0, r, 2) if case["interleaved"] else torch.arange(r // 2)
        odd = even + (1 if case["interleaved"] else r // 2)
        a, b = x[..., even], x[..., odd]
        y[..., even], y[..., odd] = a * cos - b * sin, b * cos + a * sin
        return y

    layer = case["layers"] - 1
    s["q_out"][:n] = rotated(normed(s["q"], s["q_norm"])).to(s["q_out"].dtype)
    s["k_pages"][layer, page, :, slot] = rotated(normed(s["k"], s["k_norm"])).to(s["k_pages"].dtype)
    s["v_pages"][layer, page, :, slot] = s["v"][:n]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _plain_attend(s):
    """Group by group: scores of all its rows over the prefix and of each sequence's rows over its own tokens, one softmax."""
    case = s["case"]
    Hq, H, d, ps = case["heads"], case["kv_heads"], case["dim"], case["page"]
    r, (ctx, new), b0 = Hq // H, s["lens"], 0
    for P, n in zip(s["prefixes"], s["sizes"]):
        T, S = max(new[b0:b0 + n]), max(ctx[b] - P + new[b] for b in range(b0, b0 + n))
        t, j = torch.arange(T, device="cuda"), torch.arange(S, device="cuda")
        start, own_ctx = s["q_start"].long()[b0:b0 + n + 1], s["ctx"].long()[b0:b0 + n] - P
        count = start[1:] - start[:-1]
        rows = (start[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
        q = s["q"][rows].float().view(n, T, H, r, d).permute(0, 2, 1, 3, 4).reshape(n, H, T * r, d)
        at = torch.arange(P, device="cuda")
        first = lambda pool: pool[1, s["table"][b0].long()[at // ps], :, at % ps].float().transpose(0, 1)  # noqa: E731
        place = P + j
        page = s["table"][b0:b0 + n].long()[:, (place // ps).clamp(max=s["table"].shape[1] - 1)].clamp(min=0)
        rest = lambda pool: pool[1, page, :, place % ps].float().transpose(1, 2)  # noqa: E731  [n, H, S, d]
        near = q @ rest(s["k_pages"]).transpose(2, 3)
        x = j - own_ctx[:, None]  # which new row of the sequence
        if s["mask"] is None:
            seen = x[:, None, :] <= t[:, None]
        else:
            word = s["mask"][rows].gather(2, (x.clamp(0, T - 1) // 32)[:, None].expand(n, T, S))
            seen = (x < 0)[:, None, :] | ((word >> (x.clamp(min=0) % 32)[:, None].int() & 1) == 1)
        seen = seen & (x < count[:, None])[:, None, :]
        near.view(n, H, T, r, S).masked_fill_(~seen[:, None, :, None, :], -math.inf)
        scores = torch.cat([q @ first(s["k_pages"]).transpose(1, 2), near], 3) / math.sqrt(d)
        del near
        top = scores.amax(3, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p = (scores - top).exp_()
        del scores
        total = p.sum(3, keepdim=True)
        out = p[..., :P] @ first(s["v_pages"]) + p[..., P:] @ rest(s["v_pages"])
        out = (out / total).view(n, H, T, r, d)
        lse = (top + total.log()).view(n, H, T, r)
        i = torch.arange(s["starts"][b0], s["starts"][b0 + n], device="cuda")
        b = torch.searchsorted(start[1:], i, right=True)
        s["out"][i] = out[b, :, i - start[b]].reshape(-1, Hq, d).to(s["out"].dtype)
        s["lse"][i] = lse[b, :, i - start[b]].reshape(-1, Hq)
        b0 += n
    return s["out"], s["lse"]


def _plain_weigh(s):
    case = s["case"]
    Hq, H, d, ps, B = case["heads"], case["kv_heads"], case["dim"], case["page"], case["batch"]
    r, T, n = Hq // H, max(s["lens"][1]), s["live"]
    ctx, start = s["ctx"].long(), s["q_start"].long()
    count = start[1:] - start[:-1]
    t = torch.arange(T, device="cuda")
    rows = (start[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, T, H, r, d).permute(0, 2, 1, 3, 4).reshape(B, H, T * r, d)
    keys = s["k_pages"][1][s["table"].clamp(min=0).long()].permute(0, 2, 1, 3, 4).reshape(B, H, -1, d).float()
    p = (q @ keys.transpose(2, 3)) * d ** -0.5
    S = p.shape[3]
    p = p.view(B, H, T, r, S)
    p -= s["lse"][rows].view(B, T, H, r).permute(0, 2, 1, 3)[..., None]
    p.exp_()
    j = torch.arange(S, device="cuda")
    x = j - ctx[:, None]
    seen = (x[:, None, :] <= t[:, None]) & (t[:, None] < count[:, None, None])
    p.masked_fill_(~seen[:, None, :, None, :], 0.0)
    given = p.sum((2, 3))
    cap = s["mass"].shape[2]
    given, x = torch.nn.functional.pad(given, (0, max(0, cap - S)))[..., :cap], torch.arange(cap, device="cuda") - ctx[:, None]
    old = torch.where((x < 0)[:, None], s["decay"] * s["mass"], 0.0)
    live = ((x < count[:, None]) & (count[:, None] > 0))[:, None]
    s["mass_out"].copy_(torch.where(live, old + s["gain"] * given, s["mass_out"]))
    i = torch.arange(n, device="cuda")
    b = torch.searchsorted(start[1:], i, right=True)
    s["pos_map"][b, :, ctx[b] + i - start[b]] = s["positions"][:n, None].expand(n, H)
    return s["mass_out"], s["pos_map"]


def _plain_evict(s):
    case = s["case"]
    mass, pos, ps = s["mass"], s["pos_map"], case["page"]
    L, B, H, cap = mass.shape
    place = torch.arange(cap, device="cuda")
    n = s["ctx"].long()[:, None, None]
    N = torch.minimum(s["keep"].long()[:, None, None], n)
    live = (place < n)[:, 0]
    newest = torch.where(live[None, :, None], pos, -1).amax(3, keepdim=True)
    rank = mass.double()
    rank = torch.where(pos > newest - case["protect"], 1e200, rank)
    if s["first"] is not None:
        rank = torch.where((place < s["first"].long()[:, None])[None, :, None], 1e300, rank)
    rank = torch.where(live[None, :, None], rank, -math.inf)
    by = rank.sort(dim=3, descending=True, stable=True).indices
    kept = torch.zeros(L, B, H, cap, dtype=torch.bool, device="cuda")
    kept.scatter_(3, by, (place < N).expand(B, 1, cap)[None].expand(L, B, H, cap))
    inside = (place < N)[None].expand(L, B, H, cap)
    hole, mover = (~kept & inside).nonzero(), (kept & ~inside).nonzero()
    source = place.expand(L, B, H, cap).clone()
    source[tuple(hole.T)] = mover[:, 3]
    s["mass_out"].copy_(torch.where(inside, mass.gather(3, source), s["mass_out"]))
    s["pos_out"].copy_(torch.where(inside, pos.gather(3, source), s["pos_out"]))
    table = s["table"].long()
    at = lambda x: (x[:, 0], table[x[:, 1], x[:, 3] // ps], x[:, 2], x[:, 3] % ps)  # noqa: E731
    for pool in (s["k_pages"], s["v_pages"]):
        pool[at(hole)] = pool[at(mover)]
    s["new_len"].copy_(torch.minimum(s["ctx"], s["keep"]))
    return s["k_pages"], s["v_pages"], s["mass_out"], s["pos_out"], s["new_len"]


PLAIN = {"append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh, "evict": _plain_evict}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "evict":
        return None  # weights are compared and moved as they are: no computed numbers
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "weigh": _exact_weigh}[case["op"]](case, s)


def _exact_append(case, s):
    """Norm by the vector's length, rotation as a complex product, sequence by sequence."""
    r, ps, d, layer = case["rotary"], case["page"], case["dim"], case["layers"] - 1
    q_out, ks, vs = s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()
    axis, row = s["axis"].cpu().tolist(), 0

    def turned(x, weight, phase):
        x = x.double()
        if weight is not None:
            x = x * weight.double() * math.sqrt(d) / torch.sqrt(torch.linalg.vector_norm(x, dim=2, keepdim=True) ** 2 + d * EPS)
        even = list(range(0, r, 2)) if case["interleaved"] else list(range(r // 2))
        odd = [e + (1 if case["interleaved"] else r // 2) for e in even]
        z = torch.complex(x[:, :, even], x[:, :, odd]) * phase[:, None]
        y = x.clone()
        y[:, :, even], y[:, :, odd] = z.real, z.imag
        return y

    for b, (a, t) in enumerate(zip(*s["lens"])):
        if t:
            at = slice(row, row + t)
            angle = torch.stack([s["pos"][at, axis[i]].double() * s["inv_freq"][i].double() for i in range(r // 2)], 1)
            phase = torch.polar(torch.ones_like(angle), angle)
            q_out[at] = turned(s["q"][at], s["q_norm"], phase)
            place = torch.arange(a, a + t, device="cuda")
            page = s["table"][b].long()[place // ps]
            ks[layer, page, :, place % ps] = turned(s["k"][at], s["k_norm"], phase)
            vs[layer, page, :, place % ps] = s["v"][at].double()
            row += t
    return q_out, ks, vs


def _exact_attend(case, s):
    """Every sequence over its own pages, as if nothing were shared."""
    ctx, new = s["lens"]
    if sum(a * t for a, t in zip(ctx, new)) * case["heads"] * case["dim"] > 4e12 or len(ctx) * case["heads"] > 8000:
        return None
    out, lse = s["out"].double(), s["lse"].double()
    g, d, row = case["heads"] // case["kv_heads"], case["dim"], 0
    for b, t in enumerate(new):
        n = ctx[b] + t
        seen = torch.ones(t, n, dtype=torch.bool)
        if case["tree"]:
            seen[:, ctx[b]:] = torch.tensor([[bool(x >> i & 1) for i in range(t)] for x in _ancestors(case, b, t)])
        else:
            seen[:, ctx[b]:] = torch.tril(torch.ones(t, t, dtype=torch.bool))
        hide = torch.zeros(t, n, dtype=torch.float64).masked_fill_(~seen, -math.inf).cuda()
        pages = s["table"][b, :-(-n // case["page"])].long()
        for h in range(case["heads"]):
            k = s["k_pages"][1, pages, h // g].reshape(-1, d)[:n].double()
            v = s["v_pages"][1, pages, h // g].reshape(-1, d)[:n].double()
            z = s["q"][row:row + t, h].double() @ k.T * d ** -0.5 + hide
            norm = torch.logsumexp(z, 1)
            out[row:row + t, h] = torch.exp(z - norm[:, None]) @ v
            lse[row:row + t, h] = norm
        row += t
    return out, lse


def _exact_weigh(case, s):
    """Head by head; the new tokens' own weights start from nothing."""
    g, d, row = case["heads"] // case["kv_heads"], case["dim"], 0
    ctx, new = s["lens"]
    if sum((a + t) * t for a, t in zip(ctx, new)) * case["heads"] * d > 4e12 or len(ctx) * case["heads"] > 8000:
        return None
    mass, pos = s["mass_out"].double(), s["pos_map"].clone()
    for b, t in enumerate(new):
        if t:
            n = ctx[b] + t
            pages = s["table"][b, :-(-n // case["page"])].long()
            seen = torch.tril(torch.ones(t, n, dtype=torch.float64), diagonal=ctx[b]).cuda()
            for h in range(case["kv_heads"]):
                k = s["k_pages"][1, pages, h].reshape(-1, d)[:n].double()
                total = torch.zeros(n, dtype=torch.float64, device="cuda")
                for i in range(h * g, h * g + g):
                    z = s["q"][row:row + t, i].double() @ k.T * d ** -0.5 - s["lse"][row:row + t, i].double()[:, None]
                    total += (torch.exp(z) * seen).sum(0)
                before = torch.cat([s["mass"][b, h, :ctx[b]].double() * s["decay"],
                                    torch.zeros(t, dtype=torch.float64, device="cuda")])
                mass[b, h, :n] = before + s["gain"] * total
                pos[b, h, ctx[b]:n] = s["positions"][row:row + t]
            row += t
    return mass, pos
