"""Operators of a paged KV cache and of beam search: their plain forms, their inputs and their work.

Five operators of a decode loop over a paged cache (pools [layer][page][KV head][slot][d]):

* append   rotates q and k by their positions (rotary embedding) and stores k, v in the cache's pages
* attend   attention of a ragged batch of new rows over their sequence's cached tokens and, below a
           mask of ancestor bits (a tree of drafted tokens) or causally, over the new rows themselves
* commit   moves the rows of an accepted path of drafted tokens behind the cached tokens, in every layer
* select   the best k of beams x vocabulary by summed log-probability, with parents and tokens
* fork     reorders the beams' page tables by their parents and copies each parent's last, part-filled page

`own` False computes them in plain torch operations, True calls the framework.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one sequence of a small model takes one token: latency alone counts
        dict(name="append-1-token", op="append", dtype="fp16", layers=12, batch=1, rows=1, ctx=1024, heads=12,
             kv_heads=12, dim=64, page=16, rotary=64, interleaved=False, ragged=False),
        # a chunk of four prompts of unequal lengths enters a GQA cache from a fused projection's output
        dict(name="append-prompt-chunk", op="append", dtype="bf16", layers=2, batch=4, rows=2048, ctx=4096, heads=40,
             kv_heads=8, dim=128, page=64, rotary=128, interleaved=False, ragged=True),
        # plain decoding of one sequence of a small multi-head model, one new token
        dict(name="attend-decode-1", op="attend", dtype="fp16", batch=1, rows=1, ctx=2048, heads=12, kv_heads=12,
             dim=64, page=16, tree=False, ragged=False),
        # decoding of a batch of long sequences of unequal lengths, bandwidth counts
        dict(name="attend-decode-32", op="attend", dtype="bf16", batch=32, rows=1, ctx=16384, heads=64, kv_heads=8,
             dim=64, page=64, tree=False, ragged=True),
        # a tree of 64 drafted tokens per sequence over 8k cached tokens
        dict(name="attend-tree-64", op="attend", dtype="fp16", batch=8, rows=64, ctx=8192, heads=40, kv_heads=8,
             dim=128, page=32, tree=True, ragged=False),
        # a small tree over a long cache of one sequence: few rows, a long axis
        dict(name="attend-tree-13-long", op="attend", dtype="bf16", batch=1, rows=13, ctx=32768, heads=40, kv_heads=8,
             dim=128, page=16, tree=True, ragged=False),
        # a prompt's chunk over what is cached of it already: the matrix products count
        dict(name="attend-prompt-chunk", op="attend", dtype="bf16", batch=2, rows=2048, ctx=6144, heads=40, kv_heads=8,
             dim=128, page=128, tree=False, ragged=False),
        # the accepted path of one small tree
        dict(name="commit-1", op="commit", dtype="fp16", layers=12, batch=1, rows=16, accept=5, ctx=1000, heads=12,
             kv_heads=12, dim=64, page=16),
        # the accepted paths of 32 sequences' trees in every layer of a deep model
        dict(name="commit-32", op="commit", dtype="bf16", layers=64, batch=32, rows=48, accept=9, ctx=333, heads=40,
             kv_heads=8, dim=128, page=32),
        # four beams of one sequence over a small vocabulary
        dict(name="select-4-beams", op="select", dtype="fp32", batch=1, beams=4, vocab=50257, keep=8, finished=False),
        # eight beams of 16 sequences over a large vocabulary, some of them at their end
        dict(name="select-8-beams", op="select", dtype="bf16", batch=16, beams=8, vocab=201088, keep=16, finished=True),
        # the beams' tables and part-filled pages of eight sequences in every layer of a deep model
        dict(name="fork-32", op="fork", dtype="fp16", layers=64, batch=8, beams=4, ctx=1069, heads=40, kv_heads=8,
             dim=128, page=64),
    ]


def _log(rng, low, high):
    """A whole number between low and high, evenly spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


SHAPES = [(12, 12, 64), (40, 8, 128), (64, 8, 64), (16, 16, 128), (7, 1, 64), (24, 3, 128)]


def draw(rng):
    most = max(work(c)["flops"] for c in listed()), max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["append", "attend", "attend", "attend", "commit", "select", "fork"])
        heads, kv_heads, dim = rng.choice(SHAPES)
        case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), heads=heads, kv_heads=kv_heads, dim=dim,
                    page=rng.choice([16, 32, 64, 128]))
        if op == "append":
            case.update(layers=rng.randint(1, 12), batch=_log(rng, 1, 64), rows=_log(rng, 1, 2048),
                        ctx=_log(rng, 1, 4096), rotary=rng.choice([dim, dim // 2]),
                        interleaved=rng.random() < 0.3, ragged=rng.random() < 0.5)
        elif op == "attend":
            tree = rng.random() < 0.5
            case.update(batch=_log(rng, 1, 48), rows=_log(rng, 2, 200) if tree else _log(rng, 1, 2048),
                        ctx=_log(rng, 1, 32768), tree=tree, ragged=rng.random() < 0.5)
        elif op == "commit":
            rows = _log(rng, 4, 64)
            case.update(layers=_log(rng, 1, 64), batch=_log(rng, 1, 32), rows=rows, accept=rng.randint(1, min(rows, 10)),
                        ctx=_log(rng, 1, 400))
        elif op == "select":
            beams = _log(rng, 1, 16)
            case = dict(op=op, dtype=rng.choice(["fp32", "fp16", "bf16"]), batch=_log(rng, 1, 16), beams=beams,
                        vocab=_log(rng, 500, 201088), keep=rng.choice([beams, 2 * beams]), finished=rng.random() < 0.5)
        else:
            case.update(layers=_log(rng, 1, 64), batch=_log(rng, 1, 8), beams=_log(rng, 1, 8), ctx=_log(rng, 1, 1500))
        w = work(case)
        if w["flops"] <= most[0] and w["bytes"] <= most[1] and _footprint(case) <= 24e9:
            return case


def _footprint(case):
    """Bytes that the plain form holds at most, about."""
    if case["op"] == "attend":
        lens, new = _lens(case)
        long = max(a + b for a, b in zip(lens, new)) + 2 * case["page"]
        return case["batch"] * long * (16 * max(new) * case["heads"] + 24 * max(new) + 16 * case["kv_heads"] * case["dim"])
    if case["op"] == "select":
        return 40.0 * case["batch"] * case["beams"] * case["vocab"]
    return 4 * _pages(case) * case["layers"] * case["kv_heads"] * case["page"] * case["dim"]


def _lens(case):
    """Cached tokens and new rows of each sequence: all alike, or unequal (a sequence without new rows among them)."""
    ctx, new = [], []
    for b in range(case["batch"]):
        f = (b * 0.6180339887) % 1.0
        ctx.append(int(round(case["ctx"] * (1 - 0.6 * f))) if case.get("ragged") else case["ctx"])
        new.append(max(1, int(round(case["rows"] * (1 - 0.7 * f)))) if case.get("ragged") else case.get("rows", 0))
    if case.get("ragged") and case["batch"] >= 4:
        new[2] = 0
    return ctx, new


def _parents(case, b):
    """The drafted tokens' parents in sequence b's tree (-1: hangs below the last cached token)."""
    r = random.Random(1000 * case["rows"] + b)
    return [max(-1, i - 1 - r.randrange(0, 6)) for i in range(case["rows"])]


def _ancestors(case, b, count):
    """Row i's visible drafted tokens, as a whole number of bits: its ancestors and itself."""
    bits = []
    for i, p in enumerate(_parents(case, b)[:count]):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return bits


def _pages(case):
    ctx, new = _lens(case)
    if case["op"] == "fork":
        return case["batch"] * (-(-ctx[0] // case["page"]) + 2 * case["beams"])
    return sum(-(-(a + b) // case["page"]) for a, b in zip(ctx, new)) + 3


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "select":
        rows = case["batch"] * case["beams"]
        live = rows - (len(_finished(case)) if case["finished"] else 0)
        return {"bytes": live * case["vocab"] * size + rows * 5 + case["batch"] * case["keep"] * 12,
                "flops": live * case["vocab"] * 4}
    ctx, new = _lens(case)
    token = 2 * case["kv_heads"] * case["dim"] * size
    if op == "append":
        n = sum(new)
        moved = n * (2 * token + 2 * case["heads"] * case["dim"] * size + 4) + case["rotary"] * 2
        return {"bytes": moved, "flops": n * (case["heads"] + case["kv_heads"]) * case["rotary"] * 3}
    if op == "attend":
        pairs = read = words = 0
        for b, (a, t) in enumerate(zip(ctx, new)):
            drafts = sum(x.bit_count() for x in _ancestors(case, b, t)) if case["tree"] else t * (t + 1) // 2
            pairs += a * t + drafts
            read += a + t if t else 0
            words += t * 4 * -(-case["rows"] // 32) if case["tree"] else 0
        rows = sum(new) * case["heads"] * (2 * case["dim"] * size + 4)
        return {"bytes": read * token + rows + words, "flops": 4 * pairs * case["heads"] * case["dim"]}
    if op == "commit":
        moved = sum(sum(1 for j, i in enumerate(p) if i != j) for p in _paths(case))
        return {"bytes": 2 * moved * token * case["layers"] + case["batch"] * 12, "flops": 0}
    fill, rows = ctx[0] % case["page"], case["batch"] * case["beams"]
    return {"bytes": 2 * rows * fill * token * case["layers"] + 8 * rows * -(-ctx[0] // case["page"]), "flops": 0}


def _paths(case):
    """An accepted path of each sequence: the first drafts of a chain, then drafts behind the path's own places, so that a
    pass over a cache that has been committed already moves the same rows."""
    paths = []
    for b in range(case["batch"]):
        r = random.Random(7 * case["rows"] + b)
        n = max(1, case["accept"] - b % 3)
        stay = r.randrange(0, n + 1) if case["rows"] > n else n
        far = sorted(r.sample(range(n, case["rows"]), min(n - stay, case["rows"] - n)))
        paths.append((list(range(stay)) + far)[:n])
    return paths


def _finished(case):
    """The finished beams' rows: every sequence but the first has one for each three beams."""
    return [b * case["beams"] + w for b in range(1, case["batch"]) for w in range(case["beams"]) if (b + w) % 3 == 0]


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    state = {"case": case, "op": case["op"]}
    if case["op"] == "select":
        B, W, V, K = case["batch"], case["beams"], case["vocab"], case["keep"]
        state["logits"] = (2.5 * torch.randn(B, W, V, generator=g, device="cuda")).to(dt)
        state["scores"] = -4 * torch.rand(B, W, generator=g, device="cuda").cumsum(1)
        ended = torch.zeros(B * W, dtype=torch.bool, device="cuda")
        ended[ints(_finished(case)).long()] = True
        state["finished"] = ended.view(B, W) if case["finished"] else None
        state["out"] = (torch.empty(B, K, device="cuda"), torch.empty(B, K, dtype=torch.int32, device="cuda"),
                        torch.empty(B, K, dtype=torch.int32, device="cuda"))
        if own:
            import confidence_gated_kv_logits_gb300 as pkg
            state["selector"] = pkg.BeamSelect(B, W, V, K, dtype=dt)
        return state

    L = case.get("layers", 2)
    Hq, H, d, ps, B = case["heads"], case["kv_heads"], case["dim"], case["page"], case["batch"]
    ctx, new = _lens(case)
    pages = _pages(case)
    pool = lambda: torch.randn(L, pages, H, ps, d, generator=g, device="cuda", dtype=dt)  # noqa: E731
    state["k_pages"], state["v_pages"] = pool(), pool()
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    beams = case.get("beams", 1)
    blocks = [-(-(a + b) // ps) for a, b in zip(ctx, new)]
    table = torch.full((B * beams, max(blocks) + 1), -1, dtype=torch.int32, device="cuda")
    if case["op"] == "fork":
        # full pages are shared by a sequence's beams; each beam has its own page of the part-filled block,
        # and a spare one, which takes the copy
        full, at = ctx[0] // ps, 0
        for b in range(B):
            table[b * beams:(b + 1) * beams, :full] = order[at:at + full]
            at += full
            if ctx[0] % ps:
                table[b * beams:(b + 1) * beams, full] = order[at:at + beams]
                at += beams
        state["tail_pages"] = order[at:at + B * beams].contiguous()
        state["table"], state["lens"] = table, ints([ctx[0]] * (B * beams))
        state["parent"] = torch.randint(0, beams, (B * beams,), generator=g, device="cuda", dtype=torch.int32)
        state["table_out"], state["lens_out"] = torch.full_like(table, -1), torch.zeros_like(state["lens"])
    else:
        at = 0
        for b, n in enumerate(blocks):
            table[b, :n] = order[at:at + n]
            at += n
        state["table"], state["ctx"] = table, ints(ctx)
        starts = [sum(new[:b]) for b in range(B + 1)]
        state["q_start"], state["live"] = ints(starts), starts[-1]
    n = sum(new) + (2 if case.get("ragged") else 0)  # a padded batch: rows behind the last sequence
    if case["op"] == "append":
        qkv = torch.randn(n, Hq + 2 * H, d, generator=g, device="cuda", dtype=dt)  # a fused projection's output
        state["q"], state["k"], state["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        state["q_out"] = torch.zeros(n, Hq, d, device="cuda", dtype=dt)
        state["pos"] = ints([a + i for a, t in zip(ctx, new) for i in range(t)] + [0] * (n - sum(new)))
        r = case["rotary"]
        state["inv_freq"] = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()
    if case["op"] == "attend":
        state["q"] = torch.randn(n, Hq, d, generator=g, device="cuda", dtype=dt)
        state["out"] = torch.zeros(n, Hq, d, device="cuda", dtype=dt)
        state["lse"] = torch.zeros(n, Hq, device="cuda")
        state["mask"] = None
        state["longest"] = max(new)
        if case["tree"]:
            words = -(-max(new) // 32)
            rows = [x for b, t in enumerate(new) for x in _ancestors(case, b, t)] + [0] * (n - sum(new))
            cut = [[(x >> 32 * w) & 0xFFFFFFFF for w in range(words)] for x in rows]
            state["mask"] = ints([[w - (1 << 32) if w >> 31 else w for w in x] for x in cut])
    if case["op"] == "commit":
        paths = _paths(case)
        state["path"] = ints([p + [-1] * (case["accept"] - len(p)) for p in paths])
        state["path_len"] = ints([len(p) for p in paths])
        state["lens_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if own:
        import confidence_gated_kv_logits_gb300 as pkg
        state["kv"] = pkg.PagedKV(state["k_pages"], state["v_pages"], Hq)
        if case["op"] in ("append", "attend"):
            state["batch"] = state["kv"].batch(state["table"], state["ctx"], state["q_start"], state.get("mask"))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return PLAIN[state["op"]](state)


def _run_own(s):
    op, case = s["op"], s["case"]
    if op == "append":
        s["kv"].append(case.get("layers", 2) - 1, s["batch"], s["k"], s["v"], q=s["q"], q_out=s["q_out"],
                       positions=s["pos"], inv_freq=s["inv_freq"], interleaved=case["interleaved"])
        return s["q_out"], s["k_pages"], s["v_pages"]
    if op == "attend":
        s["kv"].attend(1, s["batch"], s["q"], s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "commit":
        s["kv"].commit(s["table"], s["ctx"], s["path"], s["path_len"], s["lens_out"])
        return s["k_pages"], s["v_pages"], s["lens_out"]
    if op == "select":
        s["selector"].select(s["logits"], s["scores"], *s["out"], finished=s["finished"], pad_token=0)
        return s["out"]
    s["kv"].fork(s["parent"], case["beams"], s["table"], s["lens"], s["tail_pages"], s["table_out"], s["lens_out"])
    return s["table_out"], s["lens_out"], s["k_pages"], s["v_pages"]


def _plain_append(s):
    case, n = s["case"], s["live"]
    rows = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), rows, right=True)
    place = s["ctx"].long()[seq] + rows - s["q_start"].long()[seq]
    page, slot = s["table"].long()[seq, place // case["page"]], place % case["page"]
    angle = s["pos"][:n, None].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotated(x):
        x, r = x[:n].float(), case["rotary"]
        y = x.clone()
        if case["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
        return y

    layer = case["layers"] - 1
    s["q_out"][:n] = rotated(s["q"]).to(s["q_out"].dtype)
    s["k_pages"][layer, page, :, slot] = rotated(s["k"]).to(s["k_pages"].dtype)
    s["v_pages"][layer, page, :, slot] = s["v"][:n]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _plain_attend(s):
    case, n, T = s["case"], s["live"], s["longest"]
    B, Hq, H, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    g, dev = Hq // H, s["q"].device
    ctx, start = s["ctx"].long(), s["q_start"].long()
    new = start[1:] - start[:-1]

    def cached(pages):
        x = pages[1][s["table"].clamp(min=0).long()]  # [B, blocks, H, page, d]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, -1, d).float()

    t = torch.arange(T, device=dev)
    rows = (start[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, T, H, g, d).permute(0, 2, 1, 3, 4).reshape(B, H, T * g, d)
    scores = (q @ cached(s["k_pages"]).transpose(2, 3)) / math.sqrt(d)
    S = scores.shape[3]
    at = torch.arange(S, device=dev)
    j = at - ctx[:, None]  # [B, S]: which new row of the sequence
    if s["mask"] is None:
        seen = j[:, None, :] <= t[:, None]
    else:
        word = s["mask"][rows].gather(2, (j.clamp(0, T - 1) // 32)[:, None].expand(B, T, S))
        seen = (j < 0)[:, None, :] | ((word >> (j.clamp(min=0) % 32)[:, None].int() & 1) == 1)
    seen = seen & (j < new[:, None])[:, None, :]
    scores.view(B, H, T, g, S).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (scores - top).exp_()
    del scores
    total = p.sum(3, keepdim=True)
    out = (p @ cached(s["v_pages"])) / torch.where(total == 0, torch.ones_like(total), total)
    lse = top + total.log()
    i = torch.arange(n, device=dev)
    b = torch.searchsorted(start[1:], i, right=True)
    out, lse = out.view(B, H, T, g, d), lse.view(B, H, T, g)
    s["out"][:n] = out[b, :, i - start[b]].reshape(n, Hq, d).to(s["out"].dtype)
    s["lse"][:n] = lse[b, :, i - start[b]].reshape(n, Hq)
    return s["out"], s["lse"]


def _plain_commit(s):
    case = s["case"]
    table, ctx, path, count = s["table"].long(), s["ctx"].long(), s["path"].long(), s["path_len"].long()
    j = torch.arange(path.shape[1], device=table.device)
    to = ctx[:, None] + j
    use = j < count[:, None]
    # behind the path's end a row moves onto itself
    source = torch.where(use, ctx[:, None] + path, to.clamp(max=ctx[:, None] + case["rows"] - 1))
    to = torch.where(use, to, source)
    page = lambda x: table.gather(1, x // case["page"])  # noqa: E731
    for pool in (s["k_pages"], s["v_pages"]):
        moved = pool[:, page(source), :, source % case["page"]]
        pool[:, page(to), :, to % case["page"]] = moved
    s["lens_out"].copy_(s["ctx"] + s["path_len"])
    return s["k_pages"], s["v_pages"], s["lens_out"]


def _plain_select(s):
    case = s["case"]
    z = s["logits"].double()
    top = z.amax(2, keepdim=True)
    total = s["scores"].double()[..., None] + (z - top - (z - top).exp().sum(2, keepdim=True).log())
    if s["finished"] is not None:
        # a finished beam goes on as itself: one candidate, the padding token, at the score that it has
        one = torch.full_like(total, -math.inf)
        one[..., 0] = s["scores"].double()
        total = torch.where(s["finished"][..., None], one, total)
    best, at = total.view(case["batch"], -1).sort(dim=1, descending=True, stable=True)
    best, at = best[:, :case["keep"]], at[:, :case["keep"]]
    none = best == -math.inf
    s["out"][0].copy_(best)
    s["out"][1].copy_(torch.where(none, -1, at // case["vocab"]))
    s["out"][2].copy_(torch.where(none, -1, at % case["vocab"]))
    return s["out"]


def _plain_fork(s):
    case = s["case"]
    W, ps, n = case["beams"], case["page"], case["batch"] * case["beams"]
    row = torch.arange(n, device="cuda")
    parent = row // W * W + s["parent"].long()
    lens = s["lens"].long()[parent]
    block = torch.arange(s["table"].shape[1], device="cuda")
    tables = s["table"][parent]
    tail = (block == (lens // ps)[:, None]) & (lens % ps != 0)[:, None]
    mine = torch.where(tail, s["tail_pages"][:, None], tables)
    s["table_out"].copy_(torch.where(block < ((lens + ps - 1) // ps)[:, None], mine, s["table_out"]))
    s["lens_out"].copy_(lens)
    source = tables.long().gather(1, (lens // ps)[:, None])[:, 0].clamp(min=0)
    to = s["tail_pages"].long()
    filled = (torch.arange(ps, device="cuda") < (lens % ps)[:, None])[None, :, None, :, None]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, to] = torch.where(filled, pool[:, source], pool[:, to])
    return s["table_out"], s["lens_out"], s["k_pages"], s["v_pages"]


PLAIN = {"append": _plain_append, "attend": _plain_attend, "commit": _plain_commit, "select": _plain_select,
         "fork": _plain_fork}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("commit", "fork"):
        return None  # rows are copied as they are: no computed numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return _exact_select(case, s)


def _exact_append(case, s):
    """The rotation as a complex product, sequence by sequence."""
    r, ps, layer = case["rotary"], case["page"], case["layers"] - 1
    q_out, ks, vs = s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()
    ctx, new = _lens(case)
    row = 0

    def turn(x, phase):
        x = x.double()
        even = torch.arange(0, r, 2) if case["interleaved"] else torch.arange(r // 2)
        odd = even + (1 if case["interleaved"] else r // 2)
        z = torch.complex(x[:, :, even], x[:, :, odd]) * phase[:, None]
        y = x.clone()
        y[:, :, even], y[:, :, odd] = z.real, z.imag
        return y

    for b, t in enumerate(new):
        if not t:
            continue
        at = slice(row, row + t)
        angle = torch.outer(s["pos"][at].double(), s["inv_freq"].double())
        phase = torch.polar(torch.ones_like(angle), angle)
        q_out[at] = turn(s["q"][at], phase)
        place = torch.arange(ctx[b], ctx[b] + t, device="cuda")
        page = s["table"][b].long()[place // ps]
        ks[layer, page, :, place % ps] = turn(s["k"][at], phase)
        vs[layer, page, :, place % ps] = s["v"][at].double()
        row += t
    return q_out, ks, vs


def _exact_attend(case, s):
    ctx, new = _lens(case)
    if sum(a * t for a, t in zip(ctx, new)) * case["heads"] * case["dim"] > 4e12:
        return None
    out, lse = s["out"].double(), s["lse"].double()
    g, d, row = case["heads"] // case["kv_heads"], case["dim"], 0
    for b, t in enumerate(new):
        if not t:
            continue
        n = ctx[b] + t
        pages = s["table"][b, :-(-n // case["page"])].long()
        seen = torch.ones(t, n, dtype=torch.bool)
        if case["tree"]:
            bits = _ancestors(case, b, t)
            seen[:, ctx[b]:] = torch.tensor([[bool(x >> i & 1) for i in range(t)] for x in bits])
        else:
            seen[:, ctx[b]:] = torch.tril(torch.ones(t, t, dtype=torch.bool))
        hide = torch.zeros(t, n, dtype=torch.float64).masked_fill_(~seen, -math.inf).cuda()
        for h in range(case["heads"]):
            k = s["k_pages"][1, pages, h // g].reshape(-1, d)[:n].double()
            v = s["v_pages"][1, pages, h // g].reshape(-1, d)[:n].double()
            z = s["q"][row:row + t, h].double() @ k.T * d ** -0.5 + hide
            norm = torch.logsumexp(z, 1)
            out[row:row + t, h] = torch.exp(z - norm[:, None]) @ v
            lse[row:row + t, h] = norm
        row += t
    return out, lse


def _exact_select(case, s):
    B, W, V, K = case["batch"], case["beams"], case["vocab"], case["keep"]
    ended = s["finished"].cpu() if s["finished"] is not None else torch.zeros(B, W, dtype=torch.bool)
    best, parents, tokens = [], [], []
    for b in range(B):
        found = []
        for w in range(W):
            score = s["scores"][b, w].double().item()
            if ended[b, w]:
                found.append((-score, w, 0))
                continue
            logp = torch.log_softmax(s["logits"][b, w].double(), 0)
            # the row's best K and what ties with the last of them
            edge = logp.sort(descending=True).values[min(K, V) - 1]
            ids = (logp >= edge).nonzero()[:, 0]
            found += [(-(score + x), w, i) for x, i in zip(logp[ids].tolist(), ids.tolist())]
        found = [f for f in sorted(found) if f[0] < math.inf][:K]
        found += [(math.inf, -1, -1)] * (K - len(found))
        best.append([-f[0] for f in found])
        parents.append([f[1] for f in found])
        tokens.append([f[2] for f in found])
    return (torch.tensor(best, dtype=torch.float64), torch.tensor(parents, dtype=torch.int32),
            torch.tensor(tokens, dtype=torch.int32))
