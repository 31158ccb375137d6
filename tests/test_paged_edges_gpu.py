"""Paged-cache and beam operators where values or metadata are at the edge of what they take: NaN and infinities that a
row does see, page tables that are wrong or too narrow, a workspace that calls of several sizes share.

Tolerances are those of test_paged_gpu.py (stated there), here for any set of visible tokens."""
import ctypes
import math

import pytest
import torch

from tests.test_paged_gpu import DEV, DT, U, Case, check, check_select, ints, mask_words, reference, run_attend, run_select, select_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import confidence_gated_kv_logits_gb300 as pkg
    pkg.load_library()
    return pkg


# (heads, kv_heads, d, ctx, new, widened table): how attend shares the work out
FORMS = {
    "few, a cluster a unit": (12, 12, 64, [2047], [1], False),
    "few, whole units": (40, 8, 128, [50] * 4, [1] * 4, False),
    "few, cut units": (12, 12, 64, [9000], [1], True),
    "few, over 32 sequences": (14, 2, 64, [600] * 33, [1] * 33, False),
    "many, joined on all SMs": (40, 8, 128, [1500, 0], [13, 9], False),
    "many, joined by the last piece": (8, 2, 64, [40] * 60, [20] * 60, False),
    "many, tile pairs": (40, 8, 128, [300] * 5, [400] * 5, False),
}


def case_of(name, dt, seed=1, **kw):
    heads, kv_heads, d, ctx, new, wide = FORMS[name]
    c = Case(dt, heads, kv_heads, d, 32, ctx, new, seed=seed, **kw)
    if wide:
        c.table = torch.nn.functional.pad(c.table, (0, 4000), value=-1).contiguous()
    return c


def exact(c, vis, layer=1):
    """out, lse and their tolerances (test_paged_gpu.py's) with vis[b] [t, n] the tokens that are seen; a sequence's
    first n tokens lie in its pages."""
    u, g, scale = U[c.dt], c.heads // c.H, c.d ** -0.5
    outs, lses, tols, tol_ls = [], [], [], []
    for b, t in enumerate(c.new):
        if not t:
            continue
        seen, n, at = vis[b].to(DEV), vis[b].shape[1], c.starts[b]
        K, V = (x.double().nan_to_num(0, 0, 0).repeat_interleave(g, 1) for x in (c.get(c.k, layer, b, n), c.get(c.v, layer, b, n)))
        q = c.q[at:at + t].double()
        z = torch.einsum("thd,nhd->thn", q, K) * scale
        z = torch.where(seen[:, None], z, -math.inf)
        m = z.amax(2, keepdim=True)
        p = (z - torch.where(m == -math.inf, 0, m)).exp()
        l = p.sum(2, keepdim=True)
        p = p / torch.where(l == 0, 1, l)
        o, A = torch.einsum("thn,nhd->thd", p, V), torch.einsum("thn,nhd->thd", p, V.abs())
        size = torch.where(seen[:, None], torch.einsum("thd,nhd->thn", q.abs(), K.abs()), 0).amax(2)
        ds = (c.d + 4) * 2.0 ** -23 * scale * size
        e = u * o.abs() + (u + 2 * ds[..., None] + n * 2.0 ** -23) * A
        if c.dt is torch.float16:
            e = e + n * 2.0 ** -25 * V.abs().amax()
        lse = (m + l.log())[..., 0]
        outs.append(o), lses.append(lse), tols.append(e)
        tol_ls.append(ds + n * 2.0 ** -23 + 2.0 ** -22 * (1 + lse.abs()))
    return [torch.cat(x) for x in (outs, lses, tols, tol_ls)]


def causal(c, cap=None):
    return [torch.ones(t, a + t, dtype=torch.bool).tril(a)[:, :cap] for a, t in zip(c.ctx, c.new)]


def compare(c, got, want, lost=None):
    """lost [rows, heads]: rows that have to be NaN; the others have to be within the tolerance."""
    n = c.starts[-1]
    out, lse = got[0][:n].double(), got[1][:n].double()
    o, l, tol, tol_l = want
    lost = torch.zeros(n, c.heads, dtype=torch.bool, device=DEV) if lost is None else lost
    assert torch.isnan(out[lost]).all() and torch.isnan(lse[lost]).all()
    assert ((out - o).abs()[~lost] <= tol[~lost]).all()
    dead = l == -math.inf
    assert torch.equal((lse == -math.inf)[~lost], dead[~lost])
    live = ~lost & ~dead
    assert ((lse - l).abs()[live] <= tol_l[live]).all()
    assert (got[0][n:] == 7).all() and (got[1][n:] == 7).all()


# --------------------------------------------------------------------------- NaN that a row sees
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("form", list(FORMS))
def test_attend_a_nan_query_gives_nan(pkg, form, dt):
    c = case_of(form, DT[dt])
    want = reference(c)
    n = c.starts[-1]
    lost = torch.zeros(n, c.heads, dtype=torch.bool, device=DEV)
    lost[0, 0] = lost[n - 1, c.heads - 1] = lost[n // 2, c.heads // 2] = True
    q = c.q.clone()
    q[:n][lost] = torch.where(torch.arange(c.d, device=DEV) == 3, math.nan, q[:n][lost].float()).to(c.dt)
    compare(c, run_attend(pkg, c, q=q), want, lost)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("form", list(FORMS))
def test_attend_nan_keys_reach_every_row_that_sees_them(pkg, form, dt):
    """Keys that are all NaN over a stretch of tokens that begins and ends with the tiles, so that some warps and pieces
    hold nothing else and none holds both."""
    c = case_of(form, DT[dt])
    want = exact(c, causal(c))
    b = 0
    n = c.ctx[b] + c.new[b]
    lo, hi = (n // 3 // 128 * 128, n // 2 // 128 * 128 + 128) if n > 500 else (16, 32)
    at = torch.arange(lo, hi, device=DEV)
    h = c.H - 1
    c.k[:, c.table[b].long()[at // c.page], h, at % c.page] = math.nan
    lost = torch.zeros(c.starts[-1], c.heads, dtype=torch.bool, device=DEV)
    first = c.starts[b] + max(0, lo - c.ctx[b])             # causal: the rows from token lo on
    lost[first:c.starts[b] + c.new[b], h * c.heads // c.H:] = True
    compare(c, run_attend(pkg, c), want, lost)


# --------------------------------------------------------------------------- infinities that a row sees
@pytest.mark.parametrize("dt", list(DT))
def test_attend_an_infinite_value_behind_tiles_that_the_row_does_not_see(pkg, dt):
    """Row 200 sees drafts 140 and 145 alone; draft 140's V is infinite in some channels."""
    c = Case(DT[dt], 2, 2, 128, 32, [0] * 32, [300] + [1] * 31, seed=9)
    bits = [(1 << i + 1) - 1 for i in range(300)] + [1] * 31
    bits[200] = 1 << 140 | 1 << 145
    for i in range(140, 300):
        if i != 200:
            bits[i] &= ~(1 << 140)
    pg, s = int(c.table[0, 140 // 32]), 140 % 32
    vis = [torch.tensor([[x >> j & 1 for j in range(t)] for x in bits[a:a + t]], dtype=torch.bool) for a, t in zip(c.starts, c.new)]
    c.v[:, pg, :, s, ::3] = math.inf
    c.v[:, pg, :, s, 1::3] = -math.inf
    want = exact(c, vis)                                    # (with zeroes in the place of the infinities)
    got = run_attend(pkg, c, bits)
    assert (got[0][200, :, ::3] == math.inf).all() and (got[0][200, :, 1::3] == -math.inf).all()
    rest = got[0].clone()
    rest[200, :, ::3] = rest[200, :, 1::3] = 0
    want[0][200, :, ::3] = want[0][200, :, 1::3] = 0
    compare(c, (rest, got[1]), want)


# --------------------------------------------------------------------------- scores far beyond what 32 bits tell apart
@pytest.mark.parametrize("dt,most", [("fp16", 6e4), ("bf16", 6e4), ("bf16", 1e17)])
@pytest.mark.parametrize("form", list(FORMS))
def test_attend_huge_scores_leave_the_largest(pkg, form, dt, most):
    """Queries of `most` in every channel and keys that rise from 0 to it: a score is 1e10 and more, the next lower one a
    hundredth of it away or further, so that one token's weight is 1 and the others' are 0, as in 64 bits."""
    c = case_of(form, DT[dt])
    for b, (a, t) in enumerate(zip(c.ctx, c.new)):
        size = torch.zeros(a + t, dtype=torch.float64)
        size[:] = -most * torch.arange(1, a + t + 1) / (a + t) * 0.5
        size[0] = 0.5 * most
        if a > 2:
            size[a // 2] = most                             # seen by every row
        k = size.to(c.dt).to(DEV)[None, :, None, None].expand(c.layers, -1, c.H, c.d)
        at = torch.arange(a + t, device=DEV)
        c.k[:, c.table[b].long()[at // c.page], :, at % c.page] = k.permute(1, 0, 2, 3)
    c.q[:] = most
    got = run_attend(pkg, c)
    g = c.heads // c.H
    for b, (a, t) in enumerate(zip(c.ctx, c.new)):
        j = a // 2 if a > 2 else 0
        v = c.get(c.v, 1, b, a + t)[j].repeat_interleave(g, 0)
        assert torch.equal(got[0][c.starts[b]:c.starts[b + 1]], v[None].expand(t, -1, -1))
        z = float(torch.tensor(most, dtype=c.dt)) * float(c.k[1, c.table[b].long()[j // c.page], 0, j % c.page, 0]) * c.d ** 0.5
        assert torch.allclose(got[1][c.starts[b]:c.starts[b + 1]].double(), torch.tensor(z, dtype=torch.float64, device=DEV), rtol=(c.d + 4) * 2.0 ** -23, atol=0)


# --------------------------------------------------------------------------- page tables that are wrong
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("bad", [-1, 1 << 30])
@pytest.mark.parametrize("form", list(FORMS))
def test_attend_a_bad_page_voids_the_rows_that_see_it(pkg, form, bad, dt):
    """The second page of every other sequence is none: NaN for the rows that see it, whatever page 0 holds."""
    c = case_of(form, DT[dt])
    vis = causal(c)
    want = exact(c, vis)
    lost = torch.zeros(c.starts[-1], c.heads, dtype=torch.bool, device=DEV)
    table = c.table.clone()
    for b, v in enumerate(vis):
        if b % 2 == 0 and v.shape[1] > c.page:
            table[b, 1] = bad
            lost[c.starts[b]:c.starts[b + 1]] = v[:, c.page:2 * c.page].any(1).to(DEV)[:, None]
    assert lost.any()
    kv = pkg.PagedKV(c.k, c.v, c.heads)
    got = run_attend(pkg, c, kv=kv, batch=kv.batch(table, ints(c.ctx), ints(c.starts)))
    assert kv.status(check=False) == pkg.FLAG_BAD_PAGE
    compare(c, got, want, lost)
    check(c, run_attend(pkg, c, kv=kv), reference(c))       # nothing stays behind
    assert kv.status() == 0


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("new,d", [(1, 64), (3, 128), (90, 64), (700, 128)])
def test_attend_a_tree_over_bad_pages(pkg, new, d, dt):
    """Masks and bad pages of drafts together, small pages: rows that do not see their tokens are right."""
    c = Case(DT[dt], 6, 2, d, 16, [80, 80], [new, new], seed=new)
    bits = [1 << i | 1 << i // 2 | 1 for i in range(new)]
    vis = torch.ones(new, 80 + new, dtype=torch.bool)
    vis[:, 80:] = torch.tensor([[bool(x >> j & 1) for j in range(new)] for x in bits]).view(new, new)
    table, last = c.table.clone(), (80 + new - 1) // 16
    lost = torch.zeros(2 * new, 6, dtype=torch.bool, device=DEV)
    for blk in {last, min(last, max(6, last // 2))}:
        table[0, blk] = c.k.shape[1]
        lost[:new] |= vis[:, 16 * blk:16 * blk + 16].any(1).to(DEV)[:, None]
    kv = pkg.PagedKV(c.k, c.v, c.heads)
    mask = mask_words(2 * bits + [0] * (c.rows - 2 * new), -(-new // 32))
    got = run_attend(pkg, c, kv=kv, batch=kv.batch(table, ints(c.ctx), ints(c.starts), mask))
    assert kv.status(check=False) == pkg.FLAG_BAD_PAGE and lost.any() and not lost.all()
    compare(c, got, exact(c, [vis, vis]), lost)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,kv_heads,d,ctx,new,blocks", [
    (4, 4, 64, 30, 9, 1), (4, 4, 64, 40, 9, 3), (10, 2, 128, 20, 400, 3), (8, 1, 64, 100, 300, 9), (10, 2, 128, 90, 1500, 7),
    (40, 8, 128, 0, 700, 5), (2, 2, 64, 500, 3, 1)])
def test_attend_rows_past_the_page_table(pkg, heads, kv_heads, d, ctx, new, blocks, dt):
    """A sequence longer than its table: rows see its tokens as far as the table goes, the flag says so."""
    c = Case(DT[dt], heads, kv_heads, d, 16, [ctx, 50], [new, 2], seed=blocks)
    cap = 16 * blocks
    n = min(cap, ctx + new)
    vis = [v[:, :cap] for v in causal(c)]
    want = exact(c, vis)
    kv = pkg.PagedKV(c.k, c.v, heads)
    batch = kv.batch(c.table[:, :blocks].contiguous(), ints(c.ctx), ints(c.starts))
    got = run_attend(pkg, c, kv=kv, batch=batch)
    assert kv.status(check=False) == pkg.FLAG_CAPACITY
    compare(c, got, want)
    for _ in range(3):
        again = run_attend(pkg, c, kv=kv, batch=batch)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert n == vis[0].shape[1] and kv.status(check=False) == pkg.FLAG_CAPACITY


# --------------------------------------------------------------------------- one workspace for calls of several sizes
def test_select_one_workspace_for_every_size(pkg):
    """Zeroed once, made for the largest call, used by smaller and larger ones in turn (C ABI)."""
    L = pkg.load_library()
    sizes = [(3, 2, 700, 4, torch.float32), (100, 3, 500, 5, torch.float32), (3, 2, 700, 4, torch.float32), (1, 4, 50257, 8, torch.bfloat16),
             (700, 1, 40, 3, torch.float16), (2, 32, 9000, 64, torch.float32), (100, 3, 500, 5, torch.float32)]
    code = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
    ws = torch.zeros(max(L.confkv_beam_workspace(B, W, V, K, code[t]) for B, W, V, K, t in sizes), dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    for B, W, V, K, dt in sizes:
        z = (3 * torch.randn(B, W, V, generator=g, device=DEV)).to(dt)
        scores = -torch.rand(B, W, generator=g, device=DEV)
        so, po, to = torch.full((B, K), 7.0, device=DEV), *(torch.full((B, K), 7, dtype=torch.int32, device=DEV) for _ in range(2))
        rc = L.confkv_beam_select(z.data_ptr(), code[dt], V, B, W, V, K, scores.data_ptr(), None, 0, so.data_ptr(), po.data_ptr(),
                                  to.data_ptr(), None, ws.data_ptr(), ws.numel(), -1, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert rc == 0
        check_select((so, po, to), select_reference(z.cpu(), scores.cpu(), None, K, 0))


# --------------------------------------------------------------------------- how far scores may be off
def spread(kind, V, g):
    if kind == "flat":
        return torch.zeros(V, device=DEV)
    if kind == "peak":                                      # one token over a flat tail
        z = torch.full((V,), -12.0, device=DEV)
        z[V // 3] = 0
        return z
    return {"narrow": 1.0, "wide": 4.0}[kind] * torch.randn(V, generator=g, device=DEV)


def lse_bound(z):
    """The selection's lse against 64 bits.  A term e^d, d = z - max, is off by 2^-22 (ex2.approx) and by |d| (2^-24 + 2^-24 +
    2^-26) of its value (d and its product with log2 e rounded, log2 e's own rounding); the weighted mean of |d| is max -
    sum p z.  A thread adds its terms (64 at most) in 11 rounded steps of 2^-24; what is cut off at 2^-38 a thread is below
    2^-26 of the sum, which is 1 at least (where threads take 8 terms each, so that there are up to 2^15 of them, below
    2^-23, but the steps are 6); the logarithm's Newton step adds less than 2^-40: 12 2^-24 covers both."""
    z = z.double()
    lse = torch.logsumexp(z, 0)
    return lse, 2.0 ** -22 + float(z.max() - (torch.softmax(z, 0) * z).sum()) * 2.25 * 2.0 ** -24 + 12 * 2.0 ** -24


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [50257, 201088])
@pytest.mark.parametrize("kind", ["flat", "peak", "narrow", "wide"])
def test_select_scores_are_as_good_as_stated(pkg, kind, V, dt):
    """score = scores[w] + z - lse near 0, so that its rounding to 32 bits does not hide the error of lse."""
    z = spread(kind, V, torch.Generator(device=DEV).manual_seed(V)).to(dt)
    lse, bound = lse_bound(z)
    start = (lse - z.double().max()).float()
    so, po, to, _, _ = run_select(pkg, z.view(1, 1, V), start.view(1, 1), 1)
    want = start.double() + z.double().max() - lse
    assert int(to) == int(z.float().argmax()) and abs(float(so) - float(want)) <= bound + 2.0 ** -24 * abs(float(want))


@pytest.mark.parametrize("V", [50257, 201088])
@pytest.mark.parametrize("kinds", [("flat", "peak"), ("peak", "wide"), ("narrow", "flat"), ("wide", "narrow")])
def test_select_orders_beams_that_differ_by_more_than_the_bound(pkg, kinds, V):
    g = torch.Generator(device=DEV).manual_seed(V)
    z = torch.stack([spread(k, V, g) for k in kinds])
    (la, ba), (lb, bb) = (lse_bound(x) for x in z)
    for sign in (1, -1):
        # the second beam's best, ahead of or behind the first's by a little more than both may be off
        best = [float(z[0].double().max() - la), float(z[1].double().max() - lb)]
        gap = 1.1 * (ba + bb)
        first = torch.tensor(-best[0], dtype=torch.float64).float()
        second = torch.tensor(float(first) + best[0] - best[1] + sign * gap, dtype=torch.float64).float()
        real = float(second) + best[1] - (float(first) + best[0])
        if abs(real) <= ba + bb:                            # the score's own 32 bits are coarser
            second = torch.nextafter(second, torch.tensor(sign * math.inf))
            real = float(second) + best[1] - (float(first) + best[0])
        assert sign * real > ba + bb
        so, po, _, _, _ = run_select(pkg, z.view(1, 2, V), torch.stack([first, second]).view(1, 2).to(DEV), 1)
        assert int(po) == (1 if sign > 0 else 0)


# --------------------------------------------------------------------------- the largest and the oddest sizes
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("new", [[1, 0, 2], [40, 70, 0]])
def test_rows_before_the_first_sequence_are_left_as_they_were(pkg, new, dt):
    c = Case(DT[dt], 8, 2, 64, 16, [20, 33, 64], new, seed=5)
    n, lead = c.starts[-1], 5
    q = torch.cat([c.randn(lead, 8, 64), c.q])
    want = reference(c)
    kv = pkg.PagedKV(c.k, c.v, 8)
    batch = kv.batch(c.table, ints(c.ctx), ints([lead + x for x in c.starts]))
    out, lse = torch.full_like(q, 7), torch.full(q.shape[:2], 7.0, device=DEV)
    kv.attend(1, batch, q, out, lse=lse)
    assert (out[:lead] == 7).all() and (lse[:lead] == 7).all()
    check(c, (out[lead:], lse[lead:]), want)
    k, v, q_out, k0 = c.randn(lead + c.rows, 2, 64), c.randn(lead + c.rows, 2, 64), torch.full_like(q, 7), c.k.clone()
    kv.append(0, batch, k, v, q=q, q_out=q_out)
    assert torch.equal(q_out[lead:lead + n], q[lead:lead + n]) and (q_out[:lead] == 7).all() and (q_out[lead + n:] == 7).all()
    for b, (a, t) in enumerate(zip(c.ctx, new)):
        assert torch.equal(c.get(c.k, 0, b, a + t)[a:], k[lead + c.starts[b]:lead + c.starts[b + 1]])
        c.put(b, a, k0[:, c.table[b].long()[torch.arange(a, a + t, device=DEV) // 16], :, torch.arange(a, a + t, device=DEV) % 16].transpose(0, 1), c.get(c.v, 1, b, a + t)[None, a:].expand(2, -1, -1, -1))
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16))         # nothing else was written
    assert kv.status() == 0


@pytest.mark.parametrize("t", [40, 70])
def test_drafts_past_the_masks_words_are_seen_by_no_row(pkg, t):
    c = Case(torch.float16, 6, 2, 64, 16, [10], [t], seed=t)
    bits = [(1 << t) - 1] * t
    kv = pkg.PagedKV(c.k, c.v, 6)
    vis = torch.ones(t, 10 + t, dtype=torch.bool)
    vis[:, 10 + 32:] = False
    mask = mask_words([x & 0xFFFFFFFF for x in bits] + [0] * 3, 1)
    got = run_attend(pkg, c, kv=kv, batch=kv.batch(c.table, ints(c.ctx), ints(c.starts), mask))
    compare(c, got, exact(c, [vis]))


def test_the_most_sequences(pkg):
    """65536 sequences of up to 40 tokens: append and attend."""
    B, H, heads, d, page = 65536, 1, 2, 64, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    ctx = torch.randint(0, 40, (B,), generator=g, device=DEV, dtype=torch.int32)
    table = torch.randperm(B * 3, generator=g, device=DEV).to(torch.int32).view(B, 3)
    pool = lambda: torch.randn(1, B * 3, H, page, d, generator=g, device=DEV).half()  # noqa: E731
    k, v = pool(), pool()
    kv = pkg.PagedKV(k, v, heads)
    qkv = torch.randn(B, heads + 2 * H, d, generator=g, device=DEV).half()
    batch = kv.batch(table, ctx, torch.arange(B + 1, dtype=torch.int32, device=DEV))
    kv.append(0, batch, qkv[:, heads:heads + H], qkv[:, heads + H:])
    out = torch.empty(B, heads, d, dtype=torch.float16, device=DEV)
    kv.attend(0, batch, qkv[:, :heads], out)
    assert kv.status() == 0
    K, V = (x[0][table.long()].transpose(1, 2).reshape(B, 3 * page, d) for x in (k, v))
    row = torch.arange(B, device=DEV)
    assert torch.equal(K[row, ctx.long()], qkv[:, heads]) and torch.equal(V[row, ctx.long()], qkv[:, heads + 1])
    z = torch.einsum("bhd,bnd->bhn", qkv[:, :heads].double(), K.double()) * d ** -0.5
    z = torch.where(torch.arange(3 * page, device=DEV) <= ctx[:, None, None], z, -math.inf)
    p = torch.softmax(z, 2)
    o, A = torch.einsum("bhn,bnd->bhd", p, V.double()), torch.einsum("bhn,bnd->bhd", p, V.double().abs())
    ds = (d + 4) * 2.0 ** -23 * d ** -0.5 * float((qkv[:, :heads].double().abs().sum(2).amax() * K.double().abs().amax()))
    u = U[torch.float16]
    assert ((out.double() - o).abs() <= u * o.abs() + (u + 2 * ds + 48 * 2.0 ** -23) * A + 48 * 2.0 ** -25 * float(V.abs().amax())).all()


def test_commit_of_the_longest_path(pkg):
    """1000 of 2000 drafts, kept through pages in no order; another sequence's path of 1024 that stays where it is."""
    c = Case(torch.float16, 2, 2, 64, 16, [5, 16], [2000, 1024], layers=2, seed=8)
    g = torch.Generator().manual_seed(1)
    path = torch.randperm(2000, generator=g)[:1000].sort().values.to(torch.int32)
    want = [x.clone() for x in (c.k, c.v)]
    to = torch.arange(5, 1005, device=DEV)
    for pool, w in zip((c.k, c.v), want):
        at = path.to(DEV).long() + 5
        w[:, c.table[0].long()[to // 16], :, to % 16] = pool[:, c.table[0].long()[at // 16], :, at % 16]
    paths = torch.full((2, 1024), -1, dtype=torch.int32)
    paths[0, :1000] = path
    paths[1] = torch.arange(1024)
    kv = pkg.PagedKV(c.k, c.v, 2)
    new_len = ints([0, 0])
    kv.commit(c.table, ints(c.ctx), paths.to(DEV), ints([1000, 1024]), new_len)
    assert kv.status() == 0 and new_len.tolist() == [1005, 1040]
    assert torch.equal(c.k.view(torch.int16), want[0].view(torch.int16)) and torch.equal(c.v.view(torch.int16), want[1].view(torch.int16))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,W,V,keep", [(1, 1, 1 << 24, 64), (1, 32, 300000, 64), (65535, 1, 2, 1), (2047, 32, 5, 64)])
def test_select_the_largest_sizes(pkg, B, W, V, keep, dt):
    """Distinct logits and scores, so that the order is the definition's (with no pair nearer than the stated precision)."""
    g = torch.Generator(device=DEV).manual_seed(V)
    z = (2 * torch.randn(B, W, V, generator=g, device=DEV)).to(dt)
    scores = -torch.rand(B, W, generator=g, device=DEV)
    so, po, to, fl, _ = run_select(pkg, z, scores, keep)
    x = z.double()
    total = scores.double()[..., None] + x - torch.logsumexp(x, 2, keepdim=True)
    best, at = total.view(B, -1).topk(min(keep, W * V), dim=1)
    n = best.shape[1]
    assert ((so[:, :n].double() - best).abs() <= 2.0 ** -18 + 2.0 ** -24 * best.abs()).all() and not fl.any()
    # what was chosen has the score that the definition gives it, and is chosen once
    flat = po[:, :n].long() * V + to[:, :n]
    assert ((total.view(B, -1).gather(1, flat) - best).abs() <= 2.0 ** -18).all()
    assert (flat.sort(1).values.diff(dim=1) > 0).all()
    if n < keep:
        assert (so[:, n:] == -math.inf).all() and (po[:, n:] == -1).all() and (to[:, n:] == -1).all()


# --------------------------------------------------------------------------- handles that end
def test_a_handle_that_ends_inside_a_capture_leaves_it_whole(pkg):
    """One that ran on another stream than its own waits for the device when it ends, which no capture allows."""
    c = Case(torch.float16, 8, 2, 64, 16, [100, 9], [3, 1], seed=4)
    want = reference(c)
    side = torch.cuda.Stream()
    kv, old = (pkg.PagedKV(c.k, c.v, 8) for _ in range(2))
    batch = c.batch(kv)
    out, lse = torch.full_like(c.q, 7), torch.full(c.q.shape[:2], 7.0, device=DEV)
    run_attend(pkg, c, kv=old, stream=side)
    kv.attend(1, batch, c.q, out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.attend(1, batch, c.q, out, lse=lse)
        old.close()
        del old
        kv.attend(1, batch, c.q, out, lse=lse)
    out.fill_(7), lse.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    check(c, (out, lse), want)
    assert len(kv._parked) == 1
    pkg.PagedKV(c.k, c.v, 8)
    assert not kv._parked and kv.status() == 0


# --------------------------------------------------------------------------- with the decode step
@pytest.mark.parametrize("tma", [0, -1])
def test_a_window_step_takes_queries_that_append_rotated_right_before_it(pkg, tma):
    """append(q_out=q) and a WINDOW step on q, one behind the other on a stream, give what they give with a wait
    between them."""
    L, B, Hq, H, d, T, page = 24, 16, 32, 8, 128, 96, 64
    g = torch.Generator(device=DEV).manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).half()  # noqa: E731
    k, v = r(L, B, H, T, d), r(L, B, H, T, d)
    steps = []
    for _ in range(2):
        s = pkg.ConfKV(L, Hq, H, d, 64, 64, 0.5, 4, 32, 0.9, batch=B, vocab=100, max_context=T, policy=pkg.POLICY_WINDOW, attn_tma=tma)
        s.prefill(k, v, T)
        steps.append(s)
    rows = L * B
    kp, vp = (torch.zeros(1, rows // page + 1, H, page, d, dtype=torch.float16, device=DEV) for _ in range(2))
    kv = pkg.PagedKV(kp, vp, Hq)
    batch = kv.batch(ints([list(range(rows // page + 1))]), ints([0]), ints([0, rows]))
    inv = torch.rand(d // 2, generator=g, device=DEV)
    q = [torch.zeros(rows, Hq, d, dtype=torch.float16, device=DEV) for _ in range(2)]
    out = [torch.zeros(L, B, Hq, d, device=DEV) for _ in range(2)]
    for i in range(12):
        src, kn, vn = r(rows, Hq, d), r(rows, H, d), r(rows, H, d)
        for j, s in enumerate(steps):
            q[j].zero_()
            torch.cuda.synchronize()
            kv.append(0, batch, kn, vn, q=src, q_out=q[j], inv_freq=inv)
            if j:
                torch.cuda.synchronize()
            s.step(None, q[j], kn, vn, out[j])
            torch.cuda.synchronize()
        assert torch.equal(q[0], q[1]) and torch.equal(out[0], out[1]), i
    assert kv.status() == 0
