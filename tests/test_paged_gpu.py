"""Paged-cache operators against plain 64-bit forms.

Tolerances (u = half a step of the type, eps / 2: one rounding):
* attend: each probability is rounded once (u), the output once (u); scores are
  fp32 sums of head_dim products, off by at most ds = (d + 4) 2^-23 max_j scale
  sum_i |q_i k_ji| (twice fp32's bound, as tensor cores truncate), which moves a
  probability by 2 ds; sums over n keys are off by n 2^-23; fp16
  probabilities below 2^-14 of the largest are off by 2^-25 absolutely.  So
  |out - exact| <= u |out| + (u + 2 ds + n 2^-23) A + n 2^-25 max |v| (fp16),
  with A = sum p |v|;  |lse - exact| <= ds + n 2^-23 + 2^-22 (1 + |lse|).
* append: the angle's cosine and sine are off by 2^-23 (fraction rounded to 24
  bits, sincospi's 2 ulp), the products and sum by 2^-23 more, and one rounding:
  |y - exact| <= u |y| + 2^-21 (|a| + |b|).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = {torch.float16: torch.finfo(torch.float16).eps / 2, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pkg():
    import confidence_gated_kv_logits_gb300 as pkg
    pkg.load_library()
    return pkg


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Case:
    """Pools full of NaN but where the batch's tokens lie; page tables of shuffled pages."""

    def __init__(self, dt, heads, kv_heads, d, page, ctx, new, seed=0, layers=2, extra_rows=3, spare=2, room=0):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.dt, self.heads, self.H, self.d, self.page = dt, heads, kv_heads, d, page
        self.ctx, self.new, self.layers = ctx, new, layers
        blocks = [-(-(c + t + room) // page) for c, t in zip(ctx, new)]
        n = sum(blocks) + spare
        self.k = torch.full((layers, n, kv_heads, page, d), math.nan, dtype=dt, device=DEV)
        self.v = torch.full_like(self.k, math.nan)
        order = torch.randperm(n, generator=self.g, device=DEV).tolist()
        width = max(max(blocks), 1) + 1
        table = [[-1] * width for _ in ctx]
        for b, m in enumerate(blocks):
            for i in range(m):
                table[b][i] = order.pop()
        self.table = ints(table)
        self.spare = order
        self.starts = [sum(new[:b]) for b in range(len(new) + 1)]
        self.rows = self.starts[-1] + extra_rows
        for b, (c, t) in enumerate(zip(ctx, new)):
            self.put(b, 0, self.randn(layers, c + t, kv_heads, d), self.randn(layers, c + t, kv_heads, d))
        self.q = self.randn(self.rows, heads, d)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device=DEV).to(self.dt)

    def put(self, b, at, k, v):
        pos = torch.arange(at, at + k.shape[1], device=DEV)
        pg = self.table[b].long()[pos // self.page]
        self.k[:, pg, :, pos % self.page] = k.permute(1, 0, 2, 3)
        self.v[:, pg, :, pos % self.page] = v.permute(1, 0, 2, 3)

    def get(self, pool, layer, b, n):
        pos = torch.arange(n, device=DEV)
        return pool[layer, self.table[b].long()[pos // self.page], :, pos % self.page]   # [n, H, d]

    def batch(self, kv, mask=None):
        return kv.batch(self.table, ints(self.ctx), ints(self.starts), mask)


def mask_words(bits, words):
    return ints([[(x >> 32 * w & 0xFFFFFFFF) - (1 << 32) * (x >> (32 * w + 31) & 1) for w in range(words)] for x in bits])


def reference(c, layer=1, bits=None, scale=None):
    """out, lse and their tolerances for the live rows, in 64 bits."""
    n_live = c.starts[-1]
    out = torch.zeros(n_live, c.heads, c.d, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    lse = torch.zeros(n_live, c.heads, dtype=torch.float64, device=DEV)
    tol_l = torch.zeros_like(lse)
    u, g = U[c.dt], c.heads // c.H
    scale = c.d ** -0.5 if scale is None else scale
    for b, (ctx, t) in enumerate(zip(c.ctx, c.new)):
        if not t:
            continue
        n, at = ctx + t, c.starts[b]
        if bits is None:
            vis = torch.ones(t, n, dtype=torch.bool).tril(ctx)
        else:
            vis = torch.ones(t, n, dtype=torch.bool)
            vis[:, ctx:] = torch.tensor([[bool(bits[at + i] >> j & 1) for j in range(t)] for i in range(t)]).view(t, t)
        vis = vis.to(DEV)
        K, V = c.get(c.k, layer, b, n).double(), c.get(c.v, layer, b, n).double()
        # what no row sees does not matter, whatever it is; what some rows see is theirs alone
        for h in range(c.heads):
            q, k, v = c.q[at:at + t, h].double(), K[:, h // g], V[:, h // g]
            k0, v0 = torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0)
            s = torch.where(vis, q @ k0.T * scale, -math.inf)
            m = s.amax(1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            p = (s - m).exp()
            l = p.sum(1, keepdim=True)
            safe = torch.where(l == 0, torch.ones_like(l), l)
            p = p / safe
            o = p @ v0
            bad = (vis[:, :, None] & ~torch.isfinite(v)[None]).any(1) if n and not torch.isfinite(v).all() else None
            ds = (c.d + 4) * 2.0 ** -23 * scale * (torch.where(vis, q.abs() @ k0.abs().T, 0).amax(1, keepdim=True))
            A = p @ v0.abs()
            vmax = torch.where(vis[:, :, None], v0.abs()[None], 0).amax(1) if n * t * c.d < 5e7 else v0.abs().amax()
            e = u * o.abs() + (u + 2 * ds + n * 2.0 ** -23) * A
            if c.dt is torch.float16:
                e = e + n * 2.0 ** -25 * vmax
            if bad is not None:
                o = torch.where(bad, math.nan, o)
            out[at:at + t, h], tol[at:at + t, h] = o, e
            lse[at:at + t, h] = (m + l.log())[:, 0]
            tol_l[at:at + t, h] = (ds + n * 2.0 ** -23)[:, 0] + 2.0 ** -22 * (1 + lse[at:at + t, h].abs())
    return out, lse, tol, tol_l


def run_attend(pkg, c, bits=None, scale=0.0, q=None, stream=None, kv=None, layer=1, batch=None):
    kv = kv or pkg.PagedKV(c.k, c.v, c.heads)
    mask = None
    if bits is not None:
        mask = mask_words(list(bits) + [0] * (c.rows - len(bits)), max(1, -(-max(c.new) // 32)))
    out = torch.full((c.rows, c.heads, c.d), 7.0, dtype=c.dt, device=DEV)
    lse = torch.full((c.rows, c.heads), 7.0, device=DEV)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    kv.attend(layer, batch or c.batch(kv, mask), c.q if q is None else q, out, lse=lse, scale=scale, stream=stream)
    torch.cuda.synchronize()
    return out, lse, kv


def check(c, got, want):
    out, lse = got[0], got[1]
    o, l, tol, tol_l = want
    n = c.starts[-1]
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()        # rows behind the last sequence
    have = out[:n].double()
    fine = torch.isfinite(o)
    assert torch.equal(torch.isfinite(have), fine)
    assert ((have - o).abs()[fine] <= tol[fine]).all(), float(((have - o).abs()[fine] / tol[fine].clamp(min=1e-30)).max())
    have = lse[:n].double()
    dead = l == -math.inf
    assert torch.equal(have == -math.inf, dead)
    assert ((have - l).abs()[~dead] <= tol_l[~dead]).all(), float(((have - l).abs() / tol_l)[~dead].max())


def tree_bits(new, seed=0, reach=5):
    r = np.random.default_rng(seed)
    bits = []
    for t in new:
        own = []
        for i in range(t):
            p = i - 1 - int(r.integers(0, reach))
            own.append((own[p] if p >= 0 else 0) | 1 << i)
        bits += own
    return bits


SHAPES = [(2, 2, 64), (12, 12, 64), (5, 1, 128), (40, 8, 128), (16, 2, 64), (16, 1, 128), (14, 2, 128)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,kv_heads,d", SHAPES)
def test_attend_single_tokens(pkg, dt, heads, kv_heads, d):
    c = Case(DT[dt], heads, kv_heads, d, 16, [0, 1, 15, 16, 17, 63, 64, 127, 128, 300], [1] * 10, seed=heads)
    check(c, run_attend(pkg, c), reference(c))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads,d", [(40, 8, 128), (16, 2, 64)])
def test_attend_ragged_causal(pkg, dt, page, heads, kv_heads, d):
    c = Case(DT[dt], heads, kv_heads, d, page, [0, 130, 7, 0, 511, 40], [70, 3, 0, 1, 33, 129], seed=page)
    check(c, run_attend(pkg, c), reference(c))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,kv_heads,d,ctx,new", [
    (12, 12, 64, [2047], [1]), (40, 8, 128, [1500], [3]), (16, 1, 128, [700, 0, 5000, 1], [1, 0, 1, 1]),
    (24, 3, 64, [1033, 64, 0, 2500], [2, 2, 2, 1]), (40, 8, 128, [900, 17, 1024, 0, 333, 128, 1, 600], [1] * 8),
    (14, 2, 64, [600] * 33, [1] * 33)])
def test_attend_few_rows_whatever_the_tables_width(pkg, dt, heads, kv_heads, d, ctx, new, wide):
    """How units are shared among CTAs goes by how long a sequence can be: both ways, causal and with trees."""
    c = Case(DT[dt], heads, kv_heads, d, 32, ctx, new, seed=len(ctx))
    if wide:
        c.table = torch.nn.functional.pad(c.table, (0, 4000), value=-1).contiguous()
    first = run_attend(pkg, c)
    check(c, first, reference(c))
    again = run_attend(pkg, c, kv=first[2])                     # nothing depends on timing
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    bits = tree_bits(c.new, 3)
    check(c, run_attend(pkg, c, bits), reference(c, bits=bits))


def test_attend_few_rows_with_row_starts_that_overlap(pkg):
    """More rows in all than the tensors have: every sequence's own are still right (here the same for both)."""
    c = Case(torch.float16, 8, 8, 64, 16, [300, 300], [2, 2], extra_rows=0)
    c.table[1] = c.table[0]
    want = reference(c)
    kv = pkg.PagedKV(c.k, c.v, c.heads)
    out = torch.full((2, 8, 64), 7.0, dtype=c.dt, device=DEV)
    batch = kv.batch(torch.cat([c.table[:1]] * 5), ints([300] * 5), ints([0, 2, 0, 2, 0, 2]))
    kv.attend(1, batch, c.q[:2], out)
    torch.cuda.synchronize()
    assert ((out.double() - want[0][:2]).abs() <= want[2][:2]).all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,kv_heads,d", SHAPES)
def test_attend_trees(pkg, dt, heads, kv_heads, d):
    c = Case(DT[dt], heads, kv_heads, d, 32, [0, 257, 95, 64], [31, 13, 64, 65], seed=d)
    bits = tree_bits(c.new, heads)
    check(c, run_attend(pkg, c, bits), reference(c, bits=bits))


def test_attend_masks_that_leave_nothing(pkg):
    c = Case(torch.float16, 10, 2, 128, 16, [0, 20, 0], [9, 40, 1], seed=3)
    bits = tree_bits(c.new)
    bits[0] = bits[4] = bits[-1] = 0                 # nothing cached and nothing seen
    bits[9 + 3] = 0                                  # cached tokens alone
    bits[9 + 5] = 1 << 39                            # not even itself
    got = run_attend(pkg, c, bits)
    check(c, got, reference(c, bits=bits))
    assert (got[0][0] == 0).all() and (got[1][0] == -math.inf).all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("t", [5, 70])
def test_attend_what_masked_drafts_hold_does_not_matter(pkg, dt, t):
    c = Case(DT[dt], 10, 2, 64, 16, [33, 0], [t, t], seed=4)
    bits = tree_bits(c.new, 1)
    for b in range(2):
        for i, x in ((1, math.nan), (3, math.inf)):
            at = c.ctx[b] + i
            pg, s = int(c.table[b, at // 16]), at % 16
            c.v[:, pg, :, s, ::3] = x
            if i == 1:
                # a NaN key reaches only rows that see it: hide it from all
                c.k[:, pg, :, s] = x
                for r in range(c.starts[b], c.starts[b + 1]):
                    bits[r] &= ~(1 << i)
    check(c, run_attend(pkg, c, bits), reference(c, bits=bits))


@pytest.mark.parametrize("t", [1, 40, 200])
def test_attend_large_scores_and_scale(pkg, t):
    c = Case(torch.bfloat16, 8, 2, 128, 64, [500, 90], [t, t], seed=5)
    c.q *= 12
    check(c, run_attend(pkg, c, scale=0.3), reference(c, scale=float(np.float32(0.3))))


@pytest.mark.parametrize("ctx,t,heads,kv_heads,d", [
    (9000, 1, 12, 12, 64), (20000, 1, 8, 1, 128), (12000, 13, 40, 8, 128), (3000, 64, 40, 8, 128), (2500, 700, 10, 2, 128),
    (0, 1500, 16, 2, 64), (5000, 257, 5, 1, 64)])
def test_attend_long(pkg, ctx, t, heads, kv_heads, d):
    c = Case(torch.float16, heads, kv_heads, d, 64, [ctx], [t], seed=6)
    check(c, run_attend(pkg, c), reference(c))


def test_attend_many_sequences(pkg):
    r = np.random.default_rng(1)
    ctx = [int(x) for x in r.integers(0, 400, 300)]
    new = [int(x) for x in r.integers(0, 4, 300)]
    c = Case(torch.bfloat16, 8, 2, 64, 16, ctx, new, seed=7)
    check(c, run_attend(pkg, c), reference(c))


@pytest.mark.parametrize("n,most,heads,kv_heads", [(40, 30, 16, 2), (500, 6, 16, 2), (700, 2, 4, 2), (33, 200, 5, 1)])
def test_attend_more_sequences_than_lanes_or_threads(pkg, n, most, heads, kv_heads):
    r = np.random.default_rng(n)
    ctx = [int(x) for x in r.integers(0, 300, n)]
    new = [int(x) for x in r.integers(0, most + 1, n)]
    c = Case(torch.float16, heads, kv_heads, 64, 32, ctx, new, seed=n)
    check(c, run_attend(pkg, c), reference(c))
    bits = tree_bits(new, n)
    check(c, run_attend(pkg, c, bits), reference(c, bits=bits))


@pytest.mark.parametrize("heads,kv_heads,d,ctx,t", [
    (40, 8, 128, [32768], 4), (40, 8, 128, [32768], 1), (40, 8, 128, [9000] * 4, 26), (16, 2, 64, [20000, 5], 40),
    (40, 8, 128, [700, 3000], 400), (5, 1, 128, [100] * 30, 9)])
def test_attend_gives_the_same_bits_launch_after_launch(pkg, heads, kv_heads, d, ctx, t):
    c = Case(torch.bfloat16, heads, kv_heads, d, 64, ctx, [t] * len(ctx), seed=t, layers=1)
    kv = pkg.PagedKV(c.k, c.v, heads)
    batch = c.batch(kv)
    first = None
    outs = [torch.empty_like(c.q) for _ in range(4)]
    lses = [torch.empty(c.rows, heads, device=DEV) for _ in range(4)]
    for _ in range(40):
        for o, l in zip(outs, lses):
            kv.attend(0, batch, c.q, o, lse=l)
        for o, l in zip(outs, lses):
            n = c.starts[-1]
            first = first or (o[:n].clone(), l[:n].clone())
            assert torch.equal(o[:n], first[0]) and torch.equal(l[:n], first[1])
    assert kv.status() == 0


def test_two_handles_on_two_streams_over_the_same_pools(pkg):
    c = Case(torch.float16, 16, 2, 64, 32, [3000, 800], [40, 3], seed=21)
    want = reference(c)
    side = torch.cuda.Stream()
    a, b = pkg.PagedKV(c.k, c.v, 16), pkg.PagedKV(c.k, c.v, 16)
    ba, bb = c.batch(a), c.batch(b)
    one = [torch.full_like(c.q, 7) for _ in range(2)]
    lse = [torch.full((c.rows, 16), 7.0, device=DEV) for _ in range(2)]
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        a.attend(1, ba, c.q, one[0], lse=lse[0])
        b.attend(1, bb, c.q, one[1], lse=lse[1], stream=side)
    torch.cuda.synchronize()
    for i in range(2):
        check(c, (one[i], lse[i]), want)


def test_two_graphs_of_one_handle_in_turn(pkg):
    c = Case(torch.bfloat16, 40, 8, 128, 64, [5000], [20], seed=22, layers=2)
    kv = pkg.PagedKV(c.k, c.v, 40)
    batch = c.batch(kv)
    outs, graphs = [torch.empty_like(c.q) for _ in range(3)], []
    kv.attend(0, batch, c.q, outs[2])
    kv.attend(1, batch, c.q, outs[2])
    for layer in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv.attend(layer, batch, c.q, outs[layer])
        graphs.append(g)
    for _ in range(10):
        for g in graphs:
            g.replay()
        kv.attend(1, batch, c.q, outs[2])
    torch.cuda.synchronize()
    n = c.starts[-1]
    for layer in range(2):
        o, _, tol, _ = reference(c, layer=layer)
        assert ((outs[layer][:n].double() - o).abs() <= tol).all()
    assert torch.equal(outs[1][:n], outs[2][:n])


def test_attend_strided_rows_streams_and_repeats(pkg):
    c = Case(torch.float16, 10, 2, 128, 32, [700, 31, 0], [3, 60, 2], seed=8)
    wide = torch.full((c.rows, 16, 128), math.nan, dtype=c.dt, device=DEV)
    wide[:, 3:13] = c.q
    want = reference(c)
    a = run_attend(pkg, c, q=wide[:, 3:13])
    check(c, a, want)
    b = run_attend(pkg, c, stream=torch.cuda.Stream(), kv=a[2])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])      # the same on every run
    assert a[2].status() == 0


@pytest.mark.parametrize("t", [1, 64])
def test_attend_captured_and_replayed_with_other_lengths(pkg, t):
    c = Case(torch.bfloat16, 8, 2, 128, 16, [100, 900], [t, t], seed=9)
    kv = pkg.PagedKV(c.k, c.v, c.heads)
    ctx = ints(c.ctx)
    batch = kv.batch(c.table, ctx, ints(c.starts))
    out = torch.full((c.rows, c.heads, c.d), 7.0, dtype=c.dt, device=DEV)
    lse = torch.full((c.rows, c.heads), 7.0, device=DEV)
    kv.attend(1, batch, c.q, out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.attend(1, batch, c.q, out, lse=lse)
    for lens in ([100, 900], [3, 17], [0, 500]):
        c.ctx = lens
        ctx.copy_(ints(lens))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check(c, (out, lse), reference(c))


def test_attend_offsets_past_32_bits(pkg):
    dt, H, d, page = torch.float16, 1, 128, 256
    pages = (1 << 32) // (H * page * d) + 8           # the last pages lie past 2^32 elements
    k = torch.empty(1, pages, H, page, d, dtype=dt, device=DEV)
    v = torch.empty_like(k)
    c = Case(dt, 4, 1, d, page, [700], [2], seed=10, layers=1, spare=0)
    kv = pkg.PagedKV(k, v, 4)
    high = ints([[pages - 1, 3, pages - 2, -1]])
    for i, pg in enumerate((pages - 1, 3, pages - 2)):
        k[0, pg], v[0, pg] = c.k[0, int(c.table[0, i])], c.v[0, int(c.table[0, i])]
    got = run_attend(pkg, c, kv=kv, layer=0, batch=kv.batch(high, ints(c.ctx), ints(c.starts)))
    check(c, got, reference(c, layer=0))
    # and append writes there
    kk, vv = c.randn(2, 1, d), c.randn(2, 1, d)
    kv.append(0, kv.batch(high, ints([600]), ints([0, 2])), kk, vv)
    torch.cuda.synchronize()
    assert torch.equal(k[0, pages - 2, :, 88:90].transpose(0, 1), kk)
    assert torch.equal(v[0, pages - 2, :, 88:90].transpose(0, 1), vv)


def test_bad_metadata_is_flagged_and_touches_nothing(pkg):
    c = Case(torch.float16, 4, 2, 64, 16, [40, 40], [2, 2], seed=11, extra_rows=0)
    kv = pkg.PagedKV(c.k, c.v, 4)
    k0, v0 = c.k.clone(), c.v.clone()
    new = c.randn(4, 2, 64)
    for bad, flag in ((c.k.shape[1], pkg.FLAG_BAD_PAGE), (-5, pkg.FLAG_BAD_PAGE)):
        t = c.table.clone()
        t[:, 2] = bad
        kv.append(1, kv.batch(t, ints([40, 40]), ints([0, 2, 4])), new, new)
        assert kv.status(check=False) == flag and kv.status() == 0
        out = torch.empty(4, 4, 64, dtype=c.dt, device=DEV)
        kv.attend(1, kv.batch(t, ints([40, 40]), ints([0, 2, 4])), c.q, out)
        assert kv.status(check=False) == flag
    width = c.table.shape[1]
    kv.append(1, kv.batch(c.table, ints([16 * width - 1, 2 ** 31 - 1]), ints([0, 1, 4])), new, new)
    assert kv.status(check=False) & pkg.FLAG_CAPACITY
    kv.append(1, kv.batch(c.table, ints([-3, -2 ** 31]), ints([0, 2, 4])), new, new)
    assert kv.status(check=False) == pkg.FLAG_BAD_INDEX
    kv.attend(1, kv.batch(c.table, ints([-3, -2 ** 31]), ints([0, 2, 4])), c.q, out)
    assert kv.status(check=False) & pkg.FLAG_BAD_INDEX
    path = ints([[1, 1, 2], [2, 0, 1]])
    ln = torch.zeros(2, dtype=torch.int32, device=DEV)
    kv.commit(c.table, ints([40, 40]), path, ints([3, 3]), ln)
    assert kv.status(check=False) == pkg.FLAG_BAD_INDEX and ln.tolist() == [40, 40]
    kv.commit(c.table, ints([40, 40]), path, ints([4, -1]), ln)
    assert kv.status(check=False) == pkg.FLAG_BAD_INDEX and ln.tolist() == [40, 40]
    kv.commit(c.table, ints([40, 40]), ints([[0, 1000, 2000]] * 2), ints([3, 3]), ln)
    assert kv.status(check=False) == pkg.FLAG_CAPACITY
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(c.k, k0) and same(c.v, v0)


# --------------------------------------------------------------------------- append
def rotated(x, pos, inv, inter):
    x, r = x.double(), 2 * inv.shape[0]
    ang = pos.double()[:, None] * inv.double()
    z = torch.polar(torch.ones_like(ang), ang)[:, None]
    i = torch.arange(0, r, 2, device=DEV) if inter else torch.arange(r // 2, device=DEV)
    j = i + 1 if inter else i + r // 2
    y = x.clone()
    w = torch.complex(x[..., i], x[..., j]) * z
    y[..., i], y[..., j] = w.real, w.imag
    size = torch.zeros_like(x)
    size[..., i] = size[..., j] = x[..., i].abs() + x[..., j].abs()
    return y, size


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,kv_heads,d,rot,inter", [
    (12, 12, 64, 64, False), (40, 8, 128, 128, False), (5, 1, 128, 64, False), (16, 2, 64, 32, True), (7, 7, 128, 128, True),
    (3, 1, 64, 16, False), (4, 2, 64, 0, False)])
@pytest.mark.parametrize("new", [[1], [1, 0, 3, 7], [300, 0, 401]])
def test_append(pkg, dt, heads, kv_heads, d, rot, inter, new):
    dt = DT[dt]
    ctx = [13, 0, 31, 5][:len(new)]
    c = Case(dt, heads, kv_heads, d, 16, ctx, new, seed=rot + len(new))
    kv = pkg.PagedKV(c.k, c.v, heads)
    n, rows = c.starts[-1], c.rows
    wide = c.randn(rows, heads + 2 * kv_heads, d)
    q, k, v = wide[:, :heads], wide[:, heads:heads + kv_heads], wide[:, heads + kv_heads:]
    pos = torch.randint(0, 2 ** 20, (rows,), generator=c.g, device=DEV, dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    inv = (1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEV) if rot else None
    q_out = torch.full((rows, heads, d), 7.0, dtype=dt, device=DEV)
    k0, v0 = c.k.clone(), c.v.clone()
    kv.append(1, c.batch(kv), k, v, q=q, q_out=q_out, positions=pos, inv_freq=inv, interleaved=inter)
    torch.cuda.synchronize()
    assert kv.status() == 0 and (q_out[n:] == 7).all()
    empty = torch.zeros(0, device=DEV)
    for x, y in ((q[:n], q_out[:n]),
                 (k[:n], torch.cat([c.get(c.k, 1, b, a + t)[a:] for b, (a, t) in enumerate(zip(ctx, new))]))):
        want, size = rotated(x, pos[:n], inv if rot else empty, inter)
        assert ((y.double() - want).abs() <= U[dt] * want.abs() + 2.0 ** -21 * size + 2.0 ** -25).all()
    assert torch.equal(torch.cat([c.get(c.v, 1, b, a + t)[a:] for b, (a, t) in enumerate(zip(ctx, new))]), v[:n])
    # everything else is as it was
    for pool, old in ((c.k, k0), (c.v, v0)):
        for b, (a, t) in enumerate(zip(ctx, new)):
            at = torch.arange(a, a + t, device=DEV)
            pool[1, c.table[b].long()[at // 16], :, at % 16] = old[1, c.table[b].long()[at // 16], :, at % 16]
        assert torch.equal(pool.view(torch.int16), old.view(torch.int16))


def test_append_in_place_q_and_places_as_positions(pkg):
    c = Case(torch.bfloat16, 8, 2, 64, 32, [100, 7], [5, 2], seed=2)
    kv = pkg.PagedKV(c.k, c.v, 8)
    inv = torch.rand(32, generator=c.g, device=DEV)
    k, v = c.randn(c.rows, 2, 64), c.randn(c.rows, 2, 64)
    q = c.q.clone()
    kv.append(0, c.batch(kv), k, v, q=q, q_out=q, inv_freq=inv)
    torch.cuda.synchronize()
    pos = ints(list(range(100, 105)) + [7, 8])
    want, size = rotated(c.q[:7], pos, inv, False)
    assert ((q[:7].double() - want).abs() <= U[c.dt] * want.abs() + 2.0 ** -21 * size).all()
    assert torch.equal(q[7:], c.q[7:])


@pytest.mark.parametrize("new", [[1, 3], [40, 200]])
def test_pages_behind_two_to_the_31_elements(pkg, new):
    """Offsets that do not fit 32 bits: three layers of 2^30 elements each, the work in the last one."""
    c = Case(torch.float16, 4, 2, 64, 256, [300, 1000], new, layers=3, spare=2 ** 15 - 20, seed=31)
    assert c.k.numel() > 2 ** 31 and c.k[:2].numel() * 2 > 2 ** 31
    kv = pkg.PagedKV(c.k, c.v, 4)
    n = c.starts[-1]
    k, v = c.randn(c.rows, 2, 64), c.randn(c.rows, 2, 64)
    kv.append(2, c.batch(kv), k, v)
    torch.cuda.synchronize()
    assert torch.equal(torch.cat([c.get(c.k, 2, b, a + t)[a:] for b, (a, t) in enumerate(zip(c.ctx, new))]), k[:n])
    check(c, run_attend(pkg, c, layer=2, kv=kv), reference(c, layer=2))
    path, new_len = ints([[new[0] - 1], [new[1] - 1]]), ints([0, 0])
    kv.commit(c.table, ints(c.ctx), path, ints([1, 1]), new_len)
    tails = ints(c.spare[:2])
    out, lens = torch.full_like(c.table, -1), ints([0, 0])
    kv.fork(ints([1, 0]), 2, c.table, new_len, tails, out, lens)
    torch.cuda.synchronize()
    assert kv.status() == 0 and lens.tolist() == [1001, 301]
    for b in range(2):
        assert torch.equal(c.get(c.v, 2, b, c.ctx[b] + 1)[-1], v[c.starts[b] + new[b] - 1])
        fill = c.ctx[b] % 256 + 1
        assert torch.equal(c.k[2, tails[1 - b], :, :fill], c.k[2, c.table[b, c.ctx[b] // 256], :, :fill])


def test_attend_lse_may_not_overlap(pkg):
    c = Case(torch.float16, 8, 2, 64, 16, [5], [4], extra_rows=0)
    kv = pkg.PagedKV(c.k, c.v, 8)
    out = torch.empty_like(c.q)
    for t in (out, c.q):
        with pytest.raises(pkg.ConfKVError):
            kv.attend(0, c.batch(kv), c.q, out, lse=t.view(torch.float32).flatten()[:32].view(4, 8))


def test_python_refusals(pkg):
    c = Case(torch.float16, 8, 2, 64, 16, [5], [4], extra_rows=0)
    kv = pkg.PagedKV(c.k, c.v, 8)
    b = c.batch(kv)
    k, v = c.randn(4, 2, 64), c.randn(4, 2, 64)
    out = torch.empty_like(c.q)
    E = (ValueError, pkg.ConfKVError)
    for f in (lambda: kv.attend(2, b, c.q, out), lambda: kv.attend(-1, b, c.q, out),
              lambda: kv.attend(0, b, c.q.bfloat16(), out), lambda: kv.attend(0, b, c.q.cpu(), out),
              lambda: kv.attend(0, b, c.q, out[:3]), lambda: kv.attend(0, b, c.q, c.q),
              lambda: kv.attend(0, b, c.q, out, scale=-1.0), lambda: kv.attend(0, b, c.q, out, scale=math.nan),
              lambda: kv.attend(0, b, c.q, out, lse=torch.empty(4, 8, dtype=torch.float64, device=DEV)),
              lambda: kv.attend(0, b, c.q.transpose(0, 1), out),
              lambda: kv.append(0, b, k, v, q=c.q), lambda: kv.append(0, b, k, v[:2]),
              lambda: kv.append(0, b, k, v, inv_freq=torch.rand(12, device=DEV)),
              lambda: kv.append(0, b, k, v, inv_freq=torch.rand(40, device=DEV)),
              lambda: kv.append(0, b, k, v, positions=torch.zeros(4, dtype=torch.int64, device=DEV)),
              lambda: kv.append(0, b, k, v, q=c.q[:, :4], q_out=out[:, :4]),
              lambda: kv.batch(c.table.long(), ints([5]), ints([0, 4])), lambda: kv.batch(c.table, ints([5]), ints([0])),
              lambda: kv.batch(c.table, ints([5]), ints([0, 4]), torch.zeros(4, device=DEV)),
              lambda: kv.attend(0, kv.batch(c.table, ints([5]), ints([0, 4]), ints([[1]] * 3)), c.q, out),
              lambda: kv.attend(0, b, c.q[:, :, :32], out), lambda: kv.commit(c.table, ints([5]), ints([[0]]), ints([1, 1]), ints([0])),
              lambda: pkg.BeamSelect(1, 33, 100, 4), lambda: pkg.BeamSelect(1, 4, 100, 4, dtype=torch.float64),
              lambda: pkg.BeamSelect(1, 4, 100, 4).select(torch.zeros(1, 4, 99, device=DEV), *[torch.zeros(1, 4, device=DEV)] * 2,
                                                          ints([[0] * 4]), ints([[0] * 4])),
              lambda: pkg.PagedKV(c.k, c.v.bfloat16(), 8), lambda: pkg.PagedKV(c.k, c.v, 9),
              lambda: pkg.PagedKV(c.k.float(), c.v.float(), 8), lambda: pkg.PagedKV(c.k[:, 1:], c.v[:, 1:], 8)):
        with pytest.raises(E):
            f()
    lens = ints([5])
    with pytest.raises(E):
        kv.commit(c.table, lens, ints([[0]]), ints([1]), lens)
    with pytest.raises(E):
        kv.fork(ints([0]), 1, c.table, lens, ints([1]), c.table, ints([0]))
    with pytest.raises(E):
        kv.fork(ints([0]), 2, c.table, lens, ints([1]), c.table.clone(), ints([0]))


# --------------------------------------------------------------------------- commit, fork
@pytest.mark.parametrize("heads,kv_heads,d,page", [(12, 12, 64, 16), (40, 8, 128, 32), (4, 1, 64, 64)])
def test_commit(pkg, heads, kv_heads, d, page):
    paths = [[0, 1, 2], [2, 3, 9, 11, 12, 13, 14, 15, 16, 17, 20], [], [5], [0, 2, 3, 4], list(range(1, 22))]
    ctx = [0, 13, 40, 63, 5, 100]
    c = Case(torch.bfloat16, heads, kv_heads, d, page, ctx, [22] * 6, layers=3)
    kv = pkg.PagedKV(c.k, c.v, heads)
    want_k, want_v = c.k.clone(), c.v.clone()
    for b, p in enumerate(paths):
        for pool, w in ((c.k, want_k), (c.v, want_v)):
            for j, x in enumerate(p):
                f, t = ctx[b] + x, ctx[b] + j
                w[:, int(c.table[b, t // page]), :, t % page] = pool[:, int(c.table[b, f // page]), :, f % page]
    cap = max(map(len, paths))
    new_len = torch.zeros(6, dtype=torch.int32, device=DEV)
    kv.commit(c.table, ints(ctx), ints([p + [-1] * (cap - len(p)) for p in paths]), ints([len(p) for p in paths]), new_len)
    torch.cuda.synchronize()
    assert kv.status() == 0
    assert new_len.tolist() == [a + len(p) for a, p in zip(ctx, paths)]
    assert torch.equal(c.k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(c.v.view(torch.int16), want_v.view(torch.int16))


@pytest.mark.parametrize("kv_heads,d,page,length", [(12, 64, 16, 39), (8, 128, 64, 64), (1, 64, 32, 5), (2, 128, 128, 255), (2, 64, 16, 0)])
def test_fork(pkg, kv_heads, d, page, length):
    W, B = 4, 3
    L, blocks = 2, length // page + 2
    g = torch.Generator(device=DEV).manual_seed(length)
    n = B * (blocks + 2 * W)
    k = torch.randn(L, n, kv_heads, page, d, generator=g, device=DEV).half()
    v = torch.randn(L, n, kv_heads, page, d, generator=g, device=DEV).half()
    pages = torch.randperm(n, generator=g, device=DEV).tolist()
    full, fill = divmod(length, page)
    table = []
    for b in range(B):
        shared = [pages.pop() for _ in range(full)]
        table += [shared + ([pages.pop()] if fill else []) + [-1] * (blocks - full - (1 if fill else 0)) for _ in range(W)]
    tails = [pages.pop() for _ in range(B * W)]
    parent = [1, 0, 3, 3, -1, 0, 0, 0, 2, 2, -1, 1]
    want_k, want_v, want_t = k.clone(), v.clone(), [[-9] * blocks for _ in range(B * W)]
    for r, p in enumerate(parent):
        src = r if p < 0 else r // W * W + p
        want_t[r][:full] = table[src][:full]
        if fill:
            want_t[r][full] = tails[r]
            for pool, w in ((k, want_k), (v, want_v)):
                w[:, tails[r], :, :fill] = pool[:, table[src][full], :, :fill]
    kv = pkg.PagedKV(k, v, kv_heads)
    out, lens = ints([[-9] * blocks] * (B * W)), torch.zeros(B * W, dtype=torch.int32, device=DEV)
    kv.fork(ints(parent), W, ints(table), ints([length] * (B * W)), ints(tails), out, lens)
    torch.cuda.synchronize()
    assert kv.status() == 0 and lens.tolist() == [length] * (B * W)
    assert out.tolist() == want_t and torch.equal(k, want_k) and torch.equal(v, want_v)


def test_fork_onto_the_parents_own_page_and_bad_parents(pkg):
    c = Case(torch.float16, 2, 2, 64, 16, [20, 20], [0, 0], layers=1)
    kv = pkg.PagedKV(c.k, c.v, 2)
    k0 = c.k.clone()
    tails = c.table[:, 1].contiguous()
    out, lens = torch.full_like(c.table, -9), ints([0, 0])
    kv.fork(ints([0, 1]), 2, c.table, ints([20, 20]), tails, out, lens)     # each keeps its own page
    assert kv.status() == 0 and torch.equal(out[:, :2], c.table[:, :2])
    kv.fork(ints([2, -2]), 2, c.table, ints([20, 20]), tails, out, lens)    # no such parents: their own
    assert kv.status(check=False) == pkg.FLAG_BAD_INDEX
    kv.fork(ints([0, 1]), 2, c.table, ints([20, 20]), ints([99, -1]), out, lens)
    assert kv.status(check=False) == pkg.FLAG_BAD_PAGE
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16))


# --------------------------------------------------------------------------- select
def select_reference(z, scores, finished, keep, pad):
    """Scores in 64 bits, ordered by (score, lower beam and token)."""
    B, W, V = z.shape
    res = []
    for b in range(B):
        found = []
        for w in range(W):
            s = float(scores[b, w])
            if not math.isfinite(s):
                continue
            if finished is not None and finished[b, w]:
                found.append((s, w, pad))
                continue
            x = z[b, w].double()
            if torch.isnan(x).any() or (x == math.inf).any() or not (x > -math.inf).any():
                continue
            lp = (x - torch.logsumexp(x, 0)).tolist()
            found += [(s + a, w, v) for v, a in enumerate(lp) if a > -math.inf]
        found.sort(key=lambda f: (-f[0], f[1], f[2]))
        res.append((found + [(-math.inf, -1, -1)] * keep)[:keep])
    return res


def run_select(pkg, z, scores, keep, finished=None, pad=0, sel=None):
    B, W, V = z.shape
    sel = sel or pkg.BeamSelect(B, W, V, keep, dtype=z.dtype)
    so = torch.full((B, keep), 7.0, device=DEV)
    po, to = torch.full((B, keep), 7, dtype=torch.int32, device=DEV), torch.full((B, keep), 7, dtype=torch.int32, device=DEV)
    fl = torch.full((B, W), 7, dtype=torch.int32, device=DEV)
    sel.select(z, scores, so, po, to, finished=finished, pad_token=pad, flags_out=fl)
    torch.cuda.synchronize()
    return so, po, to, fl, sel


def check_select(got, want):
    so, po, to = (x.cpu().tolist() for x in got[:3])
    for b, rows in enumerate(want):
        assert po[b] == [r[1] for r in rows] and to[b] == [r[2] for r in rows], b
        for x, r in zip(so[b], rows):
            # the sum's error (exponentials 2^-22, sums in double) and one fp32 rounding
            assert x == r[0] or abs(x - r[0]) <= 2.0 ** -21 + 2.0 ** -24 * abs(r[0]), (x, r)


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,W,V,keep", [(1, 1, 2, 1), (1, 4, 1000, 8), (3, 5, 4099, 10), (2, 32, 777, 64), (1, 3, 50257, 33),
                                        (9, 8, 33000, 16), (2, 1, 7, 64)])
def test_select(pkg, dt, B, W, V, keep):
    g = torch.Generator(device=DEV).manual_seed(V)
    z = (3 * torch.randn(B, W, V, generator=g, device=DEV)).to(dt)
    z[..., :: max(2, V // 5)] = -math.inf
    z[..., 1] = 0.5
    scores = -3 * torch.rand(B, W, generator=g, device=DEV)
    fin = torch.rand(B, W, generator=g, device=DEV) < 0.3
    got = run_select(pkg, z, scores, keep)
    check_select(got, select_reference(z.cpu(), scores.cpu(), None, keep, 0))
    assert not got[3].any()
    got = run_select(pkg, z, scores, keep, fin, V - 1, got[4])                 # the same scratch again
    check_select(got, select_reference(z.cpu(), scores.cpu(), fin.cpu(), keep, V - 1))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [640, 9001, 70001])
def test_select_ties_and_orders(pkg, dt, V):
    keep = 12
    z = torch.zeros(2, 3, V, device=DEV)
    z[1] = torch.linspace(8, -8, V, device=DEV)          # long runs of equal values in bf16, sorted
    z[1, 1] = z[1, 0].flip(0)
    z[1, 2, ::2] = -0.0
    z = z.to(dt)
    scores = torch.tensor([[0.0, 0.0, 0.0], [-1.0, -1.0, -0.5]], device=DEV)
    check_select(run_select(pkg, z, scores, keep), select_reference(z.cpu(), scores.cpu(), None, keep, 0))
    scores = torch.tensor([[0.0, -math.inf, -math.inf], [-math.inf] * 3], device=DEV)     # a first step, a dead sequence
    check_select(run_select(pkg, z, scores, keep), select_reference(z.cpu(), scores.cpu(), None, keep, 0))


def test_select_leaves_bad_rows_out(pkg):
    z = torch.randn(2, 4, 500, device=DEV)
    z[0, 0, 17] = math.nan
    z[0, 1, 3] = math.inf
    z[0, 2] = -math.inf
    z[1, :, 1:] = -math.inf                             # one candidate each
    scores = torch.zeros(2, 4, device=DEV)
    scores[1, 2] = math.nan
    scores[1, 3] = math.inf
    got = run_select(pkg, z, scores, 6)
    check_select(got, select_reference(z.cpu(), scores.cpu(), None, 6, 0))
    N = pkg.FLAG_NONFINITE
    assert got[3].tolist() == [[N, N, N, 0], [0, 0, N, N]]


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
def test_select_a_nan_among_masked_tokens(pkg, dt):
    """A NaN in a part of the vocabulary that is masked out otherwise, or wholly NaN, far from the finite logits."""
    V = 70001
    z = torch.full((1, 4, V), -math.inf, device=DEV)
    z[..., :50] = torch.linspace(-1, 1, 50, device=DEV)
    z[0, 1, V - 1] = math.nan
    z[0, 2, 100:] = math.nan
    z = z.to(dt)
    scores = torch.zeros(1, 4, device=DEV)
    got = run_select(pkg, z, scores, 6)
    check_select(got, select_reference(z.cpu(), scores.cpu(), None, 6, 0))
    assert got[3].tolist() == [[0, pkg.FLAG_NONFINITE, pkg.FLAG_NONFINITE, 0]]


def test_select_strided_rows_and_replay(pkg):
    B, W, V, keep = 2, 4, 5001, 8
    wide = torch.randn(B * W, V + 13, device=DEV).to(torch.float16)
    z = wide[:, :V].unflatten(0, (B, W))
    scores = -torch.rand(B, W, device=DEV)
    got = run_select(pkg, z, scores, keep)
    check_select(got, select_reference(z.cpu(), scores.cpu(), None, keep, 0))
    sel, so, po, to = got[4], *(torch.empty_like(x) for x in got[:3])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sel.select(z, scores, so, po, to)
    for i in range(3):
        scores.copy_(-torch.rand(B, W, device=DEV) * (i + 1))
        wide.copy_(torch.randn_like(wide))
        g.replay()
        torch.cuda.synchronize()
        check_select((so, po, to), select_reference(z.cpu(), scores.cpu(), None, keep, 0))


# --------------------------------------------------------------------------- together
@pytest.mark.parametrize("dt", list(DT))
def test_a_prompt_in_chunks_a_tree_and_its_accepted_path(pkg, dt):
    """Chunks of a prompt, then drafted trees whose accepted path is kept, give at each step what attention over the
    sequence's own tokens, rotated at their positions, gives."""
    dt = DT[dt]
    heads, H, d, page, B = 10, 2, 64, 16, 2
    g = torch.Generator(device=DEV).manual_seed(0)
    inv = (1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().to(DEV)
    c = Case(dt, heads, H, d, page, [0, 0], [0, 0], layers=1, spare=40)
    kv = pkg.PagedKV(c.k, c.v, heads)
    c.table = ints([[c.spare.pop() for _ in range(16)] for _ in range(B)])
    lens = ints([0, 0])
    told = [([], []) for _ in range(B)]                # each sequence's kept (k, v) rows, as the cache must hold them

    def step(new, pos, bits=None):
        n = sum(new)
        qkv = torch.randn(n, heads + 2 * H, d, generator=g, device=DEV).to(dt)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + H], qkv[:, heads + H:]
        c.new, c.starts, c.rows, c.ctx = new, [0, new[0], n], n, lens.tolist()
        mask = mask_words(bits, -(-max(new) // 32)) if bits else None
        b = kv.batch(c.table, lens, ints(c.starts), mask)
        c.q = torch.empty(n, heads, d, dtype=dt, device=DEV)
        kv.append(0, b, k, v, q=q, q_out=c.q, positions=ints(pos), inv_freq=inv)
        out, lse, _ = run_attend(pkg, c, kv=kv, layer=0, batch=b)
        check(c, (out, lse), reference(c, layer=0, bits=bits))
        return [(c.get(c.k, 0, i, c.ctx[i] + t)[c.ctx[i]:], v[s:s + t]) for i, (s, t) in enumerate(zip(c.starts, new))]

    for new in ([40, 7], [33, 64], [1, 1]):
        at = lens.tolist()
        rows = step(new, [a + i for a, t in zip(at, new) for i in range(t)])
        for i, (k, v) in enumerate(rows):
            told[i][0].append(k)
            told[i][1].append(v)
        lens.add_(ints(new))
    for turn in range(3):
        new = [20, 35]
        bits = tree_bits(new, turn)
        pos = [a + bin(x).count("1") - 1 for a, s, t in zip(lens.tolist(), (0, 20), new) for x in bits[s:s + t]]
        rows = step(new, pos, bits)
        leaf = [17, 30]
        path = [[j for j in range(t) if bits[s + l] >> j & 1] for s, t, l in zip((0, 20), new, leaf)]
        cap = max(map(len, path))
        out = torch.empty_like(lens)
        kv.commit(c.table, lens, ints([p + [0] * (cap - len(p)) for p in path]), ints([len(p) for p in path]), out)
        for i, (k, v) in enumerate(rows):
            told[i][0].append(k[path[i]])
            told[i][1].append(v[path[i]])
        lens = out
    assert kv.status() == 0
    for i in range(B):
        n = int(lens[i])
        assert torch.equal(c.get(c.k, 0, i, n), torch.cat(told[i][0]))
        assert torch.equal(c.get(c.v, 0, i, n), torch.cat(told[i][1]))


def test_a_beam_search_over_shared_pages(pkg):
    """Beams that share a prompt's pages, reordered after every selection, attend to their own histories."""
    dt, heads, H, d, page, B, W, V = torch.float16, 4, 2, 64, 16, 2, 3, 300
    g = torch.Generator(device=DEV).manual_seed(5)
    k, v = (torch.full((1, 200, H, page, d), math.nan, dtype=dt, device=DEV) for _ in range(2))
    kv = pkg.PagedKV(k, v, heads)
    sel = pkg.BeamSelect(B, W, V, W)
    free = list(range(200))
    prompt, n = 37, B * W
    hist = []
    table = ints([[-1] * 8] * n)
    for b in range(B):
        rows = torch.randn(prompt, 2 * H, d, generator=g, device=DEV).to(dt)
        first = [free.pop() for _ in range(3)]
        kv.append(0, kv.batch(ints([first]), ints([0]), ints([0, prompt])), rows[:, :H], rows[:, H:])
        for w in range(W):
            table[b * W + w, :3] = ints(first)
            hist.append(rows)
    lens = ints([prompt] * n)
    scores = torch.tensor([[0.0] + [-math.inf] * (W - 1)] * B, device=DEV)
    so, po, to = torch.empty(B, W, device=DEV), ints([[0] * W] * B), ints([[0] * W] * B)
    for step in range(14):                              # crosses page borders at 48 tokens
        z = 2 * torch.randn(B, W, V, generator=g, device=DEV)
        sel.select(z, scores, so, po, to)
        check_select((so, po, to), select_reference(z.cpu(), scores.cpu(), None, W, 0))
        new_table, new_lens = torch.full_like(table, -1), torch.empty_like(lens)
        length = prompt + step
        tails = [free.pop(0) for _ in range(n)]         # never one that is in use: this test frees none
        kv.fork(po, W, table, lens, ints(tails), new_table, new_lens)
        table, lens, scores = new_table, new_lens, so.clone()
        hist = [hist[r // W * W + p] for r, p in enumerate(po.view(-1).tolist())]
        if length % page == 0:
            table[:, length // page] = ints([free.pop(0) for _ in range(n)])
        qkv = torch.randn(n, heads + 2 * H, d, generator=g, device=DEV).to(dt)
        batch = kv.batch(table, lens, ints(list(range(n + 1))))
        kv.append(0, batch, qkv[:, heads:heads + H], qkv[:, heads + H:])
        hist = [torch.cat([h, qkv[r:r + 1, heads:]]) for r, h in enumerate(hist)]
        out = torch.empty(n, heads, d, dtype=dt, device=DEV)
        kv.attend(0, batch, qkv[:, :heads], out)
        lens.add_(0)
        for r in range(n):
            kk, vv = hist[r][:, :H].double(), hist[r][:, H:].double()
            for h in range(heads):
                p = torch.softmax(kk[:, h // 2] @ qkv[r, h].double() * d ** -0.5, 0)
                want = p @ vv[:, h // 2]
                assert ((out[r, h].double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -10 * (p @ vv[:, h // 2].abs()) + 1e-5).all()
        lens = lens + 1
    assert kv.status() == 0
