"""Normed appends with several position axes, attention over shared prefixes, accumulated
attention weights and eviction by them, against plain 64-bit forms.

Tolerances (u: half a step of the type, one rounding):
* append: the sum of squares adds up to 20 positive fp32 terms in a row (2^-24 each,
  half of it in the root), rsqrt is good to 2^-22, the products with it and the
  weight to 2^-24 each: a normed value is off by 2^-20 relative.  The sines and
  the rotation add 2^-21 (|a| + |b|) of the normed pair (test_paged_gpu.py), so
  |y - exact| <= u |y| + 2^-19 (|a| + |b|).  Below the type's smallest normal number
  a step is smallest_normal * eps whatever the value is: a rounding loses up to half of
  it (fp16 2^-25, bf16 2^-126 2^-7 / 2 = 2^-134), and fp32's roundings before it, where
  bf16's range is fp32's, 2^-150 each (norm's product, weight's, the rotation's four).
* attend over a prefix: as in test_paged_gpu.py, and the join's two factors
  (2^-22 each), products and sum (2^-24 each): 2^-20 max |v| in all, 2^-20 of lse's sum.
* weigh: a score is off by ds = (d + 4) 2^-23 max_t scale sum |q k_t| (fp32 sums of
  products, twice fp32's bound as tensor cores truncate), its difference to lse and the
  product with log2 e by 2^-22 (|s| + |lse|), exp2 by 2^-22, and sums of R rows by R 2^-24
  relative (all terms positive): a weight w by w (2 ds + 2^-21 (1 + |s| + |lse|) + R 2^-24); then
  decay mass + gain sum by 2^-22 relative.  Weights below fp32's normal range (2^-126) are flushed.
* evict: whole numbers and copies, equal.
"""
import math

import numpy as np
import pytest
import torch

from tests.test_paged_gpu import DT, U, Case, ints, mask_words, reference, tree_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkg():
    import confidence_gated_kv_logits_gb300 as pkg
    pkg.load_library()
    return pkg


# ---------------------------------------------------------------------------
# append with norms and axes
# ---------------------------------------------------------------------------
def normed(x, w, eps):
    x = x.double()
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(2, keepdim=True) + eps) * w.double()


def turned(x, angle, r, inter):
    """The rotated rows and the size of each channel's pair."""
    size, y = x.abs(), x.clone()
    if r:
        even = torch.arange(0, r, 2) if inter else torch.arange(r // 2)
        odd = even + (1 if inter else r // 2)
        a, b = x[:, :, even], x[:, :, odd]
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        y[:, :, even], y[:, :, odd] = a * c - b * s, b * c + a * s
        size[:, :, even] = size[:, :, odd] = a.abs() + b.abs()
    return y, size


def check_append(pkg, c, r, inter, axes, wq, wk, eps=1e-6, q=None, k=None, strided=False, in_place=False):
    kv = pkg.PagedKV(c.k, c.v, c.heads)
    n = c.rows
    q = c.randn(n, c.heads, c.d) if q is None else q
    k = c.randn(n, c.H, c.d) if k is None else k
    v = c.randn(n, c.H, c.d)
    if strided:
        row = torch.zeros(n, c.heads + 2 * c.H + 1, c.d, dtype=c.dt, device=DEV)
        for x, at in ((q, 0), (k, c.heads), (v, c.heads + c.H)):
            row[:, at:at + x.shape[1]] = x
        q, k, v = row[:, :c.heads], row[:, c.heads:c.heads + c.H], row[:, c.heads + c.H:-1]
    q_in, q_out = q.clone(), q if in_place else torch.full_like(q.contiguous(), 7)
    pos = axis = inv = None
    angle = None
    if r:
        inv = (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()
        shape = (n, axes) if axes else (n,)
        pos = torch.randint(0, 1 << 20, shape, generator=c.g, device=DEV, dtype=torch.int32)
        axis = torch.randint(0, axes, (r // 2,), generator=c.g, device=DEV, dtype=torch.int32) if axes else None
        p = pos.double()[:, axis.long()] if axes else pos.double()[:, None]
        angle = p * inv.double()
    k0, v0 = c.k.clone(), c.v.clone()
    kv.append(1, c.batch(kv), k, v, q=q, q_out=q_out, positions=pos, inv_freq=inv, interleaved=inter, q_norm=wq, k_norm=wk,
              eps=eps, axis=axis)
    torch.cuda.synchronize()
    live = c.starts[-1]
    u = U[c.dt]
    low = torch.finfo(c.dt).smallest_normal * torch.finfo(c.dt).eps / 2
    for x, w, name in ((q_in, wq, "q"), (k, wk, "k")):
        y, size = turned(normed(x, w, eps), angle, r, inter)
        tol = u * y.abs() + 2.0 ** -19 * size + low + 6 * 2.0 ** -150
        if name == "q":
            assert ((q_out[:live].double() - y[:live]).abs() <= tol[:live]).all()
            if not in_place:
                assert (q_out[live:] == 7).all()
            else:
                assert torch.equal(q_out[live:], q_in[live:])
            continue
        for b, (ctx, t) in enumerate(zip(c.ctx, c.new)):
            if t:
                rows, place = slice(c.starts[b], c.starts[b] + t), torch.arange(ctx, ctx + t, device=DEV)
                pg, at = c.table[b].long()[place // c.page], place % c.page
                assert ((c.k[1, pg, :, at].double() - y[rows]).abs() <= tol[rows]).all()
                assert torch.equal(c.v[1, pg, :, at], v[rows])
                for pool, old in ((c.k, k0), (c.v, v0)):
                    old[1, pg, :, at] = pool[1, pg, :, at]
    for pool, old in ((c.k, k0), (c.v, v0)):        # nothing else was touched
        assert torch.equal(pool.view(torch.int16), old.view(torch.int16))
    assert kv.status() == 0


def some_weights(c, dtype):
    return [(1 + 0.3 * torch.randn(c.d, generator=c.g, device=DEV)).to(dtype) for _ in range(2)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,kv_heads,d", [(2, 2, 64), (40, 8, 128), (7, 1, 64), (5, 1, 128), (64, 8, 64)])
@pytest.mark.parametrize("part,inter,axes", [(1, False, 3), (1, True, 0), (2, False, 0), (4, True, 4), (0, False, 0)])
def test_append_normed(pkg, dt, heads, kv_heads, d, part, inter, axes):
    c = Case(DT[dt], heads, kv_heads, d, 32, [0, 5, 31, 100], [3, 0, 40, 1], seed=heads + axes)
    wq, wk = some_weights(c, torch.float32 if inter else DT[dt])
    check_append(pkg, c, d // part if part else 0, inter, axes, wq, wk, strided=part == 1, in_place=part == 2)


@pytest.mark.parametrize("which", ["q", "k", "neither", "axes"])
def test_append_normed_one_of_both(pkg, which):
    c = Case(torch.bfloat16, 10, 2, 128, 16, [0, 77], [9, 2], seed=3)
    wq, wk = some_weights(c, torch.bfloat16)
    check_append(pkg, c, 64, False, 2 if which in ("neither", "axes") else 0, wq if which == "q" else None, wk if which == "k" else None)


def test_append_axes_alike_are_one_position(pkg):
    """With the same position on every axis and no weights the rows are append's own, bit for bit."""
    c = Case(torch.float16, 8, 2, 128, 16, [3], [50], seed=5, extra_rows=0)
    kv = pkg.PagedKV(c.k, c.v, 8)
    q, k, v = c.randn(50, 8, 128), c.randn(50, 2, 128), c.randn(50, 2, 128)
    inv = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).float().cuda()
    pos = torch.randint(-(1 << 30), 1 << 30, (50,), device=DEV, dtype=torch.int32)
    out = [torch.zeros_like(q) for _ in range(2)]
    kv.append(0, c.batch(kv), k, v, q=q, q_out=out[0], positions=pos, inv_freq=inv)
    kv.append(1, c.batch(kv), k, v, q=q, q_out=out[1], positions=pos[:, None].repeat(1, 3), inv_freq=inv,
              axis=(torch.arange(64, device=DEV) % 3).int())
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1])
    assert torch.equal(c.get(c.k, 0, 0, 53)[3:], c.get(c.k, 1, 0, 53)[3:])


@pytest.mark.parametrize("dt", list(DT))
def test_append_normed_extremes(pkg, dt):
    """Zeros, the type's largest and smallest values, single outliers: the root mean square keeps its range."""
    c = Case(DT[dt], 4, 4, 64, 16, [0], [8], seed=6, extra_rows=0)
    x = c.randn(8, 4, 64)
    x[0] = 0
    x[1] = torch.finfo(DT[dt]).max
    x[2] = torch.finfo(DT[dt]).tiny
    x[3, :, 7] = torch.finfo(DT[dt]).max
    x[4] *= 1e-3
    x[5] = 0
    x[5, :, 3] = 1
    x[6] = -torch.finfo(DT[dt]).max * (torch.rand(4, 64, generator=c.g, device=DEV) < 0.5).to(DT[dt])
    wq, wk = some_weights(c, DT[dt])
    check_append(pkg, c, 64, False, 0, wq, wk, q=x, k=x.flip(0).contiguous())


def test_append_normed_nan_stays_in_its_head(pkg):
    c = Case(torch.bfloat16, 8, 8, 64, 16, [0], [3], seed=7, extra_rows=0)
    kv = pkg.PagedKV(c.k, c.v, 8)
    q = c.randn(3, 8, 64)
    q[1, 2, 5], q[2, 3, 6] = math.nan, math.inf
    wq, wk = some_weights(c, torch.float32)
    out = torch.zeros_like(q)
    kv.append(0, c.batch(kv), c.randn(3, 8, 64), c.randn(3, 8, 64), q=q, q_out=out, q_norm=wq, k_norm=wk)
    torch.cuda.synchronize()
    assert out[1, 2].isnan().all() and out[2, 3, 6].isnan()
    out[1, 2], out[2, 3] = 0, 0
    assert torch.isfinite(out).all()


def test_append_bad_axis_is_flagged(pkg):
    c = Case(torch.float16, 4, 4, 64, 16, [0], [4], seed=8, extra_rows=0)
    kv = pkg.PagedKV(c.k, c.v, 4)
    q = c.randn(4, 4, 64)
    out = torch.zeros_like(q)
    inv = torch.ones(32, device=DEV)
    axis = torch.zeros(32, device=DEV, dtype=torch.int32)
    axis[3], axis[31] = 2, -1
    kv.append(0, c.batch(kv), c.randn(4, 4, 64), c.randn(4, 4, 64), q=q, q_out=out, inv_freq=inv,
              positions=torch.full((4, 2), 5, device=DEV, dtype=torch.int32), axis=axis)
    assert kv.status(check=False) == 16
    for i in (3, 31):
        assert torch.equal(out[..., i], q[..., i]) and torch.equal(out[..., 32 + i], q[..., 32 + i])
    assert not torch.equal(out[..., 4], q[..., 4])


# ---------------------------------------------------------------------------
# attention over shared prefixes
# ---------------------------------------------------------------------------
class Grouped(Case):
    """Groups of sequences with a prefix in common: (sequences, prefix) each; own tokens behind it."""

    def __init__(self, dt, heads, kv_heads, d, page, groups, tail, new, **kw):
        ctx = [p + tail[i % len(tail)] for i, p in enumerate([p for n, p in groups for _ in range(n)])]
        rows = [new[i % len(new)] for i in range(len(ctx))]
        super().__init__(dt, heads, kv_heads, d, page, ctx, rows, **kw)
        self.sizes, self.prefixes = [n for n, _ in groups], [p for _, p in groups]
        b = 0
        for n, p in groups:
            full, at = p // page, torch.arange(p, device=DEV)
            for i in range(b + 1, b + n):
                rest = at[full * page:]
                for pool in (self.k, self.v):
                    src = pool[:, self.table[b].long()[rest // page], :, rest % page]
                    pool[:, self.table[i].long()[rest // page], :, rest % page] = src
                if full:
                    for pool in (self.k, self.v):       # the pages that it had are free
                        pool[:, self.table[i, :full].long()] = math.nan
                    self.table[i, :full] = self.table[b, :full]
            b += n

    def starts_of_groups(self):
        return ints([sum(self.sizes[:i]) for i in range(len(self.sizes) + 1)])


def run_shared(pkg, c, bits=None, kv=None, prefix=None, scale=0.0, layer=1):
    kv = kv or pkg.PagedKV(c.k, c.v, c.heads)
    mask = None
    if bits is not None:
        mask = mask_words(list(bits) + [0] * (c.rows - len(bits)), max(1, -(-max(c.new) // 32)))
    prefix = prefix or kv.prefix(c.starts_of_groups(), ints(c.prefixes), c.rows)
    out = torch.full((c.rows, c.heads, c.d), 7.0, dtype=c.dt, device=DEV)
    lse = torch.full((c.rows, c.heads), 7.0, device=DEV)
    kv.attend(layer, c.batch(kv, mask), c.q, out, lse=lse, scale=scale, prefix=prefix)
    torch.cuda.synchronize()
    return out, lse, kv


def check_shared(c, got, want):
    out, lse = got[0], got[1]
    o, l, tol, tol_l = want
    n = c.starts[-1]
    vmax = float(torch.nan_to_num(c.v.double(), 0, 0, 0).abs().max())
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    have, fine = out[:n].double(), torch.isfinite(o)
    assert torch.equal(torch.isfinite(have), fine)
    assert ((have - o).abs()[fine] <= tol[fine] + 2.0 ** -20 * vmax).all()
    dead = l == -math.inf
    assert torch.equal(lse[:n] == -math.inf, dead)
    assert ((lse[:n].double() - l).abs()[~dead] <= tol_l[~dead] + 2.0 ** -20).all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("heads,kv_heads,d", [(12, 12, 64), (40, 8, 128), (16, 1, 128), (7, 1, 64)])
@pytest.mark.parametrize("groups,new", [
    ([(4, 1000)], [1]), ([(3, 127), (1, 128), (2, 129), (5, 640)], [1, 2]), ([(9, 513), (2, 0)], [0, 3, 1])])
def test_attend_shared(pkg, dt, page, heads, kv_heads, d, groups, new):
    c = Grouped(DT[dt], heads, kv_heads, d, page, groups, [0, 1, 40, 130, 300], new, seed=page + d)
    check_shared(c, run_shared(pkg, c), reference(c))


@pytest.mark.parametrize("heads,kv_heads,d,groups,tail,new", [
    (40, 8, 128, [(2, 300), (3, 1500)], [5, 600], [70, 1, 200]),      # many rows of a group, few and many of a sequence
    (16, 2, 64, [(40, 700)], [3, 90, 0], [1]),                         # more sequences than lanes
    (8, 8, 64, [(20, 200), (13, 400), (7, 129)], [31, 0], [2, 5]),
    (5, 1, 128, [(1, 2000), (1, 256)], [0], [1]),                      # groups of one
    (10, 2, 128, [(3, 9000)], [17], [4]),                              # a long prefix, cut into pieces
    (16, 2, 64, [(300, 260)], [9], [1])])                              # more sequences than threads
def test_attend_shared_sizes(pkg, heads, kv_heads, d, groups, tail, new):
    c = Grouped(torch.bfloat16, heads, kv_heads, d, 32, groups, tail, new, seed=len(groups))
    first = run_shared(pkg, c)
    check_shared(c, first, reference(c))
    again = run_shared(pkg, c, kv=first[2])
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    bits = tree_bits(c.new, 5)
    check_shared(c, run_shared(pkg, c, bits), reference(c, bits=bits))
    assert first[2].status() == 0


def test_attend_shared_more_groups_than_lanes(pkg):
    r = np.random.default_rng(4)
    groups = [(int(n), int(p)) for n, p in zip(r.integers(1, 4, 70), r.integers(0, 700, 70))]
    c = Grouped(torch.float16, 8, 2, 64, 16, groups, [0, 5, 33, 140], [1, 0, 2], seed=16)
    got = run_shared(pkg, c)
    check_shared(c, got, reference(c))
    assert got[2].status() == 0


def test_attend_shared_calls_one_after_another(pkg):
    """Calls of several shapes with one handle, each right behind the other: the second phase of one starts early."""
    cases = [Grouped(torch.bfloat16, 40, 8, 128, 64, g, [7, 300], n, seed=i)
             for i, (g, n) in enumerate([([(4, 1000)], [1]), ([(40, 512)], [1]), ([(3, 2000), (2, 640)], [30]), ([(2, 300)], [150])])]
    pools = [(c.k, c.v) for c in cases]
    kvs = [pkg.PagedKV(k, v, 40) for k, v in pools]
    outs = []
    for _ in range(3):
        outs.append([])
        for c, kv in zip(cases, kvs):
            prefix = kv.prefix(c.starts_of_groups(), ints(c.prefixes), c.rows)
            batch = c.batch(kv)
            for _ in range(2):
                out, lse = torch.full_like(c.q, 7), torch.full((c.rows, 40), 7.0, device=DEV)
                kv.attend(1, batch, c.q, out, lse=lse, prefix=prefix)
                kv.attend(1, batch, out, torch.empty_like(out))          # reads what the call before it wrote
                outs[-1].append((out, lse, prefix, batch))
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        want = reference(c)
        for o in outs:
            for x in o[2 * i:2 * i + 2]:
                check_shared(c, x, want)


def test_attend_shared_large_scores(pkg):
    c = Grouped(torch.bfloat16, 8, 2, 128, 64, [(3, 500)], [7, 200], [1, 40], seed=9)
    c.q *= 12
    check_shared(c, run_shared(pkg, c, scale=0.3), reference(c, scale=float(np.float32(0.3))))


def test_attend_shared_rows_that_see_the_prefix_alone_or_nothing(pkg):
    c = Grouped(torch.float16, 10, 2, 64, 16, [(2, 256), (2, 0)], [0], [3], seed=10)
    bits = tree_bits(c.new)
    bits[1] = bits[3] = bits[6] = 0                    # cached tokens alone (256 or 0 of them)
    check_shared(c, run_shared(pkg, c, bits), reference(c, bits=bits))


def test_attend_shared_sequences_outside_the_groups(pkg):
    c = Grouped(torch.float16, 8, 2, 64, 16, [(2, 300), (3, 200), (2, 300)], [9, 50], [1, 3], seed=11)
    kv = pkg.PagedKV(c.k, c.v, 8)
    prefix = kv.prefix(ints([2, 5]), ints([200]), c.rows)           # the others are taken as attend takes them
    check_shared(c, run_shared(pkg, c, kv=kv, prefix=prefix), reference(c))
    assert kv.status() == 0


def test_attend_shared_reads_the_first_sequences_pages(pkg):
    """The others' tables need not name the whole steps of 128 tokens: bad pages there are not read."""
    c = Grouped(torch.bfloat16, 8, 2, 128, 32, [(4, 300)], [9], [2], seed=12)
    want = reference(c)
    c.table[1:, :8] = -5                               # 256 of the prefix's 300 tokens
    got = run_shared(pkg, c)
    check_shared(c, got, want)
    assert got[2].status() == 0


def test_attend_shared_sequences_that_hold_the_whole_steps_alone(pkg):
    """A prefix of 200 tokens is shared in steps of 128: sequences of 128 to 199 cached tokens have what they need."""
    c = Grouped(torch.float16, 8, 2, 64, 32, [(3, 128)], [20, 0, 72], [2, 3], seed=15)
    kv = pkg.PagedKV(c.k, c.v, 8)
    check_shared(c, run_shared(pkg, c, kv=kv, prefix=kv.prefix(ints([0, 3]), ints([200]), c.rows)), reference(c))
    assert kv.status() == 0
    c = Grouped(torch.float16, 8, 2, 64, 32, [(3, 127)], [20, 0, 72], [2, 3], seed=15)
    out = run_shared(pkg, c, kv=(kv := pkg.PagedKV(c.k, c.v, 8)), prefix=kv.prefix(ints([0, 3]), ints([200]), c.rows))[0]
    at = slice(c.starts[1], c.starts[2])                # 127 cached tokens: left out
    assert kv.status(check=False) == 16 and (out[at] == 7).all() and not (out[:c.starts[1]] == 7).any()


@pytest.mark.parametrize("tail,new", [([9, 200], [2]), ([300], [60])])
def test_attend_shared_nans_reach_what_they_touch(pkg, tail, new):
    c = Grouped(torch.bfloat16, 8, 2, 128, 32, [(3, 300)], tail, new, seed=16)
    o, l, tol, tol_l = reference(c)
    c.k[1, int(c.table[0, 0]), 0, 5] = math.nan         # a shared token of one KV head
    c.k[1, int(c.table[1, 9]), 1, 15] = math.nan        # place 303, of the second sequence alone, of the other
    out, lse, kv = run_shared(pkg, c)
    bad = torch.zeros_like(lse, dtype=torch.bool)
    bad[:c.starts[3], :4] = True
    bad[c.starts[1]:c.starts[2], 4:] = True
    assert torch.equal(lse.isnan(), bad) and torch.equal(out.isnan(), bad[..., None].expand_as(out))
    n = c.starts[3]
    good = ~bad[:n]
    vmax = float(torch.nan_to_num(c.v.double(), 0, 0, 0).abs().max())
    assert ((out[:n].double() - o).abs()[good] <= tol[good] + 2.0 ** -20 * vmax).all()
    assert ((lse[:n].double() - l).abs()[good] <= tol_l[good] + 2.0 ** -20).all()


def test_attend_shared_bad_pages_and_lengths(pkg):
    c = Grouped(torch.float16, 8, 2, 64, 32, [(2, 400), (2, 300)], [9], [2], seed=13)
    kv = pkg.PagedKV(c.k, c.v, 8)
    out = run_shared(pkg, c, kv=kv, prefix=kv.prefix(ints([0, 2, 4]), ints([400, 700]), c.rows))
    assert kv.status(check=False) & 16                 # a prefix longer than its sequences (and than their pages)
    good = reference(c)
    assert (out[0][4:] == 7).all() and (out[1][4:] == 7).all()
    vmax = float(torch.nan_to_num(c.v.double(), 0, 0, 0).abs().max())
    assert ((out[0][:4].double() - good[0][:4]).abs() <= good[2][:4] + 2.0 ** -20 * vmax).all()
    for starts, lens in (([0, 3, 1], [128, 128]), ([-4, 2, 90], [128, 128]), ([0, 2, 4], [-3, 128])):
        run_shared(pkg, c, kv=kv, prefix=kv.prefix(ints(starts), ints(lens), c.rows))
        assert kv.status(check=False) & 16
    c.table[0, 1] = c.k.shape[1]
    out = run_shared(pkg, c, kv=kv)
    assert kv.status(check=False) == 8
    assert out[0][:4].isnan().all() and out[1][:4].isnan().all() and torch.isfinite(out[0][4:]).all()


def test_attend_shared_in_graphs_and_on_another_stream(pkg):
    c = Grouped(torch.bfloat16, 40, 8, 128, 64, [(6, 900), (3, 400)], [3, 80], [1], seed=14)
    want = reference(c)
    kv = pkg.PagedKV(c.k, c.v, 40)
    prefix = kv.prefix(c.starts_of_groups(), ints(c.prefixes), c.rows)
    batch = c.batch(kv)
    out, lse = [torch.full_like(c.q, 7) for _ in range(2)], [torch.full((c.rows, 40), 7.0, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for i in range(2):                                 # two graphs that share the handle's and the prefix's scratch
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            kv.attend(1, batch, c.q, out[i], lse=lse[i], prefix=prefix)
        graphs.append(g)
    for _ in range(3):
        for o, l in zip(out, lse):
            o.fill_(7)
            l.fill_(7)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, l in zip(out, lse):
            check_shared(c, (o, l), want)
    assert torch.equal(out[0], out[1])
    kv.attend(1, batch, c.q, out[0], lse=lse[0], prefix=prefix, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1])
    assert kv.status() == 0


# ---------------------------------------------------------------------------
# accumulated weights
# ---------------------------------------------------------------------------
def weigh_reference(c, lse, mass, decay, gain, bits=None, scale=None, layer=1):
    """mass_out and its tolerance, in 64 bits; mass where nothing is written."""
    want, tol = mass.double().clone(), torch.zeros_like(mass, dtype=torch.float64)
    g, scale = c.heads // c.H, c.d ** -0.5 if scale is None else scale
    cap = mass.shape[2]
    for b, (ctx, t) in enumerate(zip(c.ctx, c.new)):
        if not t:
            continue
        n, at = ctx + t, c.starts[b]
        vis = torch.ones(t, n, dtype=torch.bool)
        if bits is None:
            vis = vis.tril(ctx)
        else:
            vis[:, ctx:] = torch.tensor([[bool(bits[at + i] >> j & 1) for j in range(t)] for i in range(t)]).view(t, t)
        vis = vis.to(DEV)
        K = c.get(c.k, layer, b, n).double()
        for h in range(c.H):
            total, err = torch.zeros(n, dtype=torch.float64, device=DEV), torch.zeros(n, dtype=torch.float64, device=DEV)
            k = torch.nan_to_num(K[:, h], 0, 0, 0)
            for i in range(h * g, h * g + g):
                q, z = c.q[at:at + t, i].double(), lse[at:at + t, i].double()[:, None]
                s = q @ k.T * scale
                dead = z == -math.inf
                w = torch.where(vis & ~dead, (s - torch.where(dead, 0.0, z)).exp(), 0.0)
                ds = (c.d + 4) * 2.0 ** -23 * scale * (q.abs() @ k.abs().T)
                w_err = w * (2 * ds + 2.0 ** -21 * (1 + s.abs() + torch.where(dead, 0.0, z).abs()) + t * g * 2.0 ** -24) + 2.0 ** -126
                total += w.sum(0)
                err += torch.where(vis, w_err, 0.0).sum(0)
            old = torch.cat([decay * mass[b, h, :ctx].double(), torch.zeros(max(0, n - min(cap, ctx)), dtype=torch.float64, device=DEV)])
            m = min(n, cap)
            want[b, h, :m] = old[:m] + gain * total[:m]
            tol[b, h, :m] = abs(gain) * err[:m] + 2.0 ** -22 * (old[:m].abs() + abs(gain) * total[:m])
    return want, tol


def run_weigh(pkg, c, bits=None, decay=0.75, gain=0.5, cap=None, lse=None, kv=None, scale=0.0, in_place=False, positions=True):
    kv = kv or pkg.PagedKV(c.k, c.v, c.heads)
    mask = None
    if bits is not None:
        mask = mask_words(list(bits) + [0] * (c.rows - len(bits)), max(1, -(-max(c.new) // 32)))
    cap = cap or max(a + t for a, t in zip(c.ctx, c.new)) + 3
    lse = reference(c, bits=bits, scale=scale or None)[1].float() if lse is None else lse
    lse = torch.cat([lse, torch.zeros(c.rows - lse.shape[0], c.heads, device=DEV)])
    mass = torch.rand(len(c.ctx), c.H, cap, generator=c.g, device=DEV)
    pos = torch.full((len(c.ctx), c.H, cap), -9, dtype=torch.int32, device=DEV)
    given = torch.randint(0, 1 << 30, (c.rows,), generator=c.g, device=DEV, dtype=torch.int32) if positions else None
    before = mass.clone()
    out = mass if in_place else mass.clone()
    kv.weigh(1, c.batch(kv, mask), c.q, lse, mass, out, pos, positions=given, decay=decay, gain=gain, scale=scale)
    torch.cuda.synchronize()
    want, tol = weigh_reference(c, lse, before, decay, gain, bits, scale or None)
    assert ((out.double() - want).abs() <= tol).all(), float(((out.double() - want).abs() / tol.clamp(min=1e-30)).max())
    at = torch.full_like(pos, -9)
    for b, (ctx, t) in enumerate(zip(c.ctx, c.new)):
        new = given[c.starts[b]:c.starts[b] + t] if positions else torch.arange(ctx, ctx + t, device=DEV).int()
        at[b, :, ctx:min(cap, ctx + t)] = new[:max(0, cap - ctx)]
    assert torch.equal(pos, at)
    return out, kv


SHAPES = [(2, 2, 64), (12, 12, 64), (5, 1, 128), (40, 8, 128), (16, 1, 128), (64, 8, 64)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,kv_heads,d", SHAPES)
def test_weigh_single_tokens(pkg, dt, heads, kv_heads, d):
    c = Case(DT[dt], heads, kv_heads, d, 16, [0, 1, 15, 16, 127, 128, 300, 129], [1, 1, 1, 1, 1, 1, 1, 0], seed=heads)
    assert run_weigh(pkg, c)[1].status() == 0


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("page", [16, 32, 128, 256])
@pytest.mark.parametrize("heads,kv_heads,d", [(40, 8, 128), (16, 2, 64)])
def test_weigh_ragged(pkg, dt, page, heads, kv_heads, d):
    c = Case(DT[dt], heads, kv_heads, d, page, [0, 130, 7, 0, 511, 40], [70, 3, 0, 1, 33, 129], seed=page)
    assert run_weigh(pkg, c, in_place=page == 32, positions=page != 16)[1].status() == 0
    bits = tree_bits(c.new, heads)
    assert run_weigh(pkg, c, bits)[1].status() == 0


@pytest.mark.parametrize("heads,kv_heads,d,ctx,new", [
    (10, 2, 128, [3000, 0, 64], [1, 600, 300]), (12, 12, 64, [9000], [1]), (5, 1, 64, [100] * 40, [2] * 40),
    (16, 2, 64, [33] * 300, [1] * 300), (40, 8, 128, [4000], [64]), (8, 8, 64, [0], [1]), (16, 1, 64, [500], [200])])
def test_weigh_sizes(pkg, heads, kv_heads, d, ctx, new):
    c = Case(torch.bfloat16, heads, kv_heads, d, 32, ctx, new, seed=len(ctx))
    out, kv = run_weigh(pkg, c, decay=1.0, gain=1.0)
    assert kv.status() == 0


def test_weigh_gives_the_same_bits(pkg):
    c = Case(torch.float16, 40, 8, 128, 32, [3000, 200, 0], [1, 30, 100], seed=4)
    kv = pkg.PagedKV(c.k, c.v, 40)
    lse = torch.randn(c.rows, 40, device=DEV) + 8
    mass = torch.rand(3, 8, 3100, device=DEV)
    first = None
    for _ in range(30):
        out = torch.zeros_like(mass)
        kv.weigh(1, c.batch(kv), c.q, lse, mass, out)
        first = out if first is None else first
        assert torch.equal(out, first)


@pytest.mark.parametrize("heads,kv_heads,d,n,most,t", [(64, 8, 64, 32, 6000, 1), (40, 8, 128, 20, 4000, 1), (40, 8, 128, 9, 3000, 40), (16, 16, 64, 40, 700, 9)])
def test_weigh_many_items_launch_after_launch(pkg, heads, kv_heads, d, n, most, t):
    """Many items to a CTA, with even and odd numbers of token tiles: right, and the same bits on every run."""
    r = np.random.default_rng(n)
    c = Case(torch.bfloat16, heads, kv_heads, d, 64, [int(x) for x in r.integers(0, most, n)], [int(x) for x in r.integers(0, 2 * t, n)], seed=n)
    _, kv = run_weigh(pkg, c)
    batch, lse = c.batch(kv), torch.randn(c.rows, heads, device=DEV) + 9
    mass = torch.rand(n, kv_heads, most + 2 * t, generator=c.g, device=DEV)
    outs = [torch.zeros_like(mass) for _ in range(4)]
    kv.weigh(1, batch, c.q, lse, mass, outs[0])
    first = outs[0].clone()
    for _ in range(50):
        for o in outs:
            kv.weigh(1, batch, c.q, lse, mass, o)
    assert all(torch.equal(o, first) for o in outs)
    assert kv.status() == 0


def test_weigh_in_a_graph_and_on_two_streams(pkg):
    c = Case(torch.bfloat16, 40, 8, 128, 64, [3000, 128, 700], [1, 2, 60], seed=11)
    kv, other = pkg.PagedKV(c.k, c.v, 40), pkg.PagedKV(c.k, c.v, 40)
    batch, batch2 = c.batch(kv), c.batch(other)
    lse = torch.randn(c.rows, 40, device=DEV) + 9
    mass = torch.rand(3, 8, 3100, generator=c.g, device=DEV)
    outs = [torch.zeros_like(mass) for _ in range(4)]
    kv.weigh(1, batch, c.q, lse, mass, outs[0])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        kv.weigh(1, batch, c.q, lse, mass, outs[1])
    for _ in range(5):
        outs[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
    for _ in range(20):                                    # one handle on two streams too: nothing is shared
        kv.weigh(1, batch, c.q, lse, mass, outs[2])
        kv.weigh(1, batch, c.q, lse, mass, outs[3], stream=side)
        other.weigh(1, batch2, c.q, lse, mass, outs[1], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    assert kv.status() == 0 and other.status() == 0


def test_weigh_strided_queries(pkg):
    c = Case(torch.float16, 10, 2, 64, 16, [300, 20], [3, 40], seed=12)
    wide = torch.full((c.rows, 17, 64), math.nan, dtype=c.dt, device=DEV)
    wide[:, 2:12] = c.q
    c.q = wide[:, 2:12]
    run_weigh(pkg, c, in_place=True)


def test_weigh_masks_that_leave_nothing_and_masked_nans(pkg):
    c = Case(torch.float16, 10, 2, 64, 16, [0, 20], [5, 40], seed=5)
    bits = tree_bits(c.new)
    bits[0] = bits[4] = 0
    for b, i in ((0, 1), (1, 3)):
        at = c.ctx[b] + i
        c.k[:, int(c.table[b, at // 16]), :, at % 16] = math.nan
        for r in range(c.starts[b], c.starts[b + 1]):
            bits[r] &= ~(1 << i)
    run_weigh(pkg, c, bits)


def test_weigh_nans_reach_what_they_touch(pkg):
    c = Case(torch.bfloat16, 8, 2, 64, 16, [100, 50], [2, 1], seed=6, extra_rows=0)
    lse = reference(c)[1].float()
    kv = pkg.PagedKV(c.k, c.v, 8)
    c.k[1, int(c.table[0, 1]), 0, 3] = math.nan           # a token of one head
    lse[2, 7] = math.nan                                  # a row of another sequence
    mass = torch.zeros(2, 2, 110, device=DEV)
    kv.weigh(1, c.batch(kv), c.q, lse, mass, mass)
    torch.cuda.synchronize()
    bad = torch.zeros_like(mass, dtype=torch.bool)
    bad[0, 0, 19] = True
    bad[1, 1, :51] = True
    assert torch.equal(mass.isnan(), bad)


def test_weigh_beyond_cap_and_bad_pages(pkg):
    c = Case(torch.float16, 8, 2, 64, 16, [100, 40], [3, 3], seed=7)
    _, kv = run_weigh(pkg, c, cap=90)
    assert kv.status(check=False) == 2
    c.table[1, 1] = -1
    lse = torch.zeros(c.rows, 8, device=DEV) + 30
    mass, out = torch.zeros(2, 2, 110, device=DEV), torch.zeros(2, 2, 110, device=DEV)
    kv.weigh(1, c.batch(kv), c.q, lse, mass, out)
    assert kv.status(check=False) == 8
    assert out[1, :, 16:32].isnan().all() and torch.isfinite(out[0]).all() and torch.isfinite(out[1, :, :16]).all()


def test_weigh_a_single_sequence_without_rows_and_of_bad_lengths(pkg):
    c = Case(torch.bfloat16, 8, 2, 64, 16, [300], [0], seed=13)
    assert run_weigh(pkg, c)[1].status() == 0
    c = Case(torch.bfloat16, 8, 2, 64, 16, [100], [4], seed=14)
    kv, lse = pkg.PagedKV(c.k, c.v, 8), torch.zeros(c.rows, 8, device=DEV) + 30
    mass = torch.full((1, 2, 200), 3.0, device=DEV)
    for ctx, starts, flag in ((-5, [0, 4], 16), (100000, [0, 4], 2), (100, [-3, 1], 0), (100, [4, 0], 0)):
        out = mass.clone()
        kv.weigh(1, kv.batch(c.table, ints([ctx]), ints(starts)), c.q, lse, mass, out)
        assert kv.status(check=False) & flag == flag
        assert (out[:, :, 128:] == 3).all()             # (the table has 8 pages)
    assert torch.equal(out, mass)                       # starts that fall: no rows


def test_weigh_scale_and_long_lse(pkg):
    c = Case(torch.bfloat16, 8, 2, 128, 64, [500, 90], [1, 40], seed=8)
    c.q *= 4
    run_weigh(pkg, c, scale=0.25)


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def evict_reference(k, v, table, length, mass, pos, keep, protect, first, per_layer, page):
    """Unit by unit in Python, on the CPU."""
    k, v, mass_out, pos_out = k.clone(), v.clone(), {}, {}
    L, B, H, cap = mass.shape
    new = np.array(length).copy()
    for l in range(L):
        for b in range(B):
            n, want = (length[l][b], keep[l][b]) if per_layer else (length[b], keep[b])
            N = min(n, want)
            if per_layer:
                new[l][b] = N
            else:
                new[b] = N
            for h in range(H):
                m, p = mass[l, b, h, :n].tolist(), pos[l, b, h, :n].tolist()
                top = max(p, default=0)
                f = first[b] if first else 0

                def rank(j):
                    cls = 2 if j < f else 1 if p[j] > top - protect else 0
                    if cls:
                        return -cls, 0.0, False, j
                    nan = m[j] != m[j]                     # behind -inf
                    return 0, math.inf if nan else -m[j], nan, j

                order = sorted(range(n), key=rank)
                kept = sorted(order[:N])
                movers, stay = [j for j in kept if j >= N], set(kept)
                holes = [j for j in range(N) if j not in stay]
                assert len(movers) == len(holes)
                mo, po = m[:N], p[:N]
                for to, fr in zip(holes, movers):
                    mo[to], po[to] = m[fr], p[fr]
                    pt, pf = int(table[b, to // page]), int(table[b, fr // page])
                    for pool in (k, v):
                        pool[l, pt, h, to % page] = pool[l, pf, h, fr % page]
                mass_out[l, b, h], pos_out[l, b, h] = mo, po
    return k, v, mass_out, pos_out, new


def run_evict(pkg, L=2, B=2, H=2, heads=4, d=64, page=16, length=(40, 33), keep=(20, 33), cap=None, protect=4, first=None,
              per_layer=False, in_place=False, mass=None, pos=None, seed=0, dt=torch.float16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    flat = [x for r in length for x in r] if per_layer else list(length)
    cap = cap or max(max(flat), 1) + 3
    blocks = max(1, -(-max(flat) // page))
    pages = blocks * B + 2
    k = torch.randn(L, pages, H, page, d, generator=g, device=DEV).to(dt)
    v = torch.randn(L, pages, H, page, d, generator=g, device=DEV).to(dt)
    table = torch.randperm(pages, generator=g, device=DEV)[:B * blocks].view(B, blocks).int().contiguous()
    mass = torch.rand(L, B, H, cap, generator=g, device=DEV) if mass is None else mass.clone()
    pos = torch.rand(L, B, H, cap, generator=g, device=DEV).argsort(3).int() * 2 if pos is None else pos.clone()
    want = evict_reference(k.cpu(), v.cpu(), table.cpu(), length, mass.cpu(), pos.cpu(), keep, protect, first, per_layer, page)
    mass0, pos0 = mass.clone(), pos.clone()
    mo, po = (mass, pos) if in_place else (torch.full_like(mass, -5), torch.full_like(pos, -5))
    kv = pkg.PagedKV(k, v, heads)
    new = torch.full_like(ints(length), -7)
    kv.evict(table, ints(length), mass, pos, ints(keep), mo, po, new, protect=protect, first=ints(first) if first else None)
    torch.cuda.synchronize()
    assert torch.equal(new.cpu(), torch.tensor(want[4], dtype=torch.int32))
    for l in range(L):
        for b in range(B):
            N = int(want[4][l][b] if per_layer else want[4][b])
            for h in range(H):
                # (NaNs by their being NaN: their bits went through Python)
                assert np.array_equal(mo[l, b, h, :N].cpu().numpy(), np.array(want[2][l, b, h], np.float32), equal_nan=True), (l, b, h)
                assert po[l, b, h, :N].tolist() == want[3][l, b, h]
                assert torch.equal((mass0 if in_place else torch.full_like(mass, -5))[l, b, h, N:].view(torch.int32), mo[l, b, h, N:].view(torch.int32))
                assert torch.equal((pos0 if in_place else torch.full_like(pos, -5))[l, b, h, N:], po[l, b, h, N:])
    assert torch.equal(k.cpu().view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(v.cpu().view(torch.int16), want[1].view(torch.int16))
    if not in_place:
        assert torch.equal(mass.view(torch.int32), mass0.view(torch.int32)) and torch.equal(pos, pos0)
    assert kv.status() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("d,page,heads,H", [(64, 16, 4, 2), (128, 32, 10, 2), (128, 256, 3, 3), (64, 64, 16, 1)])
@pytest.mark.parametrize("length,keep,protect,first", [
    ((40, 33), (20, 33), 4, None), ((300, 257), (299, 256), 20, None), ((64, 65), (32, 64), 0, (3, 0)), ((1, 2), (1, 1), 1, None),
    ((500, 31), (31, 1), 8, (16, 16)), ((700, 0), (256, 9), 600, (40, 1000)), ((100, 99), (0, 200), 5, None), ((128, 96), (96, 32), 40, (64, 64)),
    ((1000, 999), (996, 990), 100, (1, 2))])
def test_evict(pkg, in_place, d, page, heads, H, length, keep, protect, first):
    run_evict(pkg, H=H, heads=heads, d=d, page=page, length=length, keep=keep, protect=protect, first=first, in_place=in_place,
              seed=d + len(length), dt=torch.bfloat16 if page == 32 else torch.float16)


@pytest.mark.parametrize("keep", [1, 7, 64, 150, 199])
def test_evict_ties_go_to_the_lower_place(pkg, keep):
    mass = (torch.randint(0, 3, (2, 1, 2, 200), generator=torch.Generator().manual_seed(keep)) * 0.5).to(DEV)
    run_evict(pkg, B=1, length=(200,), keep=(keep,), cap=200, mass=mass, protect=3)
    run_evict(pkg, B=1, length=(200,), keep=(keep,), cap=200, mass=torch.zeros_like(mass), protect=0, in_place=True)


def test_evict_odd_masses(pkg):
    """NaN below everything, infinities, both zeroes, negative and subnormal masses."""
    g = torch.Generator().manual_seed(1)
    odd = torch.tensor([math.nan, -math.nan, math.inf, -math.inf, 0.0, -0.0, -1.5, 1e-42, -1e-42, 3e38, 0.25])
    mass = odd[torch.randint(0, len(odd), (2, 2, 2, 150), generator=g)].to(DEV)
    for keep in ((10, 140), (75, 149), (130, 20)):
        run_evict(pkg, length=(150, 150), keep=keep, cap=150, mass=mass, protect=2, seed=keep[0])


def test_evict_positions_alike_negative_and_large(pkg):
    g = torch.Generator().manual_seed(2)
    for low, high in ((-50, 50), (0, 3), (2147483000, 2147483647), (-2147483648, -2147483000)):
        pos = torch.randint(low, high, (2, 2, 2, 90), generator=g, dtype=torch.int64).int().to(DEV)
        run_evict(pkg, length=(90, 70), keep=(40, 30), cap=90, pos=pos, protect=30)


def test_evict_a_budget_for_each_layer(pkg):
    run_evict(pkg, L=3, length=[[50, 40], [30, 40], [50, 1]], keep=[[20, 40], [30, 39], [1, 1]], per_layer=True, first=(2, 0))
    run_evict(pkg, L=3, length=[[50, 40], [30, 40], [50, 1]], keep=[[20, 40], [30, 39], [1, 1]], per_layer=True, in_place=True)


@pytest.mark.parametrize("length,keep,cap", [(9000, 1000, 9001), (5000, 4990, 60001), (4000, 3995, 4001), (45000, 44000, 45001)])
def test_evict_long(pkg, length, keep, cap):
    run_evict(pkg, L=1, B=1, H=1, heads=1, page=256, length=(length,), keep=(keep,), cap=cap, protect=50, first=(5,))


def test_evict_what_it_refuses_stays(pkg):
    g = torch.Generator(device=DEV).manual_seed(3)
    k = torch.randn(2, 9, 2, 16, 64, generator=g, device=DEV).half()
    v = k.clone()
    table = torch.arange(8, device=DEV).view(2, 4).int()
    mass = torch.rand(2, 2, 2, 64, generator=g, device=DEV)
    pos = torch.arange(64, device=DEV).int().expand(2, 2, 2, 64).contiguous()
    kv = pkg.PagedKV(k, v, 4)
    for length, keep, first, flag in (([-1, 40], [5, 40], None, 16), ([60, 40], [-2, 40], None, 16), ([60, 40], [10, 40], [-1, 0], 16),
                                      ([65, 40], [10, 40], None, 2)):
        k0, new = k.clone(), ints([-7, -7])
        mo, po = mass.clone(), pos.clone()
        kv.evict(table, ints(length), mo, po, ints(keep), mo, po, new, first=ints(first) if first else None)
        assert kv.status(check=False) == flag
        assert new.tolist() == length and torch.equal(k, k0) and torch.equal(mo, mass) and torch.equal(po, pos)
    table[0, 0] = 9                                    # a page outside the pool: its places take and give nothing
    new, mo, po = ints([0, 0]), torch.zeros_like(mass), torch.zeros_like(pos)
    mass[:, 0, :, :16], mass[:, 0, :, 16:] = 0.0, 1.0
    k0 = k.clone()
    kv.evict(table, ints([60, 40]), mass, pos, ints([32, 40]), mo, po, new)
    assert kv.status(check=False) == 8 and new.tolist() == [32, 40] and torch.equal(k, k0)
    assert torch.equal(mo[:, 0, :, :32], mass[:, 0, :, :32])


def test_evict_in_a_graph(pkg):
    """A decode loop at its budget: evict captured once, replayed for each token, mass and positions in place."""
    L, B, H, heads, d, page, N = 2, 2, 2, 4, 64, 16, 40
    g = torch.Generator(device=DEV).manual_seed(4)
    pages = B * 4
    k, v = (torch.randn(L, pages, H, page, d, generator=g, device=DEV).half() for _ in range(2))
    table = torch.arange(pages, device=DEV).view(B, 4).int()
    kv = pkg.PagedKV(k, v, heads)
    mass, pos = torch.rand(L, B, H, 64, generator=g, device=DEV), torch.arange(64, device=DEV).int().expand(L, B, H, 64).contiguous()
    length, new, keep = ints([41, 30]), ints([0, 0]), ints([N, N])
    eager = [x.clone() for x in (k, v, mass, pos, new)]
    kv2 = pkg.PagedKV(eager[0], eager[1], heads)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        kv.evict(table, length, mass, pos, keep, mass, pos, new, protect=5)
    for i in range(4):
        length.copy_(ints([41, 30 + i]))
        mass[..., 40] = eager[2][..., 40] = float(i)
        graph.replay()
        kv2.evict(table, length, eager[2], eager[3], keep, eager[2], eager[3], eager[4], protect=5)
        torch.cuda.synchronize()
        for a, b in zip((k, v, mass, pos, new), eager):
            assert torch.equal(a, b)


def test_arguments_that_are_refused(pkg):
    c = Case(torch.float16, 8, 2, 64, 16, [20, 9], [2, 1], seed=15, extra_rows=0)
    kv, n = pkg.PagedKV(c.k, c.v, 8), c.rows
    batch = c.batch(kv)
    q, k, v = c.randn(n, 8, 64), c.randn(n, 2, 64), c.randn(n, 2, 64)
    out, lse = torch.empty_like(q), torch.zeros(n, 8, device=DEV)
    w, inv = torch.ones(64, device=DEV), torch.ones(32, device=DEV)
    pos2, axis = torch.zeros(n, 2, device=DEV, dtype=torch.int32), torch.zeros(32, device=DEV, dtype=torch.int32)
    mass, place = torch.zeros(2, 2, 30, device=DEV), torch.zeros(2, 2, 30, device=DEV, dtype=torch.int32)
    many, where = torch.zeros(2, 2, 2, 30, device=DEV), torch.zeros(2, 2, 2, 30, device=DEV, dtype=torch.int32)
    prefix = kv.prefix(ints([0, 2]), ints([9]), n)
    small = kv.prefix(ints([0, 2]), ints([9]), 1)
    err = (ValueError, pkg.ConfKVError)
    bad = [
        lambda: kv.append(0, batch, k, v, q_norm=w),                                        # no q
        lambda: kv.append(0, batch, k, v, k_norm=w.double()),
        lambda: kv.append(0, batch, k, v, k_norm=w.bfloat16()),
        lambda: kv.append(0, batch, k, v, q=q, q_out=out, q_norm=w, k_norm=w.half()),       # two types
        lambda: kv.append(0, batch, k, v, k_norm=w[:32]),
        lambda: kv.append(0, batch, k, v, k_norm=w, eps=0.0),
        lambda: kv.append(0, batch, k, v, k_norm=w, eps=float("nan")),
        lambda: kv.append(0, batch, k, v, inv_freq=inv, axis=axis),                         # no positions
        lambda: kv.append(0, batch, k, v, positions=pos2, axis=axis),                       # nothing turns
        lambda: kv.append(0, batch, k, v, inv_freq=inv, positions=pos2[:, 0].contiguous(), axis=axis),
        lambda: kv.append(0, batch, k, v, inv_freq=inv, positions=pos2, k_norm=w),          # axes without axis
        lambda: kv.append(0, batch, k, v, inv_freq=inv, positions=pos2, axis=axis[:31]),
        lambda: kv.append(0, batch, k, v, inv_freq=inv, positions=torch.zeros(n, 9, device=DEV, dtype=torch.int32), axis=axis),
        lambda: kv.append(2, batch, k, v, k_norm=w),
        lambda: kv.append(0, batch, k, v, q=q, q_out=out, k_norm=out.view(-1)[:64]),        # an output in an input
        lambda: kv.prefix(ints([0, 2]), ints([9]), -1),
        lambda: kv.prefix(ints([0, 2]), ints([9, 9]), 1),
        lambda: kv.prefix(ints([0]), ints([]), 1),
        lambda: kv.attend(0, batch, q, out, prefix=small),                                  # scratch for one row
        lambda: kv.attend(0, batch, q, q, prefix=prefix),
        lambda: kv.attend(0, batch, q, out, prefix=kv.prefix(ints([0, 1, 2, 2]), ints([1, 1, 1]), n)),   # more groups than sequences
        lambda: kv.attend(0, batch, q, out, prefix=prefix, scale=-1.0),
        lambda: kv.weigh(0, batch, q, lse, mass, mass[:1]),
        lambda: kv.weigh(0, batch, q, lse, mass, torch.zeros(2, 2, 31, device=DEV)),
        lambda: kv.weigh(0, batch, q, lse[:2], mass, mass),
        lambda: kv.weigh(0, batch, q, lse, mass, mass, place.long()),
        lambda: kv.weigh(0, batch, q, lse, mass, mass, decay=math.inf),
        lambda: kv.weigh(0, batch, q, lse, mass, mass, gain=math.nan),
        lambda: kv.weigh(0, batch, q, lse, mass, mass, scale=-1.0),
        lambda: kv.weigh(5, batch, q, lse, mass, mass),
        lambda: kv.weigh(0, batch, q, lse, mass, mass.transpose(0, 1)),
        lambda: kv.evict(c.table, ints([9, 9]), many, where, ints([5, 5]), many, where.clone(), ints([0, 0])),   # one in place
        lambda: kv.evict(c.table, ints([9, 9]), many, where, ints([5]), many, where, ints([0, 0])),
        lambda: kv.evict(c.table, ints([9, 9]), many, where, ints([5, 5]), many, where, ints([0, 0]), protect=-1),
        lambda: kv.evict(c.table, ints([9, 9]), many[:1], where[:1], ints([5, 5]), many[:1], where[:1], ints([0, 0])),
        lambda: kv.evict(c.table, ints([[9, 9]]), many, where, ints([[5, 5]]), many, where, ints([[0, 0]])),
        lambda: kv.evict(c.table, ints([9, 9]), many, where, ints([5, 5]), many, where, ints([0, 0]), first=ints([0])),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(err):
            call()
            raise AssertionError(i)
    length = ints([9, 9])
    with pytest.raises(err):
        kv.evict(c.table, length, many, where, ints([5, 5]), many, where, length)           # lengths of their own
    both = torch.zeros(2 * 240, device=DEV)
    with pytest.raises(err):
        kv.evict(c.table, length, both[:240].view(2, 2, 2, 30), where, ints([5, 5]), both[100:340].view(2, 2, 2, 30), where.clone(), ints([0, 0]))
    assert kv.status() == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_a_decode_loop_over_a_shared_prefix_within_a_budget(pkg):
    """Two requests behind one instruction: normed and rotated rows are appended, attended over the shared prefix, weighed and
    evicted down to a budget, layer by layer; every step against dense attention over the tokens that each head still has."""
    L, H, heads, d, page, P, N, steps, dt = 2, 2, 8, 64, 16, 160, 200, 12, torch.bfloat16
    g, B, cap = torch.Generator(device=DEV).manual_seed(5), 2, 320
    r = heads // H
    own = -(-(cap - P) // page)
    pages = P // page + B * own
    k_pool, v_pool = (torch.full((L, pages, H, page, d), math.nan, dtype=dt, device=DEV) for _ in range(2))
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.stack([torch.cat([order[:P // page], order[P // page + b * own:P // page + (b + 1) * own]]) for b in range(B)])
    kv = pkg.PagedKV(k_pool, v_pool, heads)
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    axis = (torch.arange(d // 2, device=DEV) % 3).int()
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt) for _ in range(2))
    mass, pos = torch.zeros(L, B, H, cap, device=DEV), torch.full((L, B, H, cap), -1, dtype=torch.int32, device=DEV)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dt)  # noqa: E731
    # the instruction: one sequence appends it, the other's table names the same pages
    first = kv.batch(table[:1], ints([0]), ints([0, P]))
    where = torch.randint(0, 500, (P, 3), generator=g, device=DEV, dtype=torch.int32)
    for l in range(L):
        kv.append(l, first, randn(P, H, d), randn(P, H, d), positions=where, inv_freq=inv, k_norm=wk, axis=axis)
        pos[l, :, :, :P] = torch.arange(P, device=DEV).int()
    ctx, text, prefix = ints([P, P]), [P, P], kv.prefix(ints([0, B]), ints([P]), 64)
    keep, fixed = ints([N, N - 30]), ints([P, P])
    at = torch.arange(P, device=DEV)
    alive = [[[list(range(P)) for _ in range(H)] for _ in range(B)] for _ in range(L)]      # positions of each head's places
    store = [[{} for _ in range(B)] for _ in range(L)]                                      # position -> K, V rows of all heads
    for l in range(L):
        kk, vv = k_pool[l, table[0].long()[at // page], :, at % page], v_pool[l, table[0].long()[at // page], :, at % page]
        for b in range(B):
            for j in range(P):
                store[l][b][j] = (kk[j].double(), vv[j].double())
    weight = torch.zeros(L, B, H, 1000, dtype=torch.float64, device=DEV)       # by position
    for step in range(steps):
        counts = [30, 17] if step == 0 else [1, 1] if step % 3 else [1, 4]
        starts = [0, counts[0], sum(counts)]
        rows = starts[-1]
        batch = kv.batch(table, ctx, ints(starts))
        text_pos = ints([text[b] + i for b in range(B) for i in range(counts[b])])
        new_len = torch.zeros_like(ctx)
        for l in range(L):
            q, k, v = randn(rows, heads, d), randn(rows, H, d), randn(rows, H, d)
            q_rot, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(rows, heads, device=DEV)
            axes = torch.randint(0, 500, (rows, 3), generator=g, device=DEV, dtype=torch.int32)
            kv.append(l, batch, k, v, q=q, q_out=q_rot, positions=axes, inv_freq=inv, q_norm=wq, k_norm=wk, axis=axis)
            kv.attend(l, batch, q_rot, out, lse=lse, prefix=prefix)
            kv.weigh(l, batch, q_rot, lse, mass[l], mass[l], pos[l], positions=text_pos, decay=0.9, gain=0.1 / r)
            angle = axes.double()[:, axis.long()] * inv.double()
            want_k = turned(normed(k, wk, 1e-6), angle, d, False)[0]
            want_q = turned(normed(q, wq, 1e-6), angle, d, False)[0]
            assert ((q_rot.double() - want_q).abs() <= 2.0 ** -8 * want_q.abs() + 2.0 ** -17 * want_q.abs().max()).all()
            for b in range(B):
                weight[l, b] *= 0.9
                for i in range(counts[b]):
                    row, p = starts[b] + i, text[b] + i
                    place = int(ctx[b]) + i
                    pg, sl = int(table[b, place // page]), place % page
                    assert ((k_pool[l, pg, :, sl].double() - want_k[row]).abs() <= 2.0 ** -8 * want_k[row].abs() + 2.0 ** -17 * want_k.abs().max()).all()
                    store[l][b][p] = (k_pool[l, pg, :, sl].double(), v_pool[l, pg, :, sl].double())
                    for h in range(H):
                        alive[l][b][h].append(p)
                for i in range(counts[b]):
                    row, p = starts[b] + i, text[b] + i
                    for h in range(H):
                        seen = [x for x in alive[l][b][h] if x <= p]
                        K = torch.stack([store[l][b][x][0][h] for x in seen])
                        V = torch.stack([store[l][b][x][1][h] for x in seen])
                        s = q_rot[row, h * r:(h + 1) * r].double() @ K.T * d ** -0.5
                        w = torch.softmax(s, 1)
                        o = out[row, h * r:(h + 1) * r].double()
                        # P rounded once (2^-8 of its part of sum |p v|) and the output once; the scores are off by
                        # (d + 4) 2^-23 scale |q||k| <= 1e-4 (both normed, weights to 1.8), weights by twice that
                        assert ((o - w @ V).abs() <= 2.0 ** -8 * (w @ V).abs() + (2.0 ** -8 + 2.0 ** -11) * (w @ V.abs())).all()
                        weight[l, b, h, torch.tensor(seen, device=DEV)] += 0.1 / r * w.sum(0)
                for h in range(H):
                    n = len(alive[l][b][h])
                    assert pos[l, b, h, :n].tolist() == alive[l][b][h]
                    have = mass[l, b, h, :n].double()
                    assert ((have - weight[l, b, h, pos[l, b, h, :n].long()]).abs() <= 4e-4 * have + 1e-9).all()
        length = ctx + ints(counts)
        before, masses = [[[list(x) for x in y] for y in z] for z in alive], mass.clone()
        kv.evict(table, length, mass, pos, keep, mass, pos, new_len, protect=8, first=fixed)
        for l in range(L):
            for b in range(B):
                for h in range(H):
                    old, m = before[l][b][h], masses[l, b, h].tolist()
                    new = [j for j in range(P, len(old)) if old[j] > max(old) - 8]
                    rest = sorted((j for j in range(P, len(old)) if old[j] <= max(old) - 8), key=lambda j: (-m[j], j))
                    stay = (list(range(P)) + new + rest)[:int(keep[b])]
                    alive[l][b][h] = pos[l, b, h, :int(new_len[b])].tolist()
                    assert sorted(alive[l][b][h]) == sorted(old[j] for j in stay)
                    assert alive[l][b][h][:P] == list(range(P))
        text = [text[b] + counts[b] for b in range(B)]
        ctx = new_len.clone()
        assert ctx.tolist() == [min(int(length[b]), int(keep[b])) for b in range(B)]
    assert kv.status() == 0
