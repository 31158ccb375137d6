"""Normed appends, attention over shared prefixes, accumulated weights and eviction where calls meet the ends
of their ranges and one another.  Tolerances: those of test_paged_budget_gpu.py."""
import math

import numpy as np
import pytest
import torch

from tests.test_paged_budget_gpu import Grouped, check_append, check_shared, run_shared, run_weigh, weigh_reference
from tests.test_paged_gpu import DT, Case, ints, mask_words, reference, tree_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkg():
    import confidence_gated_kv_logits_gb300 as pkg
    pkg.load_library()
    return pkg


# ---------------------------------------------------------------------------
# append with norms
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("r", [0, 64])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("low,high", [(-24, -17), (-10, 0), (0, 10), (60, 100)])
def test_append_normed_huge_rows_under_any_weights(pkg, low, high, wide, r):
    """Rows from 2^118 to the type's largest value: 1 / rms is small or subnormal, and weights from 1e-7 to 2^100 times it
    would leave fp32's range, in which the normed values and the results lie."""
    c = Case(torch.bfloat16, 4, 4, 64, 16, [0], [10], seed=high + r, extra_rows=0)
    x = c.randn(10, 4, 64).float().clamp(-0.99, 0.99) * 2.0 ** torch.arange(119, 129, device=DEV).float()[:, None, None]
    x = x.to(torch.bfloat16)
    x[9] = torch.finfo(torch.bfloat16).max
    assert torch.isfinite(x).all()
    w = [(2.0 ** (low + (high - low) * torch.rand(64, generator=c.g, device=DEV))).to(torch.float32 if wide else torch.bfloat16) for _ in range(2)]
    check_append(pkg, c, r, False, 0, w[0], w[1], q=x, k=x.flip(0).contiguous())


@pytest.mark.parametrize("wide", [False, True])
def test_append_normed_tiny_rows_under_huge_weights(pkg, wide):
    """Rows so small that eps alone counts: 1 / sqrt(eps) = 1e6 times a weight of 1e33 leaves fp32, the results (1e20 and less) do not."""
    c = Case(torch.bfloat16, 4, 4, 64, 16, [0], [6], seed=3, extra_rows=0)
    x = (c.randn(6, 4, 64).float() * 10.0 ** -torch.arange(20, 26, device=DEV).float()[:, None, None]).to(torch.bfloat16)
    w = [(1e33 * (1 + torch.rand(64, generator=c.g, device=DEV))).to(torch.float32 if wide else torch.bfloat16) for _ in range(2)]
    check_append(pkg, c, 64, True, 0, w[0], w[1], eps=1e-12, q=x, k=x.flip(0).contiguous())


# ---------------------------------------------------------------------------
# attention over shared prefixes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,H,d,B,T,tail", [
    (40, 8, 128, 4, 1, 60),            # phase 2 by clusters or whole units of eight warps
    (12, 12, 64, 40, 1, 200),          # by CTAs of four warps
    (64, 8, 64, 8, 5, 300),            # 40 rows of a KV head, streamed
    (40, 8, 128, 3, 60, 500)])         # by the prompt kernel
def test_attend_shared_right_behind_what_wrote_its_inputs(pkg, dt, heads, H, d, B, T, tail):
    """Lengths, tables, masks, queries and rows change in place right before the call, eagerly and in a replayed graph: phase 2,
    which starts before phase 1 has ended, sees what the calls before wrote.  The same calls with waits between them say
    what it has to be, bit for bit."""
    P, page, V = 640, 32, 6
    g = torch.Generator(device=DEV).manual_seed(B + T)
    full, own, n = P // page, -(-(tail + T) // page), B * T
    pages = full + V * B * own                       # each variant has tails of its own
    k_pool, v_pool = (torch.randn(2, pages, H, page, d, generator=g, device=DEV).to(DT[dt]) for _ in range(2))
    order = torch.randperm(pages, generator=g, device=DEV).int()
    kv = pkg.PagedKV(k_pool, v_pool, heads)
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    words = -(-T // 32)

    def variant(i):
        tails = order[full + i * B * own:full + (i + 1) * B * own].view(B, own)
        return [torch.cat([order[:full].expand(B, full), tails], 1).contiguous(),
                (P + torch.randint(0, tail + 1, (B,), generator=g, device=DEV)).int(),
                torch.randint(-(1 << 31), 1 << 31, (n, words), generator=g, device=DEV).int()] + [
                    torch.randn(n, x, d, generator=g, device=DEV).to(DT[dt]) for x in (heads, H, H)]

    variants = [variant(i) for i in range(V)]
    staged, live = [x.clone() for x in variants[0]], [x.clone() for x in variants[0]]
    table, ctx, mask, q, k, v = live
    batch = kv.batch(table, ctx, ints([T * b for b in range(B + 1)]), mask)
    prefix = kv.prefix(ints([0, B]), ints([P]), n)
    q_rot, out, out2, lse = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q), torch.empty(n, heads, device=DEV)
    none = lambda: None  # noqa: E731

    def step(between=none):
        for x, y in zip(live, staged):
            x.copy_(y)
        between()
        kv.append(1, batch, k, v, q=q, q_out=q_rot, inv_freq=inv)
        between()
        kv.attend(1, batch, q_rot, out, lse=lse, prefix=prefix)
        between()
        kv.attend(1, batch, out, out2, prefix=prefix)          # reads what the call before it wrote
        between()

    def stage(i):
        for x, y in zip(staged, variants[i]):
            x.copy_(y)

    want = []
    for i in range(V):
        stage(i)
        step(torch.cuda.synchronize)
        want.append([x.clone() for x in (q_rot, out, lse, out2)])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    got, picks = [], np.random.default_rng(T).integers(0, V, 80).tolist()
    for j, i in enumerate(picks):
        stage(i)
        graph.replay() if j % 2 else step()
        got.append([x.clone() for x in (q_rot, out, lse, out2)])
    torch.cuda.synchronize()
    for i, have in zip(picks, got):
        for x, y in zip(have, want[i]):
            assert torch.equal(x, y)
    assert kv.status() == 0
    assert all(torch.isfinite(x).all() for w in want for x in (w[0], w[1]))


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,H,d,page,groups,tail,new", [
    # by the rows of a KV head, on average (152 SMs): from 257 on tiles of 256 rows, if there are 76 or more
    (64, 8, 64, 64, [(8, 700), (9, 520), (7, 260)], [0, 33, 300], [12]),                # phase 1; phase 2 in tiles of 128
    (40, 8, 128, 32, [(5, 400), (7, 130), (6, 900), (5, 128), (8, 0), (3, 640)], [5, 140], [12, 11, 13]),
    (40, 8, 128, 64, [(4, 300), (4, 500)], [10, 200], [60, 61, 55]),                    # both phases
    (16, 16, 64, 16, [(3, 256), (2, 390)], [7], [300, 120, 200]),
    # from 32 sequences on phase 2 by CTAs of four warps
    (12, 12, 64, 16, [(40, 300)], [0, 5, 200], [1]),
    (40, 8, 128, 64, [(30, 512), (3, 200), (20, 128)], [1, 90, 400], [1, 2, 0, 8]),
    (16, 1, 128, 256, [(33, 1000)], [3, 600], [1, 2])])
def test_attend_shared_every_form(pkg, dt, heads, H, d, page, groups, tail, new):
    c = Grouped(DT[dt], heads, H, d, page, groups, tail, new, seed=heads + len(groups))
    first = run_shared(pkg, c)
    check_shared(c, first, reference(c))
    bits = tree_bits(c.new, 2)
    check_shared(c, run_shared(pkg, c, bits, kv=first[2]), reference(c, bits=bits))
    assert first[2].status() == 0


def test_attend_shared_repeats_itself_between_other_calls(pkg):
    """The same bits on every run, whatever ran before on the same handle and scratch."""
    cases = [Grouped(DT[dt], 40, 8, 128, 64, g, [7, 300], n, seed=i)
             for i, (dt, g, n) in enumerate([("bf16", [(4, 1000)], [1]), ("fp16", [(64, 2000)], [1]), ("bf16", [(8, 2000), (3, 640)], [12]),
                                             ("bf16", [(3, 1200), (2, 200)], [90])])]
    calls = []
    for c in cases:
        kv = pkg.PagedKV(c.k, c.v, 40)
        prefix, batch = kv.prefix(c.starts_of_groups(), ints(c.prefixes), c.rows), c.batch(kv)
        calls.append(lambda out, lse, c=c, kv=kv, prefix=prefix, batch=batch: kv.attend(1, batch, c.q, out, lse=lse, prefix=prefix))
    want = []
    for c, call in zip(cases, calls):
        want.append((torch.zeros_like(c.q), torch.zeros(c.rows, 40, device=DEV)))
        call(*want[-1])
        torch.cuda.synchronize()
    for i in np.random.default_rng(0).integers(0, len(cases), 300).tolist():
        out, lse = torch.zeros_like(cases[i].q), torch.zeros(cases[i].rows, 40, device=DEV)
        calls[i](out, lse)
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


# ---------------------------------------------------------------------------
# accumulated weights
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,H,d,page,T", [(40, 8, 128, 32, 12), (12, 12, 64, 16, 40)])
def test_weigh_the_accepted_rows_behind_commit(pkg, dt, heads, H, d, page, T):
    """Trees of drafts are attended by their mask, a path of each is kept, and its rows, gathered, are weighed without the
    mask: the places that they came to hold hold their masses and positions."""
    c = Case(DT[dt], heads, H, d, page, [200, 0, 33, 129], [T, T, 0, T - 3], seed=T)
    bits = tree_bits(c.new, 3)
    mask = mask_words(bits + [0] * (c.rows - len(bits)), -(-T // 32))
    kv = pkg.PagedKV(c.k, c.v, heads)
    out, lse = torch.empty_like(c.q), torch.empty(c.rows, heads, device=DEV)
    kv.attend(1, c.batch(kv, mask), c.q, out, lse=lse)
    paths = [[j for j in range(T) if t and bits[c.starts[b] + t - 1] >> j & 1] for b, t in enumerate(c.new)]     # to the last draft
    assert any(1 < len(p) < t for p, t in zip(paths, c.new))
    new_len = ints([0] * 4)
    kv.commit(c.table, ints(c.ctx), ints([p + [0] * (T - len(p)) for p in paths]), ints([len(p) for p in paths]), new_len)
    rows = torch.tensor([c.starts[b] + j for b, p in enumerate(paths) for j in p], device=DEV)
    c.new = [len(p) for p in paths]
    c.starts = [sum(c.new[:b]) for b in range(5)]
    c.rows, c.q = c.starts[-1], c.q[rows]
    _, kv = run_weigh(pkg, c, lse=lse[rows], kv=kv)
    assert new_len.tolist() == [a + t for a, t in zip(c.ctx, c.new)] and kv.status() == 0
    # and it is what attention of the committed rows gives
    again, lse2 = torch.empty_like(c.q), torch.empty(c.rows, heads, device=DEV)
    kv.attend(1, c.batch(kv), c.q, again, lse=lse2)
    _, l, _, tol = reference(c)
    for x in (lse2, lse[rows]):
        assert ((x.double() - l).abs() <= tol).all()


def test_weigh_reads_every_sequences_own_pages(pkg):
    """Behind a prefix whose pages the others' tables do not name, attend has what it needs and weigh does not: flagged, NaN."""
    c = Grouped(torch.bfloat16, 8, 2, 128, 32, [(3, 300)], [9], [2], seed=12)
    o, l, tol, _ = reference(c)
    kept = c.table.clone()
    c.table[1:, :8] = -5                               # 256 of the prefix's 300 tokens
    out, lse, kv = run_shared(pkg, c)
    assert kv.status() == 0
    mass = torch.rand(3, 2, 330, generator=c.g, device=DEV)
    before = mass.clone()
    kv.weigh(1, c.batch(kv), c.q, lse, mass, mass, decay=0.75, gain=0.5)
    assert kv.status(check=False) == 8
    assert mass[1:, :, :256].isnan().all()
    c.table = kept
    want, tol = weigh_reference(c, lse[:c.starts[-1]], before, 0.75, 0.5)
    assert ((mass.double() - want).abs()[:1] <= tol[:1]).all()
    assert ((mass.double() - want).abs()[1:, :, 256:] <= tol[1:, :, 256:]).all()


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,H,d,n,most,t", [
    (40, 8, 128, 20, 4000, 22), (64, 8, 64, 24, 3000, 14), (16, 2, 128, 40, 3500, 14), (32, 32, 64, 12, 2500, 112), (5, 1, 128, 60, 9000, 3)])
def test_weigh_many_tiles_an_item_by_trees(pkg, dt, heads, H, d, n, most, t):
    """Items of eight token tiles (six tiles a CTA or more) and all rows in one tile of rows, causal and by the batch's mask."""
    r = np.random.default_rng(n)
    c = Case(DT[dt], heads, H, d, 64, [int(x) for x in r.integers(0, most, n)], [int(x) for x in r.integers(0, t + 1, n)], seed=n)
    assert n * H * c.table.shape[1] * 64 >= 6 * 152 * 128
    assert run_weigh(pkg, c, in_place=True)[1].status() == 0
    assert run_weigh(pkg, c, tree_bits(c.new, 4))[1].status() == 0


def test_weigh_writes_nothing_else(pkg):
    """A mass_out of its own keeps what it held for sequences without rows and behind the new tokens."""
    c = Case(torch.bfloat16, 10, 2, 64, 16, [300, 40, 0, 7], [2, 0, 5, 0], seed=2)
    kv = pkg.PagedKV(c.k, c.v, 10)
    lse = torch.randn(c.rows, 10, device=DEV) + 8
    mass = torch.rand(4, 2, 320, generator=c.g, device=DEV)
    out, pos = torch.full_like(mass, -5), torch.full((4, 2, 320), -9, dtype=torch.int32, device=DEV)
    kv.weigh(1, c.batch(kv), c.q, lse, mass, out, pos)
    assert kv.status() == 0
    for b, (a, t) in enumerate(zip(c.ctx, c.new)):
        n = a + t if t else 0
        assert (out[b, :, :n] >= 0).all() and (out[b, :, n:] == -5).all()
        assert (pos[b, :, :a] == -9).all() and (pos[b, :, a + t:] == -9).all()
        assert torch.equal(pos[b, :, a:a + t], torch.arange(a, a + t, device=DEV).int().expand(2, t))


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("cap", [64, 5000, 41000])
@pytest.mark.parametrize("length,keep,first,flag", [
    ([-1, 40], [5, 30], None, 16), ([60, 40], [-2, 30], None, 16), ([60, 40], [10, 30], [-1, 0], 16), ([65, 40], [10, 30], None, 2),
    ([1 << 30, 40], [10, 30], None, 2)])
def test_evict_out_of_place_what_it_refuses_stays(pkg, length, keep, first, flag, cap):
    """A refused sequence's masses and positions are in the outputs, as its length is; behind them nothing is written."""
    g = torch.Generator(device=DEV).manual_seed(cap)
    k = torch.randn(2, 9, 2, 16, 64, generator=g, device=DEV).half()
    v, k0 = k.clone(), k.clone()
    table = torch.arange(8, device=DEV).view(2, 4).int()
    mass = torch.rand(2, 2, 2, cap, generator=g, device=DEV)
    pos = torch.arange(cap, device=DEV).int().expand(2, 2, 2, cap).contiguous()
    mo, po, new = torch.full_like(mass, -5), torch.full_like(pos, -5), ints([-7, -7])
    kv = pkg.PagedKV(k, v, 4)
    kv.evict(table, ints(length), mass, pos, ints(keep), mo, po, new, first=ints(first) if first else None)
    assert kv.status(check=False) == flag
    n = min(max(length[0], 0), cap)
    assert new.tolist() == [length[0], 30]
    assert torch.equal(mo[:, 0, :, :n], mass[:, 0, :, :n]) and torch.equal(po[:, 0, :, :n], pos[:, 0, :, :n])
    assert (mo[:, 0, :, n:] == -5).all() and (po[:, 0, :, n:] == -5).all()
    pages = table[0].long()
    assert torch.equal(k[:, pages], k0[:, pages]) and torch.equal(v[:, pages], k0[:, pages])
    # the other sequence is evicted: the 30 largest of its masses (positions rise, none is protected)
    assert torch.equal(mo[:, 1, :, :30].sort(2).values, mass[:, 1, :, :40].sort(2).values[..., 10:])


@pytest.mark.parametrize("keep", [[150, 200, 130], [297, 295, 150]])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_behind_a_shared_prefix(pkg, keep, in_place):
    """Three sequences name the same pages for 128 tokens, which weigh least: with `first` they stay, and each sequence's own
    tokens are evicted as they are without the others."""
    P, page, L, H, d, B, n = 128, 32, 2, 2, 64, 3, 300
    g = torch.Generator(device=DEV).manual_seed(keep[0])
    own = -(-(n - P) // page)
    k, v = (torch.randn(L, P // page + B * own, H, page, d, generator=g, device=DEV).half() for _ in range(2))
    order = torch.randperm(k.shape[1], generator=g, device=DEV).int()
    table = torch.stack([torch.cat([order[:P // page], order[P // page + b * own:P // page + (b + 1) * own]]) for b in range(B)])
    mass = torch.rand(L, B, H, n, generator=g, device=DEV) + 1
    mass[..., :P] *= 1e-3
    pos = torch.rand(L, B, H, n, generator=g, device=DEV).argsort(3).int()
    alone = []
    for b in range(B):                                     # each with pools of its own
        k1, v1, m1, p1 = k.clone(), v.clone(), mass[:, b:b + 1].clone(), pos[:, b:b + 1].clone()
        pkg.PagedKV(k1, v1, 4).evict(table[b:b + 1].contiguous(), ints([n]), m1, p1, ints(keep[b:b + 1]), m1, p1, ints([0]), protect=9, first=ints([P]))
        alone.append((k1, v1, m1, p1))
    shared, k0, v0 = order[:P // page].long(), k.clone(), v.clone()
    kv = pkg.PagedKV(k, v, 4)
    mo, po, new = (mass, pos, ints([0] * B)) if in_place else (torch.zeros_like(mass), torch.zeros_like(pos), ints([0] * B))
    kv.evict(table, ints([n] * B), mass, pos, ints(keep), mo, po, new, protect=9, first=ints([P] * B))
    torch.cuda.synchronize()
    assert new.tolist() == keep and kv.status() == 0
    assert torch.equal(k[:, shared], k0[:, shared]) and torch.equal(v[:, shared], v0[:, shared])
    for b, (k1, v1, m1, p1) in enumerate(alone):
        mine = table[b, P // page:].long()
        assert torch.equal(k[:, mine], k1[:, mine]) and torch.equal(v[:, mine], v1[:, mine])
        assert torch.equal(mo[:, b, :, :keep[b]], m1[:, 0, :, :keep[b]]) and torch.equal(po[:, b, :, :keep[b]], p1[:, 0, :, :keep[b]])


def evict_want(k, v, table, length, mass, pos, keep, protect, first, page):
    """Head by head on the GPU: a stable sort by class and mass."""
    k, v, mo, po = k.clone(), v.clone(), {}, {}
    L, B, H, cap = mass.shape
    for l in range(L):
        for b in range(B):
            n, N = length[b], min(length[b], keep[b])
            t, j = table[b].long(), torch.arange(n, device=DEV)
            for h in range(H):
                m, p = mass[l, b, h, :n], pos[l, b, h, :n]
                rank = torch.where(p > (p.max() if n else 0) - protect, 1e200, m.double())
                rank = torch.where(j < (first[b] if first else 0), 1e300, rank)
                kept = torch.zeros(n, dtype=torch.bool, device=DEV)
                kept[rank.sort(descending=True, stable=True).indices[:N]] = True
                to, fr = (~kept & (j < N)).nonzero()[:, 0], (kept & (j >= N)).nonzero()[:, 0]
                source = j[:N].clone()
                source[to] = fr
                mo[l, b, h], po[l, b, h] = m[source], p[source]
                for pool in (k, v):
                    pool[l, t[to // page], h, to % page] = pool[l, t[fr // page], h, fr % page]
    return k, v, mo, po


# Units x places decide the kernel's form (152 SMs): 1024 threads up to a unit an SM above 2500 places, else 256; positions in
# shared memory up to 4096, masses up to 40960, moves listed in one go up to 8192 beyond.
LONG, MIXED = [45000], [4100, 0, 9, 300, 4099, 2500, 4097, 1, 33, 3000]
EVICTS = [
    # d, page, L, B, H, lengths, budgets, cap, first
    (64, 32, 2, 10, 8, MIXED, [1000, 5, 4, 299, 4090, 2499, 2048, 1, 1, 2999], 4100, None),           # 160 units of 256 threads
    (128, 64, 2, 10, 8, MIXED, [4000, 5, 4, 100, 4098, 1, 17, 1, 32, 1500], 4100, [40] * 10),
    (64, 256, 1, 40, 4, [41000] + [200, 77, 1500] * 13, [20000] + [100, 70, 1499] * 13, 41001, None),    # and masses read again
    (128, 256, 1, 40, 4, [20500] + [200, 77, 1500] * 13, [20495] + [100, 76, 3] * 13, 41001, [3] * 40),
    (64, 256, 1, 40, 4, [20000] + [9999, 77, 1500] * 13, [9000] + [5000, 70, 1499] * 13, 20000, None),   # and masses in shared memory
    (128, 256, 1, 40, 4, [20001] + [9999, 77, 1500] * 13, [9000] + [5000, 70, 1499] * 13, 20001, [3] * 40),
    (128, 128, 1, 3, 2, [4000, 2700, 3999], [1000, 2695, 3998], 4000, [128, 0, 5]),                      # 1024 threads
    (128, 128, 1, 2, 1, [9000, 5000], [4000, 4995], 9001, None),
    (128, 256, 1, 1, 1, LONG, [22000], 45001, [7]),                                                      # more moves than a list holds
    (64, 256, 1, 1, 2, LONG, [30000], 45001, None)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("alike", [False, True])
@pytest.mark.parametrize("case", range(len(EVICTS)))
def test_evict_every_form(pkg, case, alike, in_place):
    d, page, L, B, H, length, keep, cap, first = EVICTS[case]
    g = torch.Generator(device=DEV).manual_seed(case)
    blocks = [-(-n // page) for n in length]
    pages = sum(blocks) + 1
    k, v = (torch.randn(L, pages, H, page, d, generator=g, device=DEV).to(torch.bfloat16 if case % 2 else torch.float16) for _ in range(2))
    order = torch.randperm(pages, generator=g, device=DEV).tolist()
    table = ints([[order.pop() for _ in range(n)] + [-1] * (max(blocks) - n) for n in blocks])
    mass = torch.rand(L, B, H, cap, generator=g, device=DEV)
    if alike:                                          # a few different masses: ties by the lower place
        mass = (mass * 3).floor() * 0.5
    pos = torch.rand(L, B, H, cap, generator=g, device=DEV).argsort(3).int()
    want = evict_want(k, v, table, length, mass, pos, keep, 20, first, page)
    kv = pkg.PagedKV(k, v, H)
    mass0, pos0 = mass.clone(), pos.clone()
    mo, po = (mass, pos) if in_place else (torch.full_like(mass, -5), torch.full_like(pos, -5))
    new = ints([-7] * B)
    kv.evict(table, ints(length), mass, pos, ints(keep), mo, po, new, protect=20, first=ints(first) if first else None)
    torch.cuda.synchronize()
    assert new.tolist() == [min(n, x) for n, x in zip(length, keep)] and kv.status() == 0
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    for (l, b, h), m in want[2].items():
        n = len(m)
        assert torch.equal(mo[l, b, h, :n], m) and torch.equal(po[l, b, h, :n], want[3][l, b, h])
        if in_place:
            assert torch.equal(mo[l, b, h, n:], mass0[l, b, h, n:]) and torch.equal(po[l, b, h, n:], pos0[l, b, h, n:])
        else:
            assert (mo[l, b, h, n:] == -5).all() and (po[l, b, h, n:] == -5).all()
    if not in_place:
        assert torch.equal(mass, mass0) and torch.equal(pos, pos0)


# ---------------------------------------------------------------------------
# the oddest batches, all four
# ---------------------------------------------------------------------------
def lost_rows(c, sequences):
    lost = torch.zeros(c.starts[-1], dtype=torch.bool, device=DEV)
    for b in sequences:
        lost[c.starts[b]:c.starts[b + 1]] = True
    return lost


def check_but(c, got, want, lost):
    """Lost rows are NaN, the others within the tolerance."""
    n = c.starts[-1]
    assert got[0][:n][lost].isnan().all() and got[1][:n][lost].isnan().all()
    out, lse = got[0].clone(), got[1].clone()
    out[:n][lost], lse[:n][lost] = want[0][lost].to(c.dt), want[1][lost].float()
    check_shared(c, (out, lse), want)


FORMS = {    # heads, kv heads, d, page, groups, tails, new rows
    "clusters": (12, 12, 64, 16, [(2, 300), (2, 130)], [20, 40], [1]),
    "four warps": (40, 8, 128, 32, [(20, 256), (14, 400)], [5, 60], [1]),
    "cut": (16, 2, 64, 16, [(2, 6000), (1, 700)], [17, 900], [1]),
    "tiles": (40, 8, 128, 64, [(3, 900), (2, 300)], [30, 200], [25, 31]),
    "two tiles": (64, 8, 64, 64, [(8, 700), (9, 520), (7, 260)], [0, 33], [12])}


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("form", list(FORMS))
def test_attend_shared_over_bad_pages(pkg, form, dt):
    """A page of a group's prefix that is none voids the group, one of a sequence's own tokens that sequence."""
    heads, H, d, page, groups, tail, new = FORMS[form]
    c = Grouped(DT[dt], heads, H, d, page, groups, tail, new, seed=3)
    want, first = reference(c), groups[0][0]
    kept = c.table.clone()
    c.table[first, 1] = 1 << 30                        # the second group's prefix, by the table of its first sequence
    c.table[1, (c.ctx[1] + c.new[1] - 1) // page] = -1     # the last page of sequence 1
    got = run_shared(pkg, c)
    assert got[2].status(check=False) == pkg.FLAG_BAD_PAGE
    check_but(c, got, want, lost_rows(c, [1] + list(range(first, first + groups[1][0]))))
    c.table = kept
    check_shared(c, run_shared(pkg, c, kv=got[2]), want)   # nothing stays behind
    assert got[2].status() == 0


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("form", list(FORMS))
def test_attend_shared_infinite_values(pkg, form, dt):
    """Infinities in V of the prefix, of own tokens and of drafts that some rows do not see reach the rows that see them alone."""
    heads, H, d, page, groups, tail, new = FORMS[form]
    c = Grouped(DT[dt], heads, H, d, page, groups, tail, new, seed=4)
    for b, j, ch in ((0, 7, 3), (groups[0][0], groups[1][1] // 128 * 128 - 1, 5), (1, c.ctx[1], 9), (1, c.ctx[1] - 1, 11)):
        c.v[:, int(c.table[b, j // page]), H - 1, j % page, ch] = math.inf if ch != 5 else -math.inf
    check_shared(c, run_shared(pkg, c), reference(c))
    bits = tree_bits(c.new, 6)
    check_shared(c, run_shared(pkg, c, bits), reference(c, bits=bits))


@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("form", list(FORMS))
def test_attend_shared_huge_scores_leave_the_largest(pkg, form, where):
    """Scores of 1e10, the next lower one a hundredth of it away or further: one token, of the prefix or of the sequence's own
    cached ones, has all the weight."""
    heads, H, d, page, groups, tail, new = FORMS[form]
    most = 6e4
    c = Grouped(torch.bfloat16, heads, H, d, page, groups, [x + 3 for x in tail], new, seed=5)
    P = [p for n, p in groups for _ in range(n)]
    best = []
    for b, (a, t) in enumerate(zip(c.ctx, c.new)):
        size = -most * torch.arange(1, a + t + 1, dtype=torch.float64) / (a + t) * 0.5
        best.append(P[b] // 2 if where == "prefix" else P[b] + 1)
        size[best[-1]] = most
        if where == "own":
            size[P[b] // 2] = most / 2
        at = torch.arange(a + t, device=DEV)
        c.k[:, c.table[b].long()[at // page], :, at % page] = size.to(c.dt).to(DEV)[None, :, None, None].expand(2, -1, H, d).transpose(0, 1)
    # (the groups' prefixes are written by each of their sequences: alike but for the rest of negative sizes)
    c.q[:] = most
    out, lse, kv = run_shared(pkg, c)
    for b, (a, t) in enumerate(zip(c.ctx, c.new)):
        v = c.get(c.v, 1, b, a + t)[best[b]].repeat_interleave(heads // H, 0)
        assert torch.equal(out[c.starts[b]:c.starts[b + 1]], v[None].expand(t, -1, -1))
        z = float(torch.tensor(most, dtype=c.dt)) ** 2 * d ** 0.5
        assert torch.allclose(lse[c.starts[b]:c.starts[b + 1]].double(), torch.full((t, heads), z, dtype=torch.float64, device=DEV), rtol=(d + 4) * 2.0 ** -23, atol=0)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("heads,H,d,ctx,new,blocks,prefix", [
    (12, 12, 64, 300, 1, 17, 256), (12, 12, 64, 300, 1, 16, 256), (40, 8, 128, 250, 40, 16, 250), (16, 1, 64, 600, 3, 8, 500), (40, 8, 128, 128, 300, 9, 128)])
def test_attend_shared_and_weigh_past_the_page_table(pkg, dt, heads, H, d, ctx, new, blocks, prefix):
    """Sequences longer than their table end where it does, whatever of that is the prefix."""
    c = Grouped(DT[dt], heads, H, d, 16, [(2, prefix)], [ctx - prefix], [new], seed=blocks)
    cap = 16 * blocks
    kv = pkg.PagedKV(c.k, c.v, heads)
    batch = kv.batch(c.table[:, :blocks].contiguous(), ints(c.ctx), ints(c.starts))
    out, lse = (torch.full((c.rows, heads, *x), 7.0, dtype=y, device=DEV) for x, y in (((d,), c.dt), ((), torch.float32)))
    kv.attend(1, batch, c.q, out, lse=lse, prefix=kv.prefix(ints([0, 2]), ints([prefix]), c.rows))
    assert kv.status(check=False) == pkg.FLAG_CAPACITY
    # the same rows over the tokens that there are: drafts behind the table's end are seen by none
    seen = max(0, cap - c.ctx[0])
    if c.ctx[0] >= cap:                                # cached tokens alone, all rows alike
        c.ctx = [cap] * 2
        want = reference(c, bits=[0] * c.starts[-1])
    else:
        want = reference(c, bits=[(1 << min(i + 1, seen)) - 1 for t in c.new for i in range(t)])
    check_shared(c, (out, lse), want)
    mass = torch.full((2, H, ctx + new), 3.0, device=DEV)
    kv.weigh(1, batch, c.q, lse, mass, mass, decay=0.0, gain=1.0)
    assert kv.status(check=False) == pkg.FLAG_CAPACITY
    assert (mass[:, :, cap:] == 3).all()
    # each row's weights sum to 1, within twice 2 ds, of the weights and of lse: scale sum |q k| is 12 at most for these rows
    # (its mean is 7.2 at d = 128, 5.1 at 64, six deviations 4.6), 4 (d + 4) 2^-23 12 < 2^-10, the sums' roundings far below
    total = mass[:, :, :cap].double().sum(2)
    assert ((total - new * (heads // H)).abs() <= 2.0 ** -9 * new * (heads // H)).all()


@pytest.mark.parametrize("new", [[1, 0, 2], [40, 70, 0]])
def test_rows_before_the_first_sequence_are_left_as_they_were(pkg, new):
    c = Grouped(torch.bfloat16, 8, 2, 64, 16, [(2, 256), (1, 130)], [9, 30], new, seed=5)
    n, lead = c.starts[-1], 5
    q = torch.cat([c.randn(lead, 8, 64), c.q])
    want = reference(c)
    kv = pkg.PagedKV(c.k, c.v, 8)
    batch = kv.batch(c.table, ints(c.ctx), ints([lead + x for x in c.starts]))
    out, lse = torch.full_like(q, 7), torch.full(q.shape[:2], 7.0, device=DEV)
    kv.attend(1, batch, q, out, lse=lse, prefix=kv.prefix(c.starts_of_groups(), ints(c.prefixes), len(q)))
    assert (out[:lead] == 7).all() and (lse[:lead] == 7).all()
    check_shared(c, (out[lead:], lse[lead:]), want)
    mass = torch.rand(3, 2, 400, generator=c.g, device=DEV)
    before, where = mass.clone(), torch.full((3, 2, 400), -9, dtype=torch.int32, device=DEV)
    given = torch.randint(0, 1000, (len(q),), device=DEV, dtype=torch.int32)
    kv.weigh(1, batch, q, lse, mass, mass, where, positions=given, decay=0.75, gain=0.5)
    w, tol = weigh_reference(c, lse[lead:lead + n], before, 0.75, 0.5)
    assert ((mass.double() - w).abs() <= tol).all()
    for b, (a, t) in enumerate(zip(c.ctx, new)):
        assert (where[b, :, a:a + t] == given[lead + c.starts[b]:lead + c.starts[b + 1]]).all()
        assert (where[b, :, :a] == -9).all() and (where[b, :, a + t:] == -9).all()
    k, v, q_out, w = c.randn(len(q), 2, 64), c.randn(len(q), 2, 64), torch.full_like(q, 7), torch.ones(64, device=DEV)
    k0 = c.k.clone()
    kv.append(0, batch, k, v, q=q, q_out=q_out, q_norm=w, k_norm=w)
    assert (q_out[:lead] == 7).all() and (q_out[lead + n:] == 7).all() and not (q_out[lead:lead + n] == 7).all(2).any()
    for b, (a, t) in enumerate(zip(c.ctx, new)):
        at = torch.arange(a, a + t, device=DEV)
        assert torch.equal(c.get(c.v, 0, b, a + t)[a:], v[lead + c.starts[b]:lead + c.starts[b + 1]])
        k0[0, c.table[b].long()[at // 16], :, at % 16] = c.k[0, c.table[b].long()[at // 16], :, at % 16]
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16)) and kv.status() == 0


@pytest.mark.parametrize("t", [40, 70])
def test_drafts_past_the_masks_words_are_seen_by_no_row(pkg, t):
    c = Grouped(torch.float16, 6, 2, 64, 16, [(3, 200)], [10], [t], seed=t)
    bits = [(1 << 32) - 1] * (3 * t)
    kv = pkg.PagedKV(c.k, c.v, 6)
    batch = kv.batch(c.table, ints(c.ctx), ints(c.starts), mask_words(bits + [0] * 3, 1))
    out, lse = torch.full_like(c.q, 7), torch.full((c.rows, 6), 7.0, device=DEV)
    kv.attend(1, batch, c.q, out, lse=lse, prefix=kv.prefix(c.starts_of_groups(), ints(c.prefixes), c.rows))
    check_shared(c, (out, lse), reference(c, bits=bits))
    mass = torch.rand(3, 2, 210 + t, generator=c.g, device=DEV)
    before = mass.clone()
    kv.weigh(1, batch, c.q, lse, mass, mass, decay=0.5, gain=1.0)
    w, tol = weigh_reference(c, lse[:3 * t], before, 0.5, 1.0, bits)
    assert ((mass.double() - w).abs() <= tol).all()
    assert (mass[:, :, 210 + 32:] == 0).all() and kv.status() == 0


def test_append_normed_bad_pages_and_lengths(pkg):
    """Rows whose place is none are not stored, their queries are; flags as of append."""
    c = Case(torch.float16, 8, 2, 128, 16, [20, 14, 40, 100], [3, 4, 1, 2], seed=9, extra_rows=1)
    kv = pkg.PagedKV(c.k, c.v, 8)
    wq, wk = (1 + 0.1 * torch.randn(128, generator=c.g, device=DEV) for _ in range(2))
    q, k, v = c.randn(c.rows, 8, 128), c.randn(c.rows, 2, 128), c.randn(c.rows, 2, 128)
    inv = torch.rand(32, generator=c.g, device=DEV)
    pos, axis = torch.randint(0, 999, (c.rows, 2), generator=c.g, device=DEV, dtype=torch.int32), (torch.arange(32, device=DEV) % 2).int()
    want = torch.zeros_like(q)
    kv.append(0, c.batch(kv), k, v, q=q, q_out=want, positions=pos, inv_freq=inv, q_norm=wq, k_norm=wk, axis=axis)
    assert kv.status() == 0
    c.table[1, 1] = c.k.shape[1]                       # sequence 1: places 14, 15 and 16, 17
    k0, v0 = c.k.clone(), c.v.clone()
    out = torch.zeros_like(q)
    kv.append(1, kv.batch(c.table[:, :4].contiguous(), ints([20, 14, -1, 100]), ints(c.starts)), k, v, q=q, q_out=out, positions=pos, inv_freq=inv,
              q_norm=wq, k_norm=wk, axis=axis)
    assert kv.status(check=False) == pkg.FLAG_BAD_PAGE | 16 | pkg.FLAG_CAPACITY
    assert torch.equal(out, want)
    for b, i, at in ((0, 0, 20), (0, 1, 21), (0, 2, 22), (1, 0, 14), (1, 1, 15)):
        pg = int(c.table[b, at // 16])
        assert torch.equal(c.v[1, pg, :, at % 16], v[c.starts[b] + i]) and torch.equal(c.k[1, pg, :, at % 16], c.k[0, pg, :, at % 16])
        k0[1, pg, :, at % 16], v0[1, pg, :, at % 16] = c.k[1, pg, :, at % 16], c.v[1, pg, :, at % 16]
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16)) and torch.equal(c.v.view(torch.int16), v0.view(torch.int16))


def test_pages_behind_two_to_the_31_elements(pkg):
    """Offsets that do not fit 32 bits: three layers of 2^30 elements each, the work in the last one; eviction in all."""
    c = Grouped(torch.float16, 4, 2, 64, 256, [(2, 600), (1, 300)], [40, 500], [1, 30], layers=3, spare=2 ** 15 - 20, seed=31)
    assert c.k.numel() > 2 ** 31 and c.k[:2].numel() * 2 > 2 ** 31
    kv = pkg.PagedKV(c.k, c.v, 4)
    n = c.starts[-1]
    q, k, v, w = c.q.clone(), c.randn(c.rows, 2, 64), c.randn(c.rows, 2, 64), torch.ones(64, device=DEV)
    kv.append(2, c.batch(kv), k, v, q=q, q_out=c.q, q_norm=w, k_norm=w, eps=1e-6)
    torch.cuda.synchronize()
    for x, y in ((torch.cat([c.get(c.k, 2, b, a + t)[a:] for b, (a, t) in enumerate(zip(c.ctx, c.new))]), k[:n]), (c.q[:n], q[:n])):
        y = y.double() / torch.sqrt((y.double() ** 2).mean(2, keepdim=True) + 1e-6)
        assert ((x.double() - y).abs() <= (2.0 ** -11 + 2.0 ** -19) * y.abs() + 2.0 ** -25).all()
    out, lse, _ = run_shared(pkg, c, kv=kv, layer=2)
    check_shared(c, (out, lse), reference(c, layer=2))
    mass = torch.rand(3, 3, 2, 1200, generator=c.g, device=DEV)
    before = mass[2].clone()
    kv.weigh(2, c.batch(kv), c.q, lse, mass[2], mass[2], decay=0.75, gain=0.5)
    want, tol = weigh_reference(c, lse, before, 0.75, 0.5, layer=2)
    assert ((mass[2].double() - want).abs() <= tol).all()
    pos = torch.rand(3, 3, 2, 1200, generator=c.g, device=DEV).argsort(3).int()
    length, keep = [a + t for a, t in zip(c.ctx, c.new)], [620, 600, 341 - 4]
    first = [512, 512, 0]                              # the pages that the group shares
    want = evict_want(c.k, c.v, c.table, length, mass, pos, keep, 9, first, 256)
    new = ints([0, 0, 0])
    kv.evict(c.table, ints(length), mass, pos, ints(keep), mass, pos, new, protect=9, first=ints(first))
    assert kv.status() == 0 and new.tolist() == keep
    assert torch.equal(c.k.view(torch.int16), want[0].view(torch.int16)) and torch.equal(c.v.view(torch.int16), want[1].view(torch.int16))
    for (l, b, h), m in want[2].items():
        assert torch.equal(mass[l, b, h, :len(m)], m) and torch.equal(pos[l, b, h, :len(m)], want[3][l, b, h])


def test_the_most_sequences(pkg):
    """65536 sequences in groups of four behind 128 tokens, up to 40 of their own: append, attend, weigh, evict."""
    B, H, heads, d, page, n = 65536, 1, 2, 64, 16, 176
    g = torch.Generator(device=DEV).manual_seed(2)
    G = B // 4
    own = torch.randint(0, 40, (B,), generator=g, device=DEV, dtype=torch.int32)
    ctx = own + 128
    pages = G * 8 + B * 3
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.cat([order[:G * 8].view(G, 1, 8).expand(G, 4, 8).reshape(B, 8), order[G * 8:].view(B, 3)], 1).contiguous()
    k, v = (torch.randn(1, pages, H, page, d, generator=g, device=DEV).half() for _ in range(2))
    kv = pkg.PagedKV(k, v, heads)
    qkv = torch.randn(B, heads + 2 * H, d, generator=g, device=DEV).half()
    q, w = torch.empty(B, heads, d, dtype=torch.float16, device=DEV), torch.ones(d, device=DEV)
    batch = kv.batch(table, ctx, torch.arange(B + 1, dtype=torch.int32, device=DEV))
    prefix = kv.prefix(torch.arange(0, B + 1, 4, dtype=torch.int32, device=DEV), torch.full((G,), 128, dtype=torch.int32, device=DEV), B)
    kv.append(0, batch, qkv[:, heads:heads + H], qkv[:, heads + H:], q=qkv[:, :heads], q_out=q, q_norm=w)
    out, lse = torch.empty_like(q), torch.empty(B, heads, device=DEV)
    kv.attend(0, batch, q, out, lse=lse, prefix=prefix)
    mass = torch.rand(B, H, n, generator=g, device=DEV)
    mass0, pos = mass.clone(), torch.arange(n, dtype=torch.int32, device=DEV).expand(B, H, n).contiguous()
    kv.weigh(0, batch, q, lse, mass, mass, pos, decay=0.5, gain=0.25)
    assert kv.status() == 0
    row, at = torch.arange(B, device=DEV), torch.arange(n, device=DEV)
    y = qkv[:, :heads].double()
    y = y / torch.sqrt((y * y).mean(2, keepdim=True) + 1e-6)
    assert ((q.double() - y).abs() <= (2.0 ** -11 + 2.0 ** -19) * y.abs() + 2.0 ** -25).all()
    u, scale = 2.0 ** -11, d ** -0.5
    for lo in range(0, B, 8192):
        s = slice(lo, lo + 8192)
        K, V = (x[0][table[s].long()].transpose(1, 2).reshape(8192, n, d).double() for x in (k, v))
        assert torch.equal(K[torch.arange(8192, device=DEV), ctx[s].long()], qkv[s, heads].double())
        z = torch.einsum("bhd,bnd->bhn", q[s].double(), K) * scale
        z = torch.where(at <= ctx[s, None, None], z, -math.inf)
        p = torch.softmax(z, 2)
        o, A = torch.einsum("bhn,bnd->bhd", p, V), torch.einsum("bhn,bnd->bhd", p, V.abs())
        # scale sum |q k| <= scale |q| |k|, |q| = sqrt(d) of a normed row
        ds = (d + 4) * 2.0 ** -23 * float(K.norm(dim=2).amax()) * 1.001
        assert ((out[s].double() - o).abs() <= u * o.abs() + (u + 2 * ds + n * 2.0 ** -23) * A + n * 2.0 ** -25 * float(V.abs().amax()) + 2.0 ** -20 * float(V.abs().amax())).all()
        total = torch.logsumexp(z, 2)
        assert ((lse[s].double() - total).abs() <= ds + n * 2.0 ** -23 + 2.0 ** -22 * (1 + total.abs()) + 2.0 ** -20).all()
        wt = torch.where(at <= ctx[s, None, None], (z - lse[s].double()[..., None]).exp(), 0.0)
        err = (wt * (2 * ds + 2.0 ** -21 * (1 + torch.where(z == -math.inf, 0.0, z).abs() + total.abs()[..., None]) + heads * 2.0 ** -24) + 2.0 ** -126).sum(1)
        old = torch.where(at < ctx[s, None], 0.5 * mass0[s, 0].double(), 0.0)
        want = torch.where(at <= ctx[s, None], old + 0.25 * wt.sum(1), mass0[s, 0].double())
        tol = torch.where(at <= ctx[s, None], 0.25 * err + 2.0 ** -22 * want.abs(), 0.0)
        assert ((mass[s, 0].double() - want).abs() <= tol).all()
    assert (pos == at.int()).all()
    # each keeps its prefix, its newest two and the largest of the rest, up to 140
    keep, new = torch.full((B,), 140, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    length = ctx + 1
    k0, m0 = k.clone(), mass.clone()
    mo, po = torch.zeros_like(mass), torch.full_like(pos, -1)
    kv.evict(table, length, mass[None], pos[None], keep, mo[None], po[None], new, protect=2, first=torch.full((B,), 128, dtype=torch.int32, device=DEV))
    assert kv.status() == 0 and torch.equal(new, torch.minimum(length, keep)) and torch.equal(mass, m0)
    rank = torch.where(at[None] > ctx[:, None] - 2, 1e200, mass[:, 0].double())
    rank = torch.where(at < 128, 1e300, rank)
    rank = torch.where(at[None] < length[:, None], rank, -math.inf)
    by = rank.sort(dim=1, descending=True, stable=True).indices
    stays = torch.zeros(B, n, dtype=torch.bool, device=DEV).scatter_(1, by, at[None] < new[:, None])
    assert torch.equal(po[:, 0].clamp(min=0).long().sum(1), (stays * at).sum(1))           # (positions are the places here)
    live = at[None] < new[:, None]
    assert (po[:, 0][~live] == -1).all()
    assert torch.equal(mo[:, 0][live], mass[:, 0].gather(1, po[:, 0].clamp(min=0).long())[live])
    still = live & stays
    assert torch.equal(po[:, 0][still], at.int().expand(B, n)[still])
    moved = (live & ~stays).nonzero()
    fr = po[moved[:, 0], 0, moved[:, 1]].long()
    assert torch.equal(k[0, table[moved[:, 0], moved[:, 1] // page].long(), 0, moved[:, 1] % page], k0[0, table[moved[:, 0], fr // page].long(), 0, fr % page])
    shared = order[:G * 8].long()
    assert torch.equal(k[:, shared], k0[:, shared])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_outputs_in_the_batchs_own_tensors_are_refused(pkg):
    """One buffer holds the table, lengths, starts, mask and groups, and outputs that begin or end in one of them."""
    B, H, heads, d, n = 3, 2, 4, 64, 3
    k, v = (torch.zeros(1, 9, H, 16, d, device=DEV, dtype=torch.float16) for _ in range(2))
    kv = pkg.PagedKV(k, v, heads)
    q, lse = torch.zeros(n, heads, d, device=DEV, dtype=torch.float16), torch.zeros(n, heads, device=DEV)
    room = n * heads * d // 2                                  # words of an out or q_out
    apart = 2 * room + 64                                      # an output meets one tensor at a time
    buf = torch.zeros(8 * apart, device=DEV, dtype=torch.int32)

    def cut(at, *shape):
        size = int(np.prod(shape))
        return buf[at:at + size].view(*shape)

    places = [(B, 2), (B,), (B + 1,), (n, 1), (2,), (1,)]      # table, ctx, q_start, mask, group_start, prefix_len
    starts = [room + apart * i for i in range(len(places))]
    table, ctx, start, mask, group, length = (cut(at, *s) for at, s in zip(starts, places))
    start.copy_(torch.arange(B + 1))
    batch = kv.batch(table, ctx, start, mask)
    prefix = kv.prefix(group, length, n)
    far = torch.zeros_like(q)
    mass, cap = torch.zeros(B, H, 30, device=DEV), 30
    calls = 0
    for at, shape in zip(starts, places):
        own, last = at < starts[4], at + int(np.prod(shape)) - 1
        for words, where in ((room, last // 4 * 4), (room, (at + 4 - room) // 4 * 4)):          # the tensor's last word is the
            out = cut(where, words).view(torch.float16).view(n, heads, d)                       # output's first, its first the last
            assert where <= last and where + words > at
            bad = [lambda: kv.attend(0, batch, q, out, prefix=prefix)]
            if own:
                bad += [lambda: kv.attend(0, batch, q, out)]
            if own and at != starts[3]:
                bad += [lambda: kv.append(0, batch, far[:, :H], far[:, H:], q=q, q_out=out),
                        lambda: kv.append(0, batch, far[:, :H], far[:, H:], q=q, q_out=out, q_norm=torch.ones(d, device=DEV))]
            for call in bad:
                with pytest.raises(pkg.ConfKVError, match="overlaps"):
                    call()
                calls += 1
        for words in (B * H * cap, n * heads):
            x = cut(last, words)
            if words == n * heads:
                l = x.view(torch.float32).view(n, heads)
                bad = [lambda: kv.attend(0, batch, q, far, lse=l, prefix=prefix)] + ([lambda: kv.attend(0, batch, q, far, lse=l)] if own else [])
            elif own:
                m, p = x.view(torch.float32).view(B, H, cap), x.view(B, H, cap)
                bad = [lambda: kv.weigh(0, batch, q, lse, mass, m), lambda: kv.weigh(0, batch, q, lse, m, m),
                       lambda: kv.weigh(0, batch, q, lse, mass, mass, p)]
            else:
                bad = []
            for call in bad:
                with pytest.raises(pkg.ConfKVError, match="overlaps"):
                    call()
                calls += 1
        # the scratch
        from confidence_gated_kv_logits_gb300.paged import PrefixStruct, SharedPrefix
        need = pkg.load_library().confkv_paged_partial(n, heads, d)
        scratch = PrefixStruct(1, group.data_ptr(), length.data_ptr(), buf.data_ptr() + last // 4 * 16, need)
        with pytest.raises(pkg.ConfKVError, match="overlaps"):
            kv.attend(0, batch, q, far, prefix=SharedPrefix(scratch, (), n, kv._index))
    assert calls == 3 * 8 + 4 + 2 * 2 + 4 * 5 + 2
    assert kv.status() == 0
