// Accumulated attention weight of each cached token and KV head:
//
//   mass_out_t = decay mass_t + gain sum_r exp(scale q_r k_t - lse_r)
//
// over the rows r (new tokens x the group's query heads) that see token t, with
// the rows' lse as attend gave it: the weights are final at once, nothing is
// rescaled, and each token's sum is one thread's, in one order.
//
// Tokens are the products' M (tiles of 128, full whatever the rows are) and query
// rows their N (16 to 128), S = K Q^T in tensor memory: a thread owns a token, so
// the sum over rows needs no other thread, a single token's few rows cost a
// product of N = 16, and there is nothing to join.  An item is some token tiles of
// one KV head of one sequence: two where the rows need several tiles of up to 128
// (whole new tokens, as the heads of a group lie side by side), which go by while K
// stays in shared memory, up to eight where one tile holds all rows.  Items are laid
// end to end by their cost and cut into equal shares.
//
// Roles of a CTA's thirteen warps: two warpgroups take the exponentials of every
// second token tile each, warps 8 and 12 issue their products (one warp alone takes
// as long to issue both's as the exponentials do), warp 9 moves K, warp 10 the query
// rows (both by TMA), warp 11 plans.  Each warpgroup has two accumulators, so that
// products run beside exponentials.
#include <algorithm>
#include <cstddef>

#include "paged_attend.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 416;
constexpr int BT = 128;                   // tokens of a tile (kManyBlock: the boxes are attend's)
constexpr int BR = 128;                   // most query rows of a tile
constexpr float kL2E = 1.4426950408889634f;
constexpr int kFixed = 2;                 // an item's fixed cost in tiles of rows: its K from memory
constexpr int kPlan = 8;                  // items in the planned ring
constexpr int kReaders = 12;              // warps that read it

static_assert(BT == kManyBlock, "boxes of the pools");

template <int D>
struct Weigh {
  static constexpr int TILE = 128 * D * 2;                  // bytes of a K or Q tile
  static constexpr int HALF = 128 * 128;                    // of 64 channels of it
  static constexpr int SK = D == 128 ? 4 : 6, SQ = D == 128 ? 3 : 5;      // stages
  static constexpr int SMEM = (SK + SQ) * TILE;
};

struct Item {
  int more;                               // 0: the CTA's share ends here
  int b, h, T, ctx, len, row0;
  int j0, nb;                             // first token, token tiles
  int tile0, tiles;                       // tiles of rows that see it
};

struct __align__(16) Shared {             // behind the stages
  unsigned long long bars[2 * 6 + 2 * 5 + 4 + 4 + 2 * kPlan + 2];
  Item plan[kPlan];
  __align__(16) float lse[2][2][BR];      // [warpgroup][parity]: lse log2 e, +inf for rows that add nothing
  Sched sched;
  long long scan[kThreads / 32];
  uint32_t tmem;
  int abort;
};
static_assert(offsetof(Shared, lse) % 16 == 0, "lse is read in 16-byte words");

// The items of a sequence's heads.
struct Items : Walk<BR, BT, 0> {
  const int cap, tb, gb1, gb2;            // places of the mass; new tokens of a tile of rows; token tiles of an item
                                          // whose rows are one tile, several
  int tiles, gb, items, all;              // of the sequence: tiles of rows, token tiles of an item, items, token tiles
  __device__ __forceinline__ Items(const Pool& p_, const WeighArgs& a, int tb_, int gb1_)
      : Walk(p_, a.bt, a.rows), cap(a.cap), tb(tb_), gb1(gb1_), gb2(gb1_ < 2 ? 1 : 2) {}
  __device__ __forceinline__ void shape() {
    tiles = (T + tb - 1) / tb;
    gb = tiles > 1 ? gb2 : gb1;
    all = (len + BT - 1) / BT;
    items = (all + gb - 1) / gb;
  }
  __device__ __forceinline__ void sequence(int b_, int& flag) {
    Walk::sequence(b_, flag);
    if (T > 0 && len > cap) {             // places from cap on are dropped
      flag |= CONFKV_FLAG_CAPACITY;
      len = cap;
    }
    shape();
  }
  // the first tile whose rows see a token of item i
  __device__ __forceinline__ int first_tile(int i) const {
    const int x = i * BT * gb - ctx;
    return bt.mask || x <= 0 ? 0 : x / tb;
  }
  __device__ __forceinline__ int count(int i) const { return all - i * gb < gb ? all - i * gb : gb; }      // its token tiles
  __device__ __forceinline__ int full_items() const {       // those of gb tiles that every row sees
    const int whole = all / gb, seen = ctx / (BT * gb) + 1;
    return bt.mask || whole < seen ? whole : seen;
  }
  __device__ __forceinline__ int cost(int i) const { return count(i) * (kFixed + tiles - first_tile(i)); }
  __device__ __forceinline__ long long head_work() const {
    const int n = full_items();
    long long w = static_cast<long long>(n) * (gb * (kFixed + tiles));
#pragma unroll 1
    for (int i = n; i < items; ++i) w += cost(i);
    return w;
  }
};

// bar_wait_warp with its polling out of line: the roles' loops have to stay in the instruction cache
__device__ __noinline__ bool wait_on(uint32_t bar, unsigned parity, volatile int* abort) { return bar_wait_warp(bar, parity, abort); }
__device__ __forceinline__ bool wait_bar(uint32_t bar, unsigned parity, volatile int* abort) {
  return __all_sync(0xffffffffu, bar_try(bar, parity)) || wait_on(bar, parity, abort);
}

// warps of one warpgroup decide together whether they go on (and see what all wrote)
__device__ __forceinline__ bool group_any(int group, bool mine) {
  unsigned any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"(static_cast<unsigned>(mine)), "r"(1 + group)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

struct QueryMaps {                        // q as [rows][heads][d], boxes of 64 channels x a group's heads x n rows
  CUtensorMap one, some, all;
  int n_some, n_all;
};

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads, 1)
k_weigh(const Pool p, const WeighArgs a, const int gb1, const __grid_constant__ CUtensorMap mk, const __grid_constant__ QueryMaps mq) {
  using W = Weigh<D>;
  constexpr int SK = W::SK, SQ = W::SQ;
  extern __shared__ __align__(1024) unsigned char s_raw[];
  Shared& s = *reinterpret_cast<Shared*>(s_raw + W::SMEM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t k_ring = smem_addr(s_raw), q_ring = k_ring + SK * W::TILE, bars = smem_addr(s.bars);
  const uint32_t b_kf = bars, b_ke = b_kf + 8 * SK, b_qf = b_ke + 8 * SK, b_qe = b_qf + 8 * SQ, b_s = b_qe + 8 * SQ,
                 b_free = b_s + 32, b_plan = b_free + 32, b_read = b_plan + 8 * kPlan, b_end = b_read + 8 * kPlan;
  if (tid == 0) {
    // both issuing warps wait for every stage in turn, their own or not, and both give every stage back (were
    // the other's stages passed over, a stage that changes hands could answer a wait by an earlier phase)
    for (int i = 0; i < SK; ++i) {
      bar_init(b_kf + 8 * i, 1);
      bar_init(b_ke + 8 * i, 2);
    }
    for (int i = 0; i < SQ; ++i) {
      bar_init(b_qf + 8 * i, 1);
      bar_init(b_qe + 8 * i, 2);
    }
    for (int i = 0; i < 4; ++i) {
      bar_init(b_s + 8 * i, 1);
      bar_init(b_free + 8 * i, 128);
    }
    for (int i = 0; i < kPlan; ++i) {
      bar_init(b_plan + 8 * i, 1);
      bar_init(b_read + 8 * i, kReaders);
    }
    bar_init(b_end, 1);
    bar_init(b_end + 8, 1);
    s.abort = 0;
    fence_bar_init();
    fence_async();
  }
  if (warp == 10) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_addr(&s.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  pdl_wait();
  pdl_trigger();
  fence_async_global();
  tc_fence_before();
  const int tb = mq.n_all;
  if (a.bt.B > 32) {
    Items w(p, a, tb, gb1);
    sched_init<kThreads>(w, &s.sched, s.scan, 1);
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  unsigned plan = 0;
  auto wait_item = [&](unsigned ahead) {  // the planned item that many further is there (behind the last one there is none)
    return wait_bar(b_plan + 8 * ((plan + ahead) % kPlan), ((plan + ahead) / kPlan) & 1, &s.abort);
  };
  auto item = [&](unsigned ahead) -> const Item& { return s.plan[(plan + ahead) % kPlan]; };
  auto next_item = [&] { return wait_item(0) && item(0).more; };
  auto item_done = [&] {
    __syncwarp();
    if (lane == 0) bar_arrive(b_read + 8 * (plan % kPlan));
    ++plan;
  };
  // rows of a tile
  auto rows_of = [&](const Item& w, int tile) { return min(tb, w.T - tile * tb) * p.g; };

  if (warp == 11) {
    // ---- the plan ----
    Items w(p, a, tb, gb1);
    Sched sh;
    if (a.bt.B <= 32) sh = sched_warp(w, 1, 0, blockIdx.x, gridDim.x);
    else sh = s.sched;
    long long cur = sh.cur, at = 0;        // at: the cost at which the next item starts
    int i = 0, flag = 0;
    if (cur < sh.end) {
      w.b = sh.b;
      w.T = sh.T;
      w.ctx = sh.ctx;
      w.len = sh.len;
      w.row0 = sh.row0;
      w.shape();
      // the share's first item: the first that starts in it
      w.h = static_cast<int>(quotient(cur - sh.seq0, sh.head));
      at = sh.seq0 + w.h * sh.head;
      const int full = w.gb * (kFixed + w.tiles), n = w.full_items();
      const long long j = quotient(cur - at + full - 1, full);
      i = j < n ? static_cast<int>(j) : n;
      at += static_cast<long long>(i) * full;
      while (i < w.items && at < cur) at += w.cost(i++);
    }
    for (bool more = true; more; ++plan) {
      while (at < sh.end && cur < sh.end && i >= w.items) {
        i = 0;
        if (++w.h == p.Hkv) {
          w.h = 0;
          do w.sequence(w.b + 1, flag); while (w.T <= 0);
        }
      }
      more = cur < sh.end && at < sh.end;
      if (plan >= kPlan && !wait_bar(b_read + 8 * (plan % kPlan), (plan / kPlan - 1) & 1, &s.abort)) break;
      if (lane == 0) {
        s.plan[plan % kPlan] = more ? Item{1, w.b, w.h, w.T, w.ctx, w.len, w.row0, i * BT * w.gb, w.count(i), w.first_tile(i), w.tiles} : Item{};
        bar_arrive(b_plan + 8 * (plan % kPlan));
      }
      if (more) at += w.cost(i++);
    }
  } else if (warp == 9) {
    // ---- K ----
    const uint64_t pol = stream_policy();
    const int rows_per = p.ps < BT ? p.ps : BT, boxes = BT / rows_per;
    unsigned slot = 0;
    int flag = 0;
    bool ok = true;
    // two token tiles at a time: a lane has one box, both tiles' boxes and their channel halves side by side
    constexpr int HV = D / 64;
    const int x = lane / (8 * HV), i = lane % (8 * HV) / HV, half = lane % HV;
    auto page_of = [&](const Item& w, int y0) {
      const int j = w.j0 + (y0 + x) * BT + i * rows_per;
      return w.more && x < 2 && y0 + x < w.nb && i < boxes && j < w.len
                 ? a.bt.table[static_cast<size_t>(w.b) * a.bt.max_blocks + (j >> p.ps_shift)] : 0;
    };
    ok = wait_item(0);
    int page = ok ? page_of(item(0), 0) : 0;
    while (ok && item(0).more) {
      const Item& w = item(0);
      for (int y0 = 0; ok && y0 < w.nb; y0 += 2) {
        // the next boxes' pages are asked for before these boxes
        const bool ends = y0 + 2 >= w.nb;
        if (ends && !wait_item(1)) {
          ok = false;
          break;
        }
        const int page1 = ends ? page_of(item(1), 0) : page_of(w, y0 + 2);
        const bool none = static_cast<unsigned>(page) >= static_cast<unsigned>(p.NP);
        for (int y = y0; y < y0 + 2 && y < w.nb; ++y, ++slot) {
          const unsigned st = slot % SK;
          if (slot >= SK && !wait_bar(b_ke + 8 * st, (slot / SK - 1) & 1, &s.abort)) {
            ok = false;
            break;
          }
          const int j0 = w.j0 + y * BT, live = (w.len - j0 + rows_per - 1) >> (p.ps < BT ? p.ps_shift : 7), n = live < boxes ? live : boxes;
          if (lane == 0) bar_expect(b_kf + 8 * st, static_cast<unsigned>(n * rows_per * D * 2));
          __syncwarp();
          if (x == y - y0 && i < n) {
            if (none) flag = CONFKV_FLAG_BAD_PAGE;
            const int j = j0 + i * rows_per;
            const int row = none ? kNoRows : (((a.layer * p.NP + page) * p.Hkv + w.h) << p.ps_shift) + (j & (p.ps - 1));
            tma_box(k_ring + st * W::TILE + half * W::HALF + i * rows_per * 128, &mk, 64 * half, row, b_kf + 8 * st, pol);
          }
        }
        page = page1;
      }
      item_done();
    }
    if (flag) atomicOr(p.err, flag);
    if (!ok)                              // no copy may land after the CTA has gone
      for (unsigned k = slot > SK ? slot - SK : 0; k < slot; ++k) bar_drain(b_kf + 8 * (k % SK), (k / SK) & 1);
  } else if (warp == 10) {
    // ---- query rows ----
    unsigned slot = 0;
    bool ok = true;
    while (ok && next_item()) {
      const Item& w = item(0);
      for (int t = w.tile0; ok && t < w.tiles; ++t, ++slot) {
        const unsigned st = slot % SQ;
        if (slot >= SQ && !wait_bar(b_qe + 8 * st, (slot / SQ - 1) & 1, &s.abort)) {
          ok = false;
          break;
        }
        const int left = w.T - t * tb;
        const int n = left == 1 ? 1 : left <= mq.n_some ? mq.n_some : mq.n_all;
        const CUtensorMap* map = left == 1 ? &mq.one : left <= mq.n_some ? &mq.some : &mq.all;
        if (lane == 0) bar_expect(b_qf + 8 * st, static_cast<unsigned>(n * p.g * D * 2));
        __syncwarp();
        if (lane < D / 64)
          tma_rows(q_ring + st * W::TILE + lane * W::HALF, map, 64 * lane, w.h * p.g, w.row0 + t * tb, b_qf + 8 * st);
      }
      item_done();
    }
    if (!ok)
      for (unsigned k = slot > SQ ? slot - SQ : 0; k < slot; ++k) bar_drain(b_qf + 8 * (k % SQ), (k / SQ) & 1);
  } else if (warp == 8 || warp == 12) {
    // ---- a warpgroup's products, S = K Q^T (the warp stays together; one elected thread issues) ----
    const int g = warp == 12;
    constexpr uint32_t hi = umma_hi(1024);
    const uint32_t k_lo = uniform(umma_lo(k_ring, 16)), q_lo = uniform(umma_lo(q_ring, 16));
    unsigned ks = 0, qs = 0, used = 0;                    // stages passed; products so far
    bool ok = true;
    while (ok && next_item()) {
      const Item& w = item(0);
      const int nb = w.nb;
      for (int t = w.tile0; ok && t < w.tiles; ++t, ++qs) {
        const unsigned st = qs % SQ;
        ok = wait_bar(b_qf + 8 * st, (qs / SQ) & 1, &s.abort);
        const uint32_t idesc = umma_idesc(BF, 128, (rows_of(w, t) + 15) & ~15, false), qt = uniform(q_lo + st * (W::TILE / 16));
        for (int x = 0; ok && x < nb; ++x) {
          const unsigned k = ks + x;
          if (t == w.tile0) ok = wait_bar(b_kf + 8 * (k % SK), (k / SK) & 1, &s.abort);
          if ((x & 1) != g) {
            if (ok && t == w.tile0) bar_arrive_warp(b_ke + 8 * (k % SK));
            continue;
          }
          const unsigned n = used++;
          const uint32_t acc = 2 * g + (n & 1);
          if (ok && n >= 2) ok = wait_bar(b_free + 8 * acc, (n / 2 - 1) & 1, &s.abort);
          if (!ok) break;
          tc_fence_after();
          const uint32_t kt = uniform(k_lo + (k % SK) * (W::TILE / 16)), d = uniform(tmem + acc * BR);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t o = ((c >> 2) * W::HALF + (c & 3) * 32) / 16;
            umma_ss(d, kt + o, hi, qt + o, hi, idesc, c > 0);
          }
          umma_commit(b_s + 8 * acc);
          if (t + 1 == w.tiles) umma_commit(b_ke + 8 * (k % SK));
        }
        if (ok) umma_commit(b_qe + 8 * st);
      }
      if (!ok) break;
      ks += nb;
      item_done();
    }
    // products in flight end before the CTA does
    if (!ok) {
      umma_commit(b_end + 8 * g);
      bar_drain(b_end + 8 * g, 0);
    }
    __syncwarp();
  } else {
    // ---- weights ----
    const int g = warp >> 2, r = tid & 127;               // warpgroup; token of a tile, and column whose lse it brings
    const uint32_t ts0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 2 * g * BR;
    const float c = a.scale * kL2E;
    const int rt = r / p.g, rh = r - rt * p.g;
    // the mass of tile x's token, and the lse of a column of rows' tile t
    auto mass_of = [&](const Item& w, int x) {
      const int j = w.j0 + x * BT + r;
      return w.more && x < w.nb && j < w.len && j < w.ctx ? a.mass[(static_cast<size_t>(w.b) * p.Hkv + w.h) * a.cap + j] : 0.0f;
    };
    auto lse_of = [&](const Item& w, int t) {
      const int tok = t * tb + rt;
      return w.more && t < w.tiles && rt < tb && tok < w.T ? a.lse[static_cast<size_t>(w.row0 + tok) * p.Hq + w.h * p.g + rh] : -INFINITY;
    };
    // N columns' weights into four sums, in the columns' order; the steps of neighbouring groups of eight are
    // interleaved (written in order: the schedule is otherwise one chain after another)
    uint64_t sum[4];
    auto weights = [&](auto const& sv, const float* lse, auto keep) {
      constexpr int N = sizeof(sv) / 4;
      const float4* lq = reinterpret_cast<const float4*>(lse);
      float z[2][8];
      uint64_t e[2][4];
      auto args = [&](int k) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float4 l = lq[2 * k + y];
          z[k & 1][4 * y] = fma_o(__uint_as_float(sv[8 * k + 4 * y]), c, -l.x);
          z[k & 1][4 * y + 1] = fma_o(__uint_as_float(sv[8 * k + 4 * y + 1]), c, -l.y);
          z[k & 1][4 * y + 2] = fma_o(__uint_as_float(sv[8 * k + 4 * y + 2]), c, -l.z);
          z[k & 1][4 * y + 3] = fma_o(__uint_as_float(sv[8 * k + 4 * y + 3]), c, -l.w);
        }
      };
      args(0);
#pragma unroll
      for (int k = 0; k <= N / 8; ++k) {
        if (k + 1 < N / 8) args(k + 1);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if (k < N / 8) {
            const float e0 = ex2_o(z[k & 1][2 * y]), e1 = ex2_o(z[k & 1][2 * y + 1]);
            e[k & 1][y] = pair(keep(8 * k + 2 * y, e0), keep(8 * k + 2 * y + 1, e1));
          }
          if (k > 0) sum[y] = add2_o(sum[y], e[(k - 1) & 1][y]);
        }
      }
    };
    unsigned used = 0, steps = 0;                         // products; tiles of rows
    bool ok = wait_item(0);
    float before = ok ? mass_of(item(0), g) : 0.0f, next = ok ? lse_of(item(0), item(0).tile0) : 0.0f;
    while (!group_any(g, !(ok && item(0).more))) {
      const Item& w = item(0);
      const int nb = w.nb;
      sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
      ok = wait_item(1);
      bool dead = !ok;
      for (int t = w.tile0; t < w.tiles; ++t, ++steps) {
        float* lse = s.lse[g][steps & 1];
        lse[r] = next == -INFINITY ? INFINITY : next * kL2E;
        // the next tile's lse, the next item's behind the last
        if (t + 1 < w.tiles) next = lse_of(w, t + 1);
        else if (ok) next = lse_of(item(1), item(1).tile0);
        if (group_any(g, dead)) {
          dead = true;
          break;
        }
        const int n = rows_of(w, t);
#pragma unroll 1
        for (int x = g; x < nb; x += 2, ++used) {
          const int j = w.j0 + x * BT + r;
          const uint32_t acc = used & 1, ts = ts0 + acc * BR;
          const bool last = t + 1 == w.tiles;
          float after = before;
          if (last) after = x + 2 < nb ? mass_of(w, x + 2) : ok ? mass_of(item(1), g) : 0.0f;
          if (!wait_bar(b_s + 8 * (2 * g + acc), (used >> 1) & 1, &s.abort)) {
            dead = true;                  // the others learn of it at the next decision, to which all four warps come
            break;
          }
          tc_fence_after();
          // columns that see this token: causal ones from its own row on
          const int past = j - w.ctx - t * tb;            // new tokens of the tile that come before it
          const bool masked = a.bt.mask && w.j0 + x * BT + BT > w.ctx;
          const int from = a.bt.mask || past <= 0 ? 0 : past * p.g;
          if (masked) {
            // by the batch's mask, column by column
            int tok = t * tb, left = p.g;                 // the column's new token, its columns that are left
#pragma unroll 1
            for (int q = 0; q < n; q += 8) {
              uint32_t sv[8];
              __syncwarp();
              tmem_ld8(sv, ts + q);
              tmem_wait_ld(sv);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const bool seen = q + e < n && (seen_bits(a.bt, static_cast<size_t>(w.row0 + tok), tok, w.ctx, w.len, j) & 1u);
                const float y = seen ? ex2f(fmaf(__uint_as_float(sv[e]), c, -lse[q + e])) : 0.0f;
                sum[e >> 1] = add2(sum[e >> 1], e & 1 ? pair(0.0f, y) : pair(y, 0.0f));
                if (--left == 0) {
                  left = p.g;
                  if (tok + 1 < w.T) ++tok;
                }
              }
            }
          } else {
            int q = 0;
            if (!__any_sync(0xffffffffu, from > 0)) {
#pragma unroll 1
              for (; q + 32 <= n; q += 32) {
                uint32_t sv[32];
                tmem_ld32(sv, ts + q);
                tmem_wait_ld(sv);
                weights(sv, lse + q, [](int, float y) { return y; });
              }
            }
#pragma unroll 1
            for (; q < n; q += 8) {
              uint32_t sv[8];
              tmem_ld8(sv, ts + q);
              tmem_wait_ld(sv);
              weights(sv, lse + q, [&](int col, float y) { return q + col >= from && q + col < n ? y : 0.0f; });
            }
          }
          tc_fence_before();
          bar_arrive(b_free + 8 * (2 * g + acc));
          if (last) {
            if (j < w.len) {
              const size_t at = (static_cast<size_t>(w.b) * p.Hkv + w.h) * a.cap + j;
              const float2 y = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
              a.mass_out[at] = a.decay * before + a.gain * (y.x + y.y);
              if (j >= w.ctx && a.pos) a.pos[at] = a.positions ? a.positions[w.row0 + j - w.ctx] : j;
            }
            sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
          }
          before = after;
        }
      }
      // (a warpgroup without a tile in this item has not read the next one's mass)
      if (nb <= g && ok) before = mass_of(item(1), g);
      ok = ok && !dead;
      item_done();
    }
  }
  __syncthreads();
  if (s.abort && tid == 0) atomicOr(p.err, CONFKV_FLAG_TIMEOUT);
  if (warp == 10) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  }
}

template <typename F>
cudaError_t each_weigh(F&& f) {
  cudaError_t e = f(k_weigh<true, 64>, true, 64, Weigh<64>::SMEM);
  if (e == cudaSuccess) e = f(k_weigh<true, 128>, true, 128, Weigh<128>::SMEM);
  if (e == cudaSuccess) e = f(k_weigh<false, 64>, false, 64, Weigh<64>::SMEM);
  return e == cudaSuccess ? f(k_weigh<false, 128>, false, 128, Weigh<128>::SMEM) : e;
}
static_assert(Weigh<128>::SMEM + sizeof(Shared) <= 232448, "a CTA's shared memory");

}  // namespace

cudaError_t setup_weigh() {
  return each_weigh([](auto kernel, bool, int, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem + static_cast<int>(sizeof(Shared)));
  });
}

cudaError_t launch_weigh(const Pool& p, const WeighArgs& a, const AttendMaps& m, int ctas, cudaStream_t s) {
  QueryMaps mq;
  mq.n_all = BR / p.g;
  mq.n_some = std::min(8, mq.n_all);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.d), static_cast<cuuint64_t>(p.Hq), static_cast<cuuint64_t>(a.rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.d) * 2, static_cast<cuuint64_t>(a.qs) * 2};
  struct {
    CUtensorMap* map;
    int n;
  } const all[] = {{&mq.one, 1}, {&mq.some, mq.n_some}, {&mq.all, mq.n_all}};
  for (const auto& x : all) {
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.g), static_cast<cuuint32_t>(x.n)};
    const cudaError_t e = encode_map(x.map, p.bf16, 3, const_cast<uint16_t*>(a.q), dims, strides, box, false);
    if (e != cudaSuccess) return e;
  }
  // Token tiles of an item: one where each finds a CTA of its own, two where there are not many to a CTA, then more, so
  // that an item's cost is spread (the tables' width is what the host knows of the lengths).
  const long long tiles = static_cast<long long>(a.bt.B) * p.Hkv * ((static_cast<long long>(a.bt.max_blocks) * p.ps + BT - 1) / BT);
  const int gb = tiles <= ctas ? 1 : tiles < 64ll * ctas ? 2 : tiles < 128ll * ctas ? 4 : 8;
  const cudaError_t e = each_weigh([&](auto kernel, bool bf, int d, int smem) {
    if (bf != (p.bf16 != 0) || d != p.d) return cudaSuccess;
    return launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem + sizeof(Shared), s, p, a, gb, m.k_many, mq);
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
