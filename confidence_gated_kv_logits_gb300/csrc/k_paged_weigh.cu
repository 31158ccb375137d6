// Accumulated attention weight of each cached token and KV head:
//
//   mass_out_t = decay mass_t + gain sum_r exp(scale q_r k_t - lse_r)
//
// over the rows r (new tokens x the group's query heads) that see token t, with
// the rows' lse as attend gave it: the weights are final at once, nothing is
// rescaled.  Each token's sum is one thread's where one tile holds all rows; of several tiles
// two threads take every second one each and join once: in one order either way.
//
// Tokens are the products' M (tiles of 128, full whatever the rows are) and query
// rows their N (16 to 112), S = K Q^T in tensor memory: a thread owns a token, so
// a tile's sum over rows needs no other thread, a single token's few rows cost a
// product of N = 16, and there is little to join.  An item is some token tiles of
// one KV head of one sequence: two where the rows need several tiles of up to 112
// (whole new tokens, as the heads of a group lie side by side), which go by while K
// stays in shared memory, up to eight where one tile holds all rows.  Items are laid
// end to end by their cost and cut into equal shares.
//
// Roles of a CTA's 20 warps: a pair of warpgroups takes the exponentials of the
// even token tiles, a pair those of the odd ones; warps 16 and 17 issue a pair's
// products (one warp alone takes as long to issue both's as the exponentials do), warp
// 18 moves K and the query rows by TMA, warp 19 plans.  Each warpgroup has an
// accumulator of its own and takes every second product of its pair; where these are
// one token tile's, the pair's two sums are joined at the item's end.
//
// 32 sequences x 1 token over up to 16384, 64/8 heads of 64, bf16 (389 MB): 74 us, 5.3 TB/s,
// 78% of the copy rate, 850 cycles of fixed steps per token tile in the moving and issuing warps; 64 rows of 4 sequences over 12000, 40/8 heads of 128 (31.5 GFLOP):
// 46 us, 690 TFLOP/s, bound by the exponentials' instructions (a column's share of a
// warp's issue slots) and the steps between products; one token over 2048, 12/12 heads
// of 64: 6.8 us, of which the chain page -> K -> product takes 2 and planning the same (7.1 with the scans that
// several sequences need).  Two warpgroups instead of four: 71, 56 and 6.6 us; one issuing warp 73 (32 sequences); items of one token tile, and columns in unrolled code that did
// not fit the instruction cache, 147 to 176.
#include <algorithm>
#include <cstddef>

#include "paged_attend.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 4 * 128 + 4 * 32;      // (a 21st warp would leave each thread 80 registers instead of 96)
constexpr int BT = 128;                   // tokens of a tile (kManyBlock: the boxes are attend's)
constexpr int BR = 112;                   // most query rows of a tile (three tiles of 128 beside four of K leave no room)
constexpr float kL2E = 1.4426950408889634f;
constexpr int kFixed = 2;                 // an item's fixed cost in tiles of rows: its K from memory (1 and 4: the same times within 1%)
constexpr int kPlan = 8;                  // items in the planned ring
constexpr int kReaders = 19;              // warps that read it

static_assert(BT == kManyBlock, "boxes of the pools");

template <int D>
struct Weigh {
  static constexpr int KH = BT * 128, QH = BR * 128;        // bytes of 64 channels of a K or Q tile
  static constexpr int KT = KH * D / 64, QT = QH * D / 64;
  static constexpr int SK = D == 128 ? 4 : 6, SQ = D == 128 ? 3 : 5;      // stages (10 of K at d = 64 change nothing)
  static constexpr int SMEM = SK * KT + SQ * QT;
};

struct Item {
  int more;                               // 0: the CTA's share ends here
  int b, h, T, ctx, len, row0;
  int j0, nb;                             // first token, token tiles
  int tile0, tiles;                       // tiles of rows that see it
};

struct __align__(16) Shared {             // behind the stages
  unsigned long long bars[2 * 6 + 2 * 5 + 4 + 4 + 4 + 2 * kPlan + 2];
  Item plan[kPlan];
  __align__(16) float lse[4][2][BR];      // [warpgroup][parity]: -lse log2 e, -inf for rows that add nothing
  float part[2][BT];                      // [pair]: a token tile's sum by the warpgroup that does not end it
  Sched sched;
  long long scan[kThreads / 32];
  uint32_t tmem;
  int abort;
};
static_assert(offsetof(Shared, lse) % 16 == 0 && BR % 16 == 0, "lse is read in 16-byte words");

// The items of a sequence's heads.
struct Items : Walk<BR, BT, 0> {
  const int cap, tb, sh1, sh2;            // places of the mass; new tokens of a tile of rows; log2 of the token tiles of an
                                          // item whose rows are one tile, several
  int tiles, sh, items, all;              // of the sequence: tiles of rows, log2 of an item's token tiles, items, token tiles
  __device__ __forceinline__ Items(const Pool& p_, const WeighArgs& a, int tb_, int sh1_)
      : Walk(p_, a.bt, a.rows), cap(a.cap), tb(tb_), sh1(sh1_), sh2(sh1_ < 1 ? 0 : 1) {}
  __device__ __forceinline__ void shape() {
    tiles = T > tb ? (T + tb - 1) / tb : T > 0;
    sh = tiles > 1 ? sh2 : sh1;
    all = (len + BT - 1) / BT;
    items = (all + (1 << sh) - 1) >> sh;
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
    const int x = i * (BT << sh) - ctx;
    return bt.mask || x < tb ? 0 : x / tb;
  }
  __device__ __forceinline__ int count(int i) const { return min(all - (i << sh), 1 << sh); }       // its token tiles
  __device__ __forceinline__ int full_items() const {       // those of all tiles that every row sees
    const int whole = all >> sh, seen = (ctx / BT >> sh) + 1;
    return bt.mask || whole < seen ? whole : seen;
  }
  __device__ __forceinline__ int cost(int i) const { return count(i) * (kFixed + tiles - first_tile(i)); }
  __device__ __forceinline__ long long head_work() const {
    const int n = full_items();
    long long w = static_cast<long long>(n) * ((kFixed + tiles) << sh);
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

// x = *at where `use`, else `other`: a predicated load, so that no choice behind it can wait for the value.  (A word of
// mass is read by the one thread that writes it, so L1 may hold stale neighbours.)
__device__ __forceinline__ void load_if(float& x, const float* at, bool use, float other) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p ld.global.f32 %0, [%1];\n @!p mov.f32 %0, %3;\n}\n"
      : "+f"(x)
      : "l"(at), "r"(static_cast<unsigned>(use)), "f"(other)
      : "memory");
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
k_weigh(const Pool p, const WeighArgs a, const int sh1, const __grid_constant__ CUtensorMap mk, const __grid_constant__ QueryMaps mq) {
  using W = Weigh<D>;
  constexpr int SK = W::SK, SQ = W::SQ;
  extern __shared__ __align__(1024) unsigned char s_raw[];
  Shared& s = *reinterpret_cast<Shared*>(s_raw + W::SMEM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t k_ring = smem_addr(s_raw), q_ring = k_ring + SK * W::KT, bars = smem_addr(s.bars);
  // K and Q stages full and empty; per warpgroup: S there, S read; per pair: its part there, read; the plan; the end
  const uint32_t b_kf = bars, b_ke = b_kf + 8 * SK, b_qf = b_ke + 8 * SK, b_qe = b_qf + 8 * SQ, b_s = b_qe + 8 * SQ,
                 b_free = b_s + 32, b_part = b_free + 32, b_took = b_part + 16, b_plan = b_took + 16, b_read = b_plan + 8 * kPlan,
                 b_end = b_read + 8 * kPlan;
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
    for (int i = 0; i < 2; ++i) {
      bar_init(b_part + 8 * i, 128);
      bar_init(b_took + 8 * i, 128);
      bar_init(b_end + 8 * i, 1);
    }
    for (int i = 0; i < kPlan; ++i) {
      bar_init(b_plan + 8 * i, 1);
      bar_init(b_read + 8 * i, kReaders);
    }
    s.abort = 0;
    fence_bar_init();
    fence_async();
  }
  if (warp == 18) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_addr(&s.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  pdl_wait();
  pdl_trigger();
  fence_async_global();
  tc_fence_before();
  const int tb = mq.n_all;
  if (a.bt.B > 32) {
    Items w(p, a, tb, sh1);
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

  if (warp == 19) {
    // ---- the plan ----
    Items w(p, a, tb, sh1);
    Sched sh;
    if (a.bt.B == 1) {                    // without the scans over sequences (one token over 2048: 7.1 us with them, 6.8)
      int bad = 0;
      w.sequence(0, bad);
      if (bad && blockIdx.x == 0 && lane == 0) atomicOr(p.err, bad);
      sh.b = 0;
      sh.T = w.T;
      sh.ctx = w.ctx;
      sh.len = w.len;
      sh.row0 = w.row0;
      sh.seq0 = 0;
      sh.head = w.T > 0 ? w.head_work() : 0;
      sched_share<Items>(&sh, sh.head * p.Hkv, blockIdx.x, gridDim.x, 1);
    } else if (a.bt.B <= 32) {
      sh = sched_warp(w, 1, 0, blockIdx.x, gridDim.x);
    } else {
      sh = s.sched;
    }
    long long at = 0;                     // the cost at which the next item starts
    int i = 0, flag = 0;
    const bool any = sh.cur < sh.end;
    if (any) {
      w.b = sh.b;
      w.T = sh.T;
      w.ctx = sh.ctx;
      w.len = sh.len;
      w.row0 = sh.row0;
      w.shape();
      // the share's first item: the first that starts in it
      w.h = static_cast<int>(quotient(sh.cur - sh.seq0, sh.head));
      at = sh.seq0 + w.h * sh.head;
      const int full = (kFixed + w.tiles) << w.sh, n = w.full_items();
      const long long j = quotient(sh.cur - at + full - 1, full);
      i = j < n ? static_cast<int>(j) : n;
      at += static_cast<long long>(i) * full;
      while (i < w.items && at < sh.cur) at += w.cost(i++);
    }
    for (bool more = true; more; ++plan) {
      while (any && at < sh.end && i >= w.items) {
        i = 0;
        if (++w.h == p.Hkv) {
          w.h = 0;
          do w.sequence(w.b + 1, flag); while (w.T <= 0);
        }
      }
      more = any && at < sh.end;
      if (plan >= kPlan && !wait_bar(b_read + 8 * (plan % kPlan), (plan / kPlan - 1) & 1, &s.abort)) break;
      const int t0 = more ? w.first_tile(i) : 0, nb = more ? w.count(i) : 0;
      if (lane == 0) {
        s.plan[plan % kPlan] = more ? Item{1, w.b, w.h, w.T, w.ctx, w.len, w.row0, i * (BT << w.sh), nb, t0, w.tiles} : Item{};
        bar_arrive(b_plan + 8 * (plan % kPlan));
      }
      if (more) at += nb * (kFixed + w.tiles - t0);
      ++i;
    }
  } else if (warp == 18) {
    // ---- K and query rows ----
    const uint64_t pol = stream_policy();
    const int row_shift = p.ps < BT ? p.ps_shift : 7, rows_per = 1 << row_shift, boxes = BT >> row_shift;
    unsigned slot = 0, qslot = 0;
    int flag = 0;
    // two token tiles at a time: a lane has one box, both tiles' boxes and their channel halves side by side
    constexpr int HV = D / 64;
    const int x = lane / (8 * HV), i = lane % (8 * HV) / HV, half = lane % HV;
    const uint32_t to = k_ring + half * W::KH + i * rows_per * 128;
    auto page_of = [&](const Item& w, int y0) {
      const int j = w.j0 + (y0 + x) * BT + i * rows_per;
      return w.more && x < 2 && y0 + x < w.nb && i < boxes && j < w.len
                 ? a.bt.table[static_cast<size_t>(w.b) * a.bt.max_blocks + (j >> p.ps_shift)] : 0;
    };
    auto rows = [&](const Item& w, int t) {
      const unsigned st = qslot % SQ;
      if (qslot >= SQ && !wait_bar(b_qe + 8 * st, (qslot / SQ - 1) & 1, &s.abort)) return false;
      const int left = w.T - t * tb;
      const int n = left == 1 ? 1 : left <= mq.n_some ? mq.n_some : mq.n_all;
      const CUtensorMap* map = left == 1 ? &mq.one : left <= mq.n_some ? &mq.some : &mq.all;
      if (lane == 0) bar_expect(b_qf + 8 * st, static_cast<unsigned>(n * p.g * D * 2));
      __syncwarp();
      if (lane < D / 64)
        tma_rows(q_ring + st * W::QT + lane * W::QH, map, 64 * lane, w.h * p.g, w.row0 + t * tb, b_qf + 8 * st);
      ++qslot;
      return true;
    };
    bool ok = wait_item(0);
    int page = ok ? page_of(item(0), 0) : 0;
    while (ok && item(0).more) {
      const Item& w = item(0);
      // the first tile of rows before K, whose stages can be fewer than the item's token tiles
      ok = rows(w, w.tile0);
      for (int y0 = 0; ok && y0 < w.nb; y0 += 2) {
        const bool none = static_cast<unsigned>(page) >= static_cast<unsigned>(p.NP);
        const int j = w.j0 + (y0 + x) * BT + i * rows_per;
        const int row = none ? kNoRows : (((a.layer * p.NP + page) * p.Hkv + w.h) << p.ps_shift) + (j & (p.ps - 1));
        for (int y = y0; y < y0 + 2 && y < w.nb; ++y, ++slot) {
          const unsigned st = slot % SK;
          if (slot >= SK && !wait_bar(b_ke + 8 * st, (slot / SK - 1) & 1, &s.abort)) {
            ok = false;
            break;
          }
          const int live = (w.len - w.j0 - y * BT + rows_per - 1) >> row_shift, n = live < boxes ? live : boxes;
          if (lane == 0) bar_expect(b_kf + 8 * st, static_cast<unsigned>(n * rows_per * D * 2));
          __syncwarp();
          if (x == y - y0 && i < n) {
            if (none) flag = CONFKV_FLAG_BAD_PAGE;
            tma_box(to + st * W::KT, &mk, 64 * half, row, b_kf + 8 * st, pol);
          }
        }
        // the next boxes' pages
        if (ok && y0 + 2 < w.nb) {
          page = page_of(w, y0 + 2);
        } else if (ok) {
          ok = wait_item(1);
          if (ok) page = page_of(item(1), 0);
        }
      }
      for (int t = w.tile0 + 1; ok && t < w.tiles; ++t) ok = rows(w, t);
      item_done();
    }
    if (flag) atomicOr(p.err, flag);
    if (!ok) {                            // no copy may land after the CTA has gone
      for (unsigned k = slot > SK ? slot - SK : 0; k < slot; ++k) bar_drain(b_kf + 8 * (k % SK), (k / SK) & 1);
      for (unsigned k = qslot > SQ ? qslot - SQ : 0; k < qslot; ++k) bar_drain(b_qf + 8 * (k % SQ), (k / SQ) & 1);
    }
  } else if (warp >= 16) {
    // ---- a pair's products, S = K Q^T (the warp stays together; one elected thread issues) ----
    const int g = warp - 16;
    constexpr uint32_t hi = umma_hi(1024);
    const uint32_t k_lo = uniform(umma_lo(k_ring, 16)), q_lo = uniform(umma_lo(q_ring, 16));
    unsigned ks = 0, qs = 0, used = 0;    // stages passed; products so far
    bool ok = true;
    while (ok && next_item()) {
      const Item& w = item(0);
      const int nb = w.nb, tiles = w.tiles, tile0 = w.tile0, T = w.T;
      for (int t = tile0; ok && t < tiles; ++t, ++qs) {
        const unsigned st = qs % SQ;
        ok = wait_bar(b_qf + 8 * st, (qs / SQ) & 1, &s.abort);
        const uint32_t idesc = umma_idesc(BF, 128, (min(tb, T - t * tb) * p.g + 15) & ~15, false), qt = uniform(q_lo + st * (W::QT / 16));
        for (int x = 0; ok && x < nb; ++x) {
          const unsigned k = ks + x;
          if (t == tile0) ok = wait_bar(b_kf + 8 * (k % SK), (k / SK) & 1, &s.abort);
          if ((x & 1) != g) {
            if (ok && t == tile0) bar_arrive_warp(b_ke + 8 * (k % SK));
            continue;
          }
          const unsigned n = used++;
          const uint32_t acc = 2 * g + (n & 1);
          if (ok && n >= 2) ok = wait_bar(b_free + 8 * acc, (n / 2 - 1) & 1, &s.abort);
          if (!ok) break;
          tc_fence_after();
          const uint32_t kt = uniform(k_lo + (k % SK) * (W::KT / 16)), d = uniform(tmem + acc * 128);
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            umma_ss(d, kt + ((c >> 2) * W::KH + (c & 3) * 32) / 16, hi, qt + ((c >> 2) * W::QH + (c & 3) * 32) / 16, hi, idesc, c > 0);
          umma_commit(b_s + 8 * acc);
          if (t + 1 == tiles) umma_commit(b_ke + 8 * (k % SK));
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
    // warpgroup; its pair and place there; token of a tile, and column whose lse it brings
    const int wg = warp >> 2, g = wg >> 1, me = wg & 1, r = tid & 127;
    const uint32_t ts = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + wg * 128;
    const float c = a.scale * kL2E;
    const int rt = r / p.g, rh = r - rt * p.g;
    const bool brings = rt < tb;
    const size_t lse_at = static_cast<size_t>(rt) * p.Hq + rh;
    auto lse_of = [&](float& y, const Item& w, int t, bool use) {
      load_if(y, a.lse + (static_cast<size_t>(w.row0 + t * tb) * p.Hq + w.h * p.g + lse_at),
              use && brings && t < w.tiles && t * tb + rt < w.T, -INFINITY);
    };
    // the mass of tile x's token
    auto mass_of = [&](float& y, const Item& w, int x, bool use) {
      const int j = w.j0 + x * BT + r;
      load_if(y, a.mass + ((static_cast<size_t>(w.b) * p.Hkv + w.h) * a.cap + j), use && x < w.nb && j < w.len && j < w.ctx, 0.0f);
    };
    // of the products from the pair's n-th on: how many are the other's before this warpgroup's first
    auto skip = [&](unsigned n) { return static_cast<int>((n ^ me) & 1u); };
    // N columns' weights into four sums, in the columns' order; the steps of neighbouring groups of eight are
    // interleaved (written in order: the schedule is otherwise one chain after another)
    uint64_t sum[4];
    const uint64_t cc = pair(c, c);
    auto weights = [&](auto const& sv, const float* lse, auto keep) {
      constexpr int N = sizeof(sv) / 4;
      const ulonglong2* lq = reinterpret_cast<const ulonglong2*>(lse);
      uint64_t z[2][4], e[2][4];
      auto args = [&](int k) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const ulonglong2 l = lq[2 * k + y];
          z[k & 1][2 * y] = fma2_o(pair(__uint_as_float(sv[8 * k + 4 * y]), __uint_as_float(sv[8 * k + 4 * y + 1])), cc, l.x);
          z[k & 1][2 * y + 1] = fma2_o(pair(__uint_as_float(sv[8 * k + 4 * y + 2]), __uint_as_float(sv[8 * k + 4 * y + 3])), cc, l.y);
        }
      };
      args(0);
#pragma unroll
      for (int k = 0; k <= N / 8; ++k) {
        if (k + 1 < N / 8) args(k + 1);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if (k < N / 8) {
            const float2 x = unpair(z[k & 1][y]);
            const float e0 = ex2_o(x.x), e1 = ex2_o(x.y);
            e[k & 1][y] = pair(keep(8 * k + 2 * y, e0), keep(8 * k + 2 * y + 1, e1));
          }
          if (k > 0) sum[y] = add2_o(sum[y], e[(k - 1) & 1][y]);
        }
      }
    };
    // products of the pair so far, this warpgroup's, its tiles of rows, the pair's joins
    unsigned made = 0, used = 0, steps = 0, joins = 0;
    bool ok = wait_item(0);
    float before = 0.0f, next = -INFINITY;
    if (ok && item(0).more) {
      const Item& w = item(0);
      lse_of(next, w, w.tile0 + (w.tiles > 1 ? skip(0) : 0), true);
      mass_of(before, w, g + 2 * skip(0), true);
    }
    while (!group_any(wg, !(ok && item(0).more))) {
      const Item& w = item(0);
      const int nb = w.nb, tiles = w.tiles, j0 = w.j0, T = w.T, ctx = w.ctx, len = w.len, row0 = w.row0;
      const bool several = tiles > 1;
      const size_t at0 = (static_cast<size_t>(w.b) * p.Hkv + w.h) * a.cap;
      const int products = nb <= g ? 0 : several ? tiles - w.tile0 : (nb - g + 1) >> 1;
      const unsigned first = made;
      made += products;
      // several tiles of rows: the warpgroup that takes the last one ends the token tile
      const bool ends = !several || skip(first + products - 1) == 0;
      if (several) mass_of(before, w, g, ends && products);
      ok = wait_item(1);
      bool dead = !ok;
      sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
      auto next_lse = [&] {               // of the next item
        const Item& v = item(1);
        lse_of(next, v, v.tile0 + (v.tiles > 1 ? skip(made) : 0), ok && v.more);
      };
      auto next_mass = [&](float& y) {
        const Item& v = item(1);
        mass_of(y, v, g + 2 * skip(made), ok && v.more && v.tiles <= 1);
      };
      // one product of this warpgroup's: token tile x, rows' tile t
      auto product = [&](int x, int t, const float* lse) {
        const int j = j0 + x * BT + r, n = min(tb, T - t * tb) * p.g;
        if (!wait_bar(b_s + 8 * wg, used & 1, &s.abort)) return false;
        ++used;
        tc_fence_after();
        const bool fresh = j0 + x * BT + BT > ctx;        // the tile holds new tokens
        if (fresh && a.bt.mask) {
          // by the batch's mask, column by column
          int tok = t * tb, left = p.g;                   // the column's new token, its columns that are left
#pragma unroll 1
          for (int q = 0; q < n; q += 8) {
            uint32_t sv[8];
            __syncwarp();
            tmem_ld8(sv, ts + q);
            tmem_wait_ld(sv);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const bool seen = q + e < n && (seen_bits(a.bt, static_cast<size_t>(row0 + tok), tok, ctx, len, j) & 1u);
              const float y = seen ? ex2f(fmaf(__uint_as_float(sv[e]), c, lse[q + e])) : 0.0f;
              sum[e >> 1] = add2(sum[e >> 1], e & 1 ? pair(0.0f, y) : pair(y, 0.0f));
              if (--left == 0) {
                left = p.g;
                if (tok + 1 < T) ++tok;
              }
            }
          }
        } else {
          // causal: the columns from the token's own row on
          const int from = fresh && j - ctx > t * tb ? (j - ctx - t * tb) * p.g : 0;
          int q = 0;
          if (!fresh || !__any_sync(0xffffffffu, from > 0)) {
#pragma unroll 1
            for (; q + 32 <= n; q += 32) {
              uint32_t sv[32];
              tmem_ld32(sv, ts + q);
              tmem_wait_ld(sv);
              weights(sv, lse + q, [](int, float y) { return y; });
            }
          }
          if (n <= 8) {
            uint32_t sv[8];
            tmem_ld8(sv, ts);
            tmem_wait_ld(sv);
            weights(sv, lse, [&](int col, float y) { return col >= from && col < n ? y : 0.0f; });
          } else {
#pragma unroll 1
            for (; q < n; q += 16) {
              uint32_t sv[16];
              tmem_ld16(sv, ts + q);
              tmem_wait_ld(sv);
              weights(sv, lse + q, [&](int col, float y) { return q + col >= from && q + col < n ? y : 0.0f; });
            }
          }
        }
        tc_fence_before();
        bar_arrive(b_free + 8 * wg);
        return true;
      };
      auto total = [&] {
        const float2 y = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
        sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
        return y.x + y.y;
      };
      auto store = [&](int x, float y) {
        const int j = j0 + x * BT + r;
        if (j >= len) return;
        a.mass_out[at0 + j] = a.decay * before + a.gain * y;
        if (j >= ctx && a.pos) a.pos[at0 + j] = a.positions ? a.positions[row0 + j - ctx] : j;
      };
      // rows' tiles: of several each second one, of one the tile itself, which serves all token tiles
      for (int t = w.tile0 + (several ? skip(first) : 0); t < tiles && products; t += 2, ++steps) {
        float* lse = s.lse[wg][steps & 1];
        if (r < BR) lse[r] = next == -INFINITY ? -INFINITY : next * -kL2E;
        if (several && t + 2 < tiles) lse_of(next, w, t + 2, true);
        else next_lse();
        if (group_any(wg, dead)) {
          dead = true;
          break;
        }
        if (several) {
          dead = dead || !product(g, t, lse);             // (the others learn of it at the next decision)
        } else {
#pragma unroll 1
          for (int x = g + 2 * skip(first); x < nb; x += 4) {
            float after = 0.0f;
            if (x + 4 < nb) mass_of(after, w, x + 4, true);
            else next_mass(after);
            if (!product(x, t, lse)) {
              dead = true;
              break;
            }
            store(x, total());
            before = after;
          }
        }
      }
      if (several && products && !dead) {
        if (products == 1) {
          if (ends) store(g, total());
        } else if (ends) {
          // the other warpgroup's sum
          if (wait_bar(b_part + 8 * g, joins & 1, &s.abort)) {
            const float other = s.part[g][r];
            bar_arrive(b_took + 8 * g);
            store(g, other + total());
          } else {
            dead = true;
          }
        } else if (joins == 0 || wait_bar(b_took + 8 * g, (joins - 1) & 1, &s.abort)) {
          s.part[g][r] = total();
          bar_arrive(b_part + 8 * g);
        } else {
          dead = true;
        }
      }
      if (several && products > 1) ++joins;
      // what the item did not ask for, having no product of this warpgroup's
      if (!products || (several && skip(first) >= products)) next_lse();
      if (several || nb <= g + 2 * skip(first)) next_mass(before);
      ok = ok && !dead;
      item_done();
    }
  }
  __syncthreads();
  if (s.abort && tid == 0) atomicOr(p.err, CONFKV_FLAG_TIMEOUT);
  if (warp == 18) {
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
static_assert(Weigh<128>::SMEM + sizeof(Shared) <= 232448 && Weigh<64>::SMEM + sizeof(Shared) <= 232448, "a CTA's shared memory");

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
  // Token tiles of an item: one where each finds a CTA of its own, then as many as leave a CTA several items, so that an
  // item's fixed cost is spread (the tables' width is what the host knows of the lengths).  us with one, two, four and
  // eight tiles an item, by the tiles to a CTA: 1.3 (1 x 2048 tokens, 12/12 heads of 64) 6.6, 6.5, 6.8, 8.1; 3.4 (16 x 500,
  // 40/8 of 128) 10.1, 8.0, 7.3, 7.3; 6.7 (4 x 4000) 14.6, 11.4, 10.3, 10.2; 13 (8 x 4000, 64/8 of 64) 23.4, 15.0, 13.3,
  // 12.1; 27 (32 x 2000) 41.4, 24.8, 19.1, 18.8; 210 (32 x up to 16384) 154, 85, 65, 57; with 80 rows, 20 (4 x 12000,
  // 40/8 of 128) 37.7, 25.3, 22.0, 22.5.
  const long long tiles = static_cast<long long>(a.bt.B) * p.Hkv * ((static_cast<long long>(a.bt.max_blocks) * p.ps + BT - 1) / BT);
  const int sh1 = tiles <= ctas ? 0 : tiles < 2ll * ctas ? 1 : tiles < 6ll * ctas ? 2 : 3;
  const cudaError_t e = each_weigh([&](auto kernel, bool bf, int d, int smem) {
    if (bf != (p.bf16 != 0) || d != p.d) return cudaSuccess;
    return launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem + sizeof(Shared), s, p, a, sh1, m.k_many, mq);
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
