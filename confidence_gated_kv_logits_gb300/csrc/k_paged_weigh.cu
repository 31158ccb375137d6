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
// product of N = 16, and there is nothing to join.  An item is up to 256 tokens
// (two tiles) of one KV head of one sequence; its K stays in shared memory while the
// rows' tiles of up to 128 (whole new tokens, as the heads of a group lie side by
// side) go by.  Items are laid end to end by their cost and cut into equal shares.
//
// Roles of a CTA's twelve warps: two warpgroups take the exponentials of one of the
// item's token tiles each, warp 8 issues the products, warp 9 moves K, warp 10 the
// query rows (both by TMA), warp 11 plans.  Two accumulators per token tile let the
// products of one tile of rows run beside the exponentials of another.
#include <algorithm>
#include <cstddef>

#include "paged_attend.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 384;
constexpr int BT = 128;                   // tokens of a tile (kManyBlock: the boxes are attend's)
constexpr int BR = 128;                   // most query rows of a tile
constexpr float kL2E = 1.4426950408889634f;
constexpr int kFixed = 2;                 // an item's fixed cost in tiles of rows: its K from memory
constexpr int kPlan = 8;                  // items in the planned ring
constexpr int kReaders = 11;              // warps that read it

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
  int j0;                                 // first token
  int tile0, tiles;                       // tiles of rows that see it
};

struct __align__(16) Shared {             // behind the stages
  unsigned long long bars[2 * 6 + 2 * 5 + 4 + 4 + 2 * kPlan + 1];
  Item plan[kPlan];
  __align__(16) float lse[2][2][BR];      // [token tile][tile parity]: lse log2 e, +inf for rows that add nothing
  Sched sched;
  long long scan[kThreads / 32];
  uint32_t tmem;
  int abort;
};
static_assert(offsetof(Shared, lse) % 16 == 0, "lse is read in 16-byte words");

// The items of a sequence's heads.
struct Items : Walk<BR, BT, 0> {
  const int cap, tb, gb;                  // places of the mass; new tokens of a tile of rows; token tiles of an item
  int tiles, items;                       // of the sequence
  __device__ __forceinline__ Items(const Pool& p_, const WeighArgs& a, int tb_, int gb_)
      : Walk(p_, a.bt, a.rows), cap(a.cap), tb(tb_), gb(gb_) {}
  __device__ __forceinline__ void shape() {
    tiles = (T + tb - 1) / tb;
    items = (len + BT * gb - 1) / (BT * gb);
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
  __device__ __forceinline__ int full_items() const {       // those that every row sees
    return bt.mask || items <= ctx / (BT * gb) + 1 ? items : ctx / (BT * gb) + 1;
  }
  __device__ __forceinline__ int cost(int i) const { return kFixed + tiles - first_tile(i); }
  __device__ __forceinline__ long long head_work() const {
    const int n = full_items();
    long long w = static_cast<long long>(n) * (kFixed + tiles);
    for (int i = n; i < items; ++i) w += cost(i);
    return w;
  }
};

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
k_weigh(const Pool p, const WeighArgs a, const int gb, const __grid_constant__ CUtensorMap mk, const __grid_constant__ QueryMaps mq) {
  using W = Weigh<D>;
  constexpr int SK = W::SK, SQ = W::SQ;
  extern __shared__ __align__(1024) unsigned char s_raw[];
  Shared& s = *reinterpret_cast<Shared*>(s_raw + W::SMEM);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t k_ring = smem_addr(s_raw), q_ring = k_ring + SK * W::TILE, bars = smem_addr(s.bars);
  const uint32_t b_kf = bars, b_ke = b_kf + 8 * SK, b_qf = b_ke + 8 * SK, b_qe = b_qf + 8 * SQ, b_s = b_qe + 8 * SQ,
                 b_free = b_s + 32, b_plan = b_free + 32, b_read = b_plan + 8 * kPlan, b_end = b_read + 8 * kPlan;
  if (tid == 0) {
    for (int i = 0; i < 2 * (SK + SQ); ++i) bar_init(b_kf + 8 * i, 1);
    for (int i = 0; i < 4; ++i) {
      bar_init(b_s + 8 * i, 1);
      bar_init(b_free + 8 * i, 128);
    }
    for (int i = 0; i < kPlan; ++i) {
      bar_init(b_plan + 8 * i, 1);
      bar_init(b_read + 8 * i, kReaders);
    }
    bar_init(b_end, 1);
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
    Items w(p, a, tb, gb);
    sched_init<kThreads>(w, &s.sched, s.scan, 1);
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  unsigned plan = 0;
  auto wait_item = [&](unsigned ahead) {  // the planned item that many further is there (behind the last one there is none)
    return bar_wait_warp(b_plan + 8 * ((plan + ahead) % kPlan), ((plan + ahead) / kPlan) & 1, &s.abort);
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
    Items w(p, a, tb, gb);
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
      const int full = kFixed + w.tiles, n = w.full_items();
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
      if (plan >= kPlan && !bar_wait_warp(b_read + 8 * (plan % kPlan), (plan / kPlan - 1) & 1, &s.abort)) break;
      if (lane == 0) {
        s.plan[plan % kPlan] = more ? Item{1, w.b, w.h, w.T, w.ctx, w.len, w.row0, i * BT * gb, w.first_tile(i), w.tiles} : Item{};
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
    // lane i asks for box i of the item: both token tiles' boxes, their channel halves side by side
    constexpr int HV = D / 64;
    const int x = lane / (16 / 2 * HV), i = lane % (16 / 2 * HV) / HV, half = lane % HV;
    auto page_of = [&](const Item& w) {   // the lane's page
      const int j = w.j0 + x * BT + i * rows_per;
      return w.more && x < gb && i < boxes && j < w.len ? a.bt.table[static_cast<size_t>(w.b) * a.bt.max_blocks + (j >> p.ps_shift)] : 0;
    };
    ok = wait_item(0);
    int page = ok ? page_of(item(0)) : 0;
    while (ok && item(0).more) {
      const Item& w = item(0);
      ok = wait_item(1);                  // the next item's pages are asked for before this one's boxes
      if (!ok) break;
      const int page1 = page_of(item(1));
      const bool none = static_cast<unsigned>(page) >= static_cast<unsigned>(p.NP);
      for (int y = 0; y < gb && w.j0 + y * BT < w.len; ++y, ++slot) {
        const unsigned st = slot % SK;
        if (slot >= SK && !bar_wait_warp(b_ke + 8 * st, (slot / SK - 1) & 1, &s.abort)) {
          ok = false;
          break;
        }
        const int j0 = w.j0 + y * BT, live = (w.len - j0 + rows_per - 1) / rows_per, n = live < boxes ? live : boxes;
        if (lane == 0) bar_expect(b_kf + 8 * st, static_cast<unsigned>(n * rows_per * D * 2));
        __syncwarp();
        if (x == y && i < n) {
          if (none) flag = CONFKV_FLAG_BAD_PAGE;
          const int j = j0 + i * rows_per;
          const int row = none ? kNoRows : (((a.layer * p.NP + page) * p.Hkv + w.h) << p.ps_shift) + (j & (p.ps - 1));
          tma_box(k_ring + st * W::TILE + half * W::HALF + i * rows_per * 128, &mk, 64 * half, row, b_kf + 8 * st, pol);
        }
      }
      page = page1;
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
        if (slot >= SQ && !bar_wait_warp(b_qe + 8 * st, (slot / SQ - 1) & 1, &s.abort)) {
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
  } else if (warp == 8) {
    // ---- products: S[token tile x][parity] = K Q^T (the warp stays together; one elected thread issues) ----
    constexpr uint32_t hi = umma_hi(1024);
    const uint32_t k_lo = uniform(umma_lo(k_ring, 16)), q_lo = uniform(umma_lo(q_ring, 16));
    unsigned ks = 0, qs = 0, ns = 0;      // stages taken; tiles of rows so far
    unsigned used[2][2] = {};             // products into an accumulator so far
    bool ok = true;
    while (ok && next_item()) {
      const Item& w = item(0);
      const int blocks = min(gb, (w.len - w.j0 + BT - 1) / BT);
      for (int x = 0; ok && x < blocks; ++x) ok = bar_wait_warp(b_kf + 8 * ((ks + x) % SK), ((ks + x) / SK) & 1, &s.abort);
      for (int t = w.tile0; ok && t < w.tiles; ++t, ++qs, ++ns) {
        const unsigned st = qs % SQ;
        ok = bar_wait_warp(b_qf + 8 * st, (qs / SQ) & 1, &s.abort);
        const uint32_t idesc = umma_idesc(BF, 128, (rows_of(w, t) + 15) & ~15, false);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || x >= blocks) break;
          const uint32_t acc = 2 * x + (ns & 1);
          const unsigned before = ns & 1 ? used[x][1] : used[x][0];
          if (before) ok = bar_wait_warp(b_free + 8 * acc, (before - 1) & 1, &s.abort);
          if (!ok) break;
          if (ns & 1) ++used[x][1];
          else ++used[x][0];
          tc_fence_after();
          const uint32_t kt = uniform(k_lo + ((ks + x) % SK) * (W::TILE / 16)), qt = uniform(q_lo + st * (W::TILE / 16));
          const uint32_t d = uniform(tmem + acc * BR);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t o = ((c >> 2) * W::HALF + (c & 3) * 32) / 16;
            umma_ss(d, kt + o, hi, qt + o, hi, idesc, c > 0);
          }
          umma_commit(b_s + 8 * acc);
        }
        if (ok) umma_commit(b_qe + 8 * st);
      }
      if (!ok) break;
      for (int x = 0; x < blocks; ++x) umma_commit(b_ke + 8 * ((ks + x) % SK));
      ks += blocks;
      item_done();
    }
    // products in flight end before the CTA does
    if (!ok) {
      umma_commit(b_end);
      bar_drain(b_end, 0);
    }
    __syncwarp();
  } else {
    // ---- weights ----
    const int x = warp >> 2, r = tid & 127;               // token tile of the item; token of the tile, and column whose lse it brings
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c = a.scale * kL2E;
    const int rt = r / p.g, rh = r - rt * p.g;
    unsigned ns = 0, used0 = 0, used1 = 0;                // tiles of rows so far; those of its two accumulators
    // an item's mass, and the lse of a column of its tile t
    auto mass_of = [&](const Item& w) {
      const int j = w.j0 + x * BT + r;
      return w.more && x < gb && j < w.len && j < w.ctx ? a.mass[(static_cast<size_t>(w.b) * p.Hkv + w.h) * a.cap + j] : 0.0f;
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
      auto args = [&](int g) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float4 l = lq[2 * g + y];
          z[g & 1][4 * y] = fma_o(__uint_as_float(sv[8 * g + 4 * y]), c, -l.x);
          z[g & 1][4 * y + 1] = fma_o(__uint_as_float(sv[8 * g + 4 * y + 1]), c, -l.y);
          z[g & 1][4 * y + 2] = fma_o(__uint_as_float(sv[8 * g + 4 * y + 2]), c, -l.z);
          z[g & 1][4 * y + 3] = fma_o(__uint_as_float(sv[8 * g + 4 * y + 3]), c, -l.w);
        }
      };
      args(0);
#pragma unroll
      for (int g = 0; g <= N / 8; ++g) {
        if (g + 1 < N / 8) args(g + 1);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if (g < N / 8) {
            const float e0 = ex2_o(z[g & 1][2 * y]), e1 = ex2_o(z[g & 1][2 * y + 1]);
            e[g & 1][y] = pair(keep(8 * g + 2 * y, e0), keep(8 * g + 2 * y + 1, e1));
          }
          if (g > 0) sum[y] = add2_o(sum[y], e[(g - 1) & 1][y]);
        }
      }
    };
    // One item, whose mass and first lse were asked for two items ago; false: there is none, or a wait gave up.
    bool ok = true;
    auto step = [&](float& before, float& next) {
      if (group_any(x, !(ok && item(0).more))) return false;
      const Item& w = item(0);
      const int j = w.j0 + x * BT + r;
      const bool here = w.j0 + x * BT < w.len && x < gb;  // the item has this token tile
      sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
      for (int t = w.tile0; t < w.tiles; ++t, ++ns) {
        if (!here) continue;                              // (it counts the tile all the same)
        const unsigned par = ns & 1, acc = 2 * x + par;
        float* lse = s.lse[x][par];
        lse[r] = next == -INFINITY ? INFINITY : next * kL2E;
        if (t + 1 < w.tiles) next = lse_of(w, t + 1);
        const bool got = bar_wait_warp(b_s + 8 * acc, (par ? used1 : used0) & 1, &s.abort);
        if (par) ++used1;
        else ++used0;
        if (group_any(x, !got)) return false;
        tc_fence_after();
        const int n = rows_of(w, t);
        // columns that see this token: causal ones from its own row on
        const int past = j - w.ctx - t * tb;              // new tokens of the tile that come before it
        const bool masked = a.bt.mask && w.j0 + x * BT + BT > w.ctx;
        const int from = a.bt.mask || past <= 0 ? 0 : past * p.g;
        const uint32_t ts = tmem + lanes + acc * BR;
        if (masked) {
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
        bar_arrive(b_free + 8 * acc);
      }
      if (here && j < w.len) {
        const size_t at = (static_cast<size_t>(w.b) * p.Hkv + w.h) * a.cap + j;
        const float2 y = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
        a.mass_out[at] = a.decay * before + a.gain * (y.x + y.y);
        if (j >= w.ctx && a.pos) a.pos[at] = a.positions ? a.positions[w.row0 + j - w.ctx] : j;
      }
      // the one after the next (the next is there, it may be the end)
      ok = wait_item(1);
      if (ok && item(1).more) {
        ok = wait_item(2);
        if (ok) {
          before = mass_of(item(2));
          next = lse_of(item(2), item(2).tile0);
        }
      }
      item_done();
      return true;
    };
    float before0 = 0.0f, before1 = 0.0f, next0 = 0.0f, next1 = 0.0f;
    ok = wait_item(0);
    if (ok && item(0).more) {
      before0 = mass_of(item(0));
      next0 = lse_of(item(0), item(0).tile0);
      ok = wait_item(1);
      if (ok) {
        before1 = mass_of(item(1));
        next1 = lse_of(item(1), item(1).tile0);
      }
    }
    while (step(before0, next0) && step(before1, next1)) {
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
  // Two token tiles to an item where there are more tiles than CTAs (the tables' width is what the host knows).
  const long long tiles = (static_cast<long long>(a.bt.max_blocks) * p.ps + BT - 1) / BT;
  const int gb = static_cast<long long>(a.bt.B) * p.Hkv * tiles <= ctas ? 1 : 2;
  const cudaError_t e = each_weigh([&](auto kernel, bool bf, int d, int smem) {
    if (bf != (p.bf16 != 0) || d != p.d) return cudaSuccess;
    return launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem + sizeof(Shared), s, p, a, gb, m.k_many, mq);
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
