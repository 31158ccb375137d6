// Attention of many new rows per sequence over a paged cache (prompt chunks,
// trees of drafted tokens): tiles of 128 query rows on the fifth-generation
// tensor cores.
//
//   S = Q K^T (fp32, tensor memory);  P = exp2(c S - c m), c = scale log2 e;
//   O = P V (fp32, tensor memory);    out = O / sum P
//
// Roles of a CTA's twelve warps: two warpgroups do the softmax of a stream of
// products each, warps 8 and 9 issue a stream's tcgen05.mma each (the whole warp
// stays together and one elected lane issues, so that descriptors stay in uniform
// registers: 544 us against 747 with a lane branched off, for the chunk below),
// warp 10 moves K and V blocks of 128 tokens from the pages by TMA through a
// ring of 32 KB (d = 128) or 16 KB stages, warp 11 plans the CTA's pieces and
// hands them to the others through shared memory.  There are two streams so that the
// tensor cores work on one while the other's exponentials are taken:
//   NQ = 2: a unit is 256 query rows, a stream takes 128 of them and all blocks;
//   NQ = 1: a unit is 128 query rows, a stream takes every second block, and
//           the two are joined at the unit's end (few rows, where the bytes
//           of the cache or the length of the dependent chain count).
// A stream goes on by sub-blocks of 64 tokens with two S buffers: behind PV of
// sub-block i comes QK of i + 2 into the same buffer, so a softmax finds its
// next S there already.  Products of one thread complete in order: S is
// overwritten only behind the PV that read the P in its place.  P is written
// over S in tensor memory (the first product operand may lie there) and V is
// read as it lies, rows of channels (MN-major), so neither is transposed.
//
// The running maximum is raised only when it grows by a factor of 2^8 or more
// (P <= 2^8 meanwhile: exact in fp32, and fp16 P keeps more small values), so
// O is rarely rescaled.  Row statistics are fp32; P is rounded once to the
// cache's type.  Masks and what masked places hold: as in k_paged_attend.cu,
// with V mended in shared memory before the product, and non-finite elements
// added behind it to the rows that see them.
//
// Measured: two prompts' chunks of 2048 rows over 6144 cached tokens, 40/8 heads
// of 128 channels, bf16, 541 us, 1110 TFLOP/s of products that count; trees of 64
// over 8 x 8192 tokens, fp16, 143 us (320 rows a head fill 2.5 tiles of 128).
// What bounds it is the softmax between the products: a sub-block's QK is 64 wide
// and takes the tensor cores as long as one of 128 (its operands come from shared
// memory), exponentials take 4 cycles a warp instruction, and each hand-over
// between a product and a softmax costs 100 to 200 cycles.  Of a launch's cycles
// the tensor pipe is active in 45%, the issue slots in 41%.  One stream of
// 128-wide products with a single issuer took 577 us, streams that take turns more.
#include "paged_attend.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 384;               // three warpgroups
constexpr int kSoft = 256;                  // softmax threads
constexpr int BN = kManyBlock;
constexpr int SB = BN / 2;                 // tokens of a sub-block
constexpr float kL2E = 1.4426950408889634f;
constexpr float kRaise = 8.0f;              // log2 of the growth that rescales
// From here on (in units of log2) the rounding of the maximum's product with c, 2^-24
// of it, counts: s c - max c is taken as (s - max) c and the maximum always raised
// (nearer ones are raised the earlier the larger they are).  One fma: with a second
// comparison the prompt chunk below takes 565 us instead of 540, the trees 146
// instead of 142.6.
constexpr float kHuge = 65536.0f;
constexpr int kOver = 2;                    // a unit's fixed cost in blocks

template <int D, int NQ>
struct Many {
  static constexpr int TILE = 128 * D * 2;                  // bytes of a Q tile, K or V block
  static constexpr int HALF = 128 * 128;                    // bytes of 64 channels of it
  static constexpr int ST = D == 128 ? 5 : 8;               // ring stages
  static constexpr int RING = NQ * TILE;
  static constexpr int SMEM = NQ * TILE + ST * TILE + 1024; // alignment slack
};

// The ring's order.  NQ = 2: K0 V0 K1 V1 ..; NQ = 1: K0 K1 V0 K2 V1 K3 .. V(n-1).
// Place of V of block b of n; the K that its stream needs next lies behind it.
template <int NQ>
__device__ __forceinline__ unsigned v_slot(int b, int n) {
  if (NQ == 2) return 2 * b + 1;
  return (n > 1 ? 2 : 1) + b + (n > 2 ? (b < n - 2 ? b : n - 2) : 0);
}

// A piece of a unit as the planning warp hands it to the others, through a
// ring in shared memory: none of them carries the walk's state in registers.
struct Piece {
  int more;                              // 0: the CTA's share ends here
  int b, h, mt, T, ctx, len, row0, lo, hi, pieces, first_cta;
  int tb, pre;                           // SH: as in WalkState
};
constexpr int kPlan = 8;                 // pieces in the ring
constexpr int kReaders = 11;             // warps that read it

// The softmax warps among themselves.  These barriers have no limit, so all eight
// warps have to come: whether they go on with a piece is decided by all of them
// together (soft_any), and what follows up to the next decision holds no wait.
// (Did each decide by itself, one could see that another warp has given up where
// the next still finds what it waits for and goes on to a barrier alone.)
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;\n" ::: "memory"); }
__device__ __forceinline__ bool soft_any(bool mine) {
  unsigned any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 2, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"(static_cast<unsigned>(mine))
      : "memory");
  return any != 0;
}

template <bool BF, int D, int NQ, bool SH>
__global__ void __launch_bounds__(kThreads, 1)
k_attend_many(const Pool p, const AttendArgs a, const Scratch sc, const int defer, const __grid_constant__ CUtensorMap mk,
              const __grid_constant__ CUtensorMap mv) {
  using M = Many<D, NQ>;
  constexpr int ST = M::ST;
  constexpr int TM = 128 * NQ;
  extern __shared__ unsigned char s_raw[];
  __shared__ __align__(8) unsigned long long s_bar[2 * ST + 15 + 2 * kPlan];
  __shared__ Piece s_plan[kPlan];
  __shared__ Sched s_sched;
  __shared__ long long s_scan[kThreads / 32];
  __shared__ float s_x[NQ == 1 ? 2 * 128 * 2 : 1];          // NQ = 1: the streams' (maximum, sum)
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_last, s_poison;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t ring = base + M::RING;
  const uint32_t bars = smem_addr(s_bar);
  // K and V stages full and empty; per stream: S there (two buffers), P there
  // (two), PV done, O done; Q there; a giving-up stream's products done
  const uint32_t b_full = bars, b_empty = bars + 8 * ST, b_s = bars + 16 * ST, b_p = b_s + 32, b_pv = b_p + 32,
                 b_o = b_pv + 16, b_q = b_o + 16, b_end = b_q + 8, b_plan = b_end + 16, b_read = b_plan + 8 * kPlan;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      bar_init(b_full + 8 * i, 1);
      bar_init(b_empty + 8 * i, 2);       // both streams give every stage back
    }
    for (int i = 0; i < 4; ++i) {
      bar_init(b_s + 8 * i, 1);
      bar_init(b_p + 8 * i, 128);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(b_pv + 8 * i, 1);
      bar_init(b_o + 8 * i, 1);
      bar_init(b_end + 8 * i, 1);
    }
    bar_init(b_q, kSoft);
    for (int i = 0; i < kPlan; ++i) {
      bar_init(b_plan + 8 * i, 1);
      bar_init(b_read + 8 * i, kReaders);
    }
    s_abort = s_poison = 0;
    fence_bar_init();
    fence_async();
  }
  if (warp == 10) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_addr(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  // (phase 2 of a shared prefix waits for phase 1 where it joins the two: k_paged_attend.cu)
  const bool joins = SH && a.bt.phase == 2;
  if (!joins) {
    pdl_wait();
    pdl_trigger();
  } else {
    __threadfence();
  }
  fence_async_global();
  tc_fence_before();
  if (a.bt.B > 32) {
    Walk<TM, BN, kOver, SH> w(p, a.bt, a.rows);
    sched_init<kThreads>(w, &s_sched, s_scan, 4);
  } else {
    __syncthreads();          // barriers and tensor memory are there
  }
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // reading the plan, by whole warps: the next piece (false at the end or when
  // another warp has given up), and done with it
  unsigned plan = 0;
  auto next_piece = [&] {
    return bar_wait_warp(b_plan + 8 * (plan % kPlan), (plan / kPlan) & 1, &s_abort) && s_plan[plan % kPlan].more;
  };
  auto piece_done = [&] {
    __syncwarp();
    if (lane == 0) bar_arrive(b_read + 8 * (plan % kPlan));
    ++plan;
  };

  // 384 threads x 168 registers at launch = 256 x 216 + 128 x 72
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
    if (warp == 11) {
      // ---- the plan ----
      Walk<TM, BN, kOver, SH> w(p, a.bt, a.rows);
      if (a.bt.B <= 32) {
        const Sched sh = sched_warp(w, 4, 0, blockIdx.x, gridDim.x);
        w.start(sh);
      } else {
        w.start(s_sched);
      }
      for (bool more = true; more; ++plan) {
        more = w.next();
        if (plan >= kPlan && !bar_wait_warp(b_read + 8 * (plan % kPlan), (plan / kPlan - 1) & 1, &s_abort)) break;
        if (lane == 0) {
          s_plan[plan % kPlan] = Piece{more, w.b, w.h, w.mt, w.T, w.ctx, w.len, w.row0, w.lo, w.hi, w.pieces, w.first_cta,
                                     SH ? w.tb : 0, SH ? w.pre : 0};
          bar_arrive(b_plan + 8 * (plan % kPlan));
        }
      }
    } else if (warp == 10) {
      // ---- K and V blocks into the ring ----
      const uint64_t once = stream_policy(), again = reuse_policy();
      const int rows_per = p.ps < BN ? p.ps : BN;
      const int boxes = BN / rows_per;
      unsigned slot = 0;
      int flag = 0;
      bool ok = true;
      while (ok && next_piece()) {
        const Piece& w = s_plan[plan % kPlan];
        const int32_t* table = a.bt.table + static_cast<size_t>(SH ? w.tb : w.b) * a.bt.max_blocks;
        // other tiles of the head read the same blocks
        const uint64_t pol = w.T * p.g > TM ? again : once;
        auto load = [&](const CUtensorMap* map, int blk) {
          if (!ok) return;
          const unsigned st = slot % ST;
          if (slot >= ST && !bar_wait_warp(b_empty + 8 * st, (slot / ST - 1) & 1, &s_abort)) {
            ok = false;
            return;
          }
          const int j0 = blk * BN;
          const int live = (w.len - j0 + rows_per - 1) / rows_per;     // boxes with tokens of the sequence
          const int n = live < boxes ? live : boxes;
          if (lane == 0) bar_expect(b_full + 8 * st, static_cast<unsigned>(n * rows_per * D * 2));
          __syncwarp();
          if (lane < n * (D / 64)) {
            const int i = D == 128 ? lane >> 1 : lane, half = D == 128 ? lane & 1 : 0;
            const int j = j0 + i * rows_per;
            const int page = table[j >> p.ps_shift];
            const bool none = static_cast<unsigned>(page) >= static_cast<unsigned>(p.NP);
            if (none) flag = CONFKV_FLAG_BAD_PAGE;
            const int y = none ? kNoRows : (((a.layer * p.NP + page) * p.Hkv + w.h) << p.ps_shift) + (j & (p.ps - 1));
            tma_box(ring + st * M::TILE + half * M::HALF + i * rows_per * 128, map, 64 * half, y, b_full + 8 * st, pol);
          }
          ++slot;
        };
        if (NQ == 2) {
          for (int b = w.lo; b < w.hi; ++b) {
            load(&mk, b);
            load(&mv, b);
          }
        } else {
          load(&mk, w.lo);
          if (w.lo + 1 < w.hi) load(&mk, w.lo + 1);
          for (int b = w.lo; b < w.hi; ++b) {
            load(&mv, b);
            if (b + 2 < w.hi) load(&mk, b + 2);
          }
        }
        piece_done();
      }
      if (flag) atomicOr(p.err, flag);
      if (!ok)                    // no copy may land after the CTA has gone
        for (unsigned k = slot > ST ? slot - ST : 0; k < slot; ++k) bar_drain(b_full + 8 * (k % ST), (k / ST) & 1);
    } else if (warp < 10) {
      // ---- matrix products of one stream (the warp stays together; one elected thread issues) ----
      constexpr uint32_t id_qk = umma_idesc(BF, 128, SB, false), id_pv = umma_idesc(BF, 128, D, true);
      constexpr uint32_t hi = umma_hi(1024);
      const int s = warp - 8;
      const uint32_t ts = uniform(tmem + s * 128), to = uniform(tmem + 256 + s * 128),
                     q_lo = uniform(umma_lo(base + (NQ == 2 ? s * M::TILE : 0), 16)), k_lo = uniform(umma_lo(ring, 16)),
                     v_lo = uniform(umma_lo(ring, M::HALF));
      unsigned slot0 = 0, np = 0, nq = 0, seen = 0;
      bool ok = true;
      // Slot k is there.  A stream waits for every slot in turn, its own or not:
      // those before k that it has not waited for are the other stream's (NQ = 1)
      // and are given back at once.  (Were they passed over, a stage whose earlier
      // slot is still on its way would answer for the later one: a wait knows a
      // phase by its parity alone.)
      auto full = [&](unsigned k) {
        while (ok && seen <= k) {
          ok = bar_wait_warp(b_full + 8 * (seen % ST), (seen / ST) & 1, &s_abort);
          if (ok && seen < k) bar_arrive_warp(b_empty + 8 * (seen % ST));
          ++seen;
        }
        return ok;
      };
      auto give_back = [&](unsigned end) {    // what is left of the piece is the other stream's
        while (ok && seen < end) {
          ok = bar_wait_warp(b_full + 8 * (seen % ST), (seen / ST) & 1, &s_abort);
          if (ok) bar_arrive_warp(b_empty + 8 * (seen % ST));
          ++seen;
        }
      };
      auto release = [&](unsigned k) { umma_commit(b_empty + 8 * (k % ST)); };
      auto qk = [&](int i, unsigned k) {      // S of sub-block i = Q K^T, half i & 1 of K's stage
        const uint32_t kt = uniform(k_lo + (k % ST) * (M::TILE / 16) + (i & 1) * (SB * 128 / 16));
        const uint32_t d = uniform(ts + (i & 1) * SB);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint32_t o = ((x >> 2) * M::HALF + (x & 3) * 32) / 16;
          umma_ss(d, q_lo + o, hi, kt + o, hi, id_qk, x > 0);
        }
        umma_commit(b_s + 16 * s + 8 * (i & 1));
        if (i & 1) release(k);
      };
      auto pv = [&](int i, unsigned k) {      // O += P V
        const uint32_t vt = uniform(v_lo + (k % ST) * (M::TILE / 16) + (i & 1) * (SB * 128 / 16));
        const uint32_t pt = uniform(ts + (i & 1) * SB);
#pragma unroll
        for (int x = 0; x < SB / 16; ++x) umma_ts(to, pt + x * 8, vt + x * 128, hi, id_pv, i > 0 || x > 0);
        umma_commit(b_pv + 8 * s);
        if (i & 1) release(k);
      };
      while (ok && next_piece()) {
        const Piece& w = s_plan[plan % kPlan];
        const int nb = w.hi - w.lo;
        ok = bar_wait_warp(b_q, nq & 1, &s_abort);
        ++nq;
        if (!ok) break;
        tc_fence_after();
        const int mine = NQ == 2 ? nb : (nb + 1 - s) >> 1;
        if (mine > 0) {
          const unsigned k0 = slot0 + (NQ == 2 ? 0 : s);
          if (!full(k0)) break;
          qk(0, k0);
          qk(1, k0);
        }
        for (int i = 0; i < 2 * mine; ++i) {
          const unsigned v = slot0 + v_slot<NQ>(NQ == 2 ? i >> 1 : (i & ~1) + s, nb);
          const bool more = i + 2 < 2 * mine;  // this stream's next K lies behind V
          if (!(i & 1)) {
            if (!full(v)) break;
            if (more && !full(v + 1)) break;
          }
          ok = bar_wait_warp(b_p + 16 * s + 8 * (i & 1), (np >> 1) & 1, &s_abort);
          ++np;
          if (!ok) break;
          tc_fence_after();
          pv(i, v);
          if (more) qk(i, v + 1);
        }
        if (!ok) break;
        umma_commit(b_o + 8 * s);             // (also where the stream has no block: it is waited for)
        slot0 += 2 * nb;
        give_back(slot0);
        if (!ok) break;
        piece_done();
      }
      if (!ok) {
        // products in flight end before the CTA does
        umma_commit(b_end + 8 * s);
        bar_drain(b_end + 8 * s, 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
    // ---- softmax and epilogue ----
    const int s = warp >> 2;                              // stream
    const int r = (warp & 3) * 32 + lane;                 // row of its tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + s * 128, to = tmem + lanes + 256;
    const float c = a.scale * kL2E;
    unsigned ns = 0, no = 0, slot0 = 0;
    int4 cut = make_int4(0, 0, 0, 0);                     // the unit whose first piece this CTA ends with
    bool waited = !joins;
    while (!soft_any(!next_piece())) {
      const Piece& w = s_plan[plan % kPlan];
      const int nb = w.hi - w.lo;
      const int R = w.T * p.g;                           // rows of the head
      const int tile0 = w.mt * TM;
      // query rows into shared memory
      {
        constexpr int WD = D / 8;
        const int first = NQ == 2 ? s * 128 : 0;
        constexpr int NTH = NQ == 2 ? 128 : 256;
        const int me = NQ == 2 ? tid & 127 : tid;
#pragma unroll 8
        for (int i = me; i < 128 * WD; i += NTH) {
          const int row = i / WD, wd = i % WD, x = tile0 + first + row;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (x < R) {
            const int t = x / p.g;
            v = *reinterpret_cast<const uint4*>(a.q + (w.row0 + t) * a.qs + (w.h * p.g + x - t * p.g) * D + 8 * wd);
          }
          const uint32_t ad = swz128(base + (NQ == 2 ? s * M::TILE : 0) + (wd >> 3) * M::HALF, row, wd & 7);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(ad), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
        }
        fence_async();
        bar_arrive(b_q);
      }
      const int x = tile0 + (NQ == 2 ? s * 128 : 0) + r;  // this thread's row of the head
      const bool live = x - lane < R;                     // the warp holds rows
      const int t = x < R ? x / p.g : 0;
      const size_t row = w.row0 + t;
      // tokens that the whole unit sees (a sequence may be longer than its table)
      const int all_seen = a.bt.mask ? w.ctx : min(w.ctx + tile0 / p.g + 1, w.len);
      float m = -INFINITY, l = 0.0f;
      const int mine = NQ == 2 ? nb : (nb + 1 - s) >> 1;  // this stream's blocks
      for (int i = 0; i < 2 * mine; ++i) {
        const int bb = NQ == 2 ? i >> 1 : (i & ~1) + s;
        const int blk0 = (w.lo + bb) * BN, j0 = blk0 + (i & 1) * SB;
        const bool masked = j0 + SB > all_seen;
        const uint32_t tb = ts + (i & 1) * SB;
        if (!bar_wait_warp(b_s + 16 * s + 8 * (i & 1), (ns >> 1) & 1, &s_abort)) break;
        ++ns;
        tc_fence_after();
        if (!(i & 1) && blk0 + BN > all_seen) {
          // before the product may start: V's rows past the end and non-finite elements become zeroes
          const unsigned k = slot0 + v_slot<NQ>(bb, nb);
          if (!bar_wait_warp(b_full + 8 * (k % ST), (k / ST) & 1, &s_abort)) break;
          const uint32_t vt = ring + (k % ST) * M::TILE;
          for (int y = tid & 127; y < M::TILE / 16; y += 128) {
            const uint32_t ad = vt + 16 * y;
            uint32_t v[4], z = 0u;
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(ad) : "memory");
            const bool past = blk0 + ((y >> 3) & 127) >= w.len;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t bad = past ? 0xffffffffu : nonfinite2<BF>(v[e]);
              z |= v[e] & bad;
              if (!past && bad) *const_cast<volatile int*>(&s_poison) = 1;
              v[e] &= ~bad;
            }
            if (z) {
              __threadfence_block();
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(ad), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
            }
          }
          fence_async();
        }
        if (live) {
          // P with the maximum of what came before, while the sub-block's own is
          // found beside it: only where that has grown by 2^kRaise (always at
          // the start) is O rescaled and P taken again
          uint32_t sv[2][32];
          float mc = m == -INFINITY ? 0.0f : m * c;
          uint64_t sum[4];
          // 64 weights in groups of eight, the groups' steps interleaved (written
          // in order: the schedule is otherwise one pipe after another)
          float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
          // one fma at first; taken again, the difference first, which is exact near
          // the maximum however large both are (kHuge)
          auto arg = [&](float x, bool first) { return first ? fma_o(x, c, -mc) : mul_o(x - mc, c); };
          auto weights = [&](bool top) {
            uint32_t pk[2][16];
            float z[2][8];
            uint64_t e[2][4];
            auto sval = [&](int k) { return __uint_as_float(sv[k >> 5][k & 31]); };
#pragma unroll
            for (int y = 0; y < 8; ++y) z[0][y] = arg(sval(y), top);
#pragma unroll
            for (int g = 0; g <= 8; ++g) {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                if (g < 8) {
                  const float e0 = ex2_o(z[g & 1][2 * y]);
                  if (g < 7) {
                    z[(g + 1) & 1][2 * y] = arg(sval(8 * g + 8 + 2 * y), top);
                    z[(g + 1) & 1][2 * y + 1] = arg(sval(8 * g + 9 + 2 * y), top);
                  }
                  const float e1 = ex2_o(z[g & 1][2 * y + 1]);
                  if (top) mx[y] = max3_o(mx[y], sval(8 * g + 2 * y), sval(8 * g + 2 * y + 1));
                  e[g & 1][y] = pair(e0, e1);
                }
                if (g > 0) {
                  const uint64_t d2 = e[(g - 1) & 1][y];
                  sum[y] = add2_o(sum[y], d2);
                  const float2 f2 = unpair(d2);
                  pk[(g - 1) >> 2][((g - 1) & 3) * 4 + y] = pack2_o<BF>(f2.x, f2.y);
                }
              }
              if (g == 4) tmem_st16(tb, pk[0]);          // over columns that have been read
            }
            tmem_st16(tb + 16, pk[1]);
          };
          sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
          {
            tmem_ld32(sv[0], tb);
            tmem_ld32(sv[1], tb + 32);
            tmem_wait_ld(sv[0]);
            tmem_wait_ld(sv[1]);
            if (masked) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t bits = x < R ? seen_bits(a.bt, row, t, w.ctx, w.len, j0 + 32 * q) : 0u;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(bits >> e & 1u)) sv[q][e] = 0xff800000u;
              }
            }
            __syncwarp();
            weights(true);
          }
          const float mn = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
          const bool raise = (m == -INFINITY) ? mn > -INFINITY : fmaf(fabsf(mc), kRaise / kHuge, (mn - m) * c) > kRaise;
          if (__any_sync(0xffffffffu, raise)) {
            const float f = m == -INFINITY ? 0.0f : ex2f((m - mn) * c);
            m = mn;
            l *= f;
            mc = m == -INFINITY ? 0.0f : m;
            tmem_wait_st();                   // the first P before its replacement
            if (i > 0) {
              // the product before this one has to be in O
              if (bar_wait_warp(b_pv + 8 * s, (ns - 2) & 1, &s_abort)) tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < D; q += 32) {
                uint32_t o[32];
                tmem_ld32(o, to + s * 128 + q);
                tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(to + s * 128 + q, o);
              }
            }
            sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
            weights(false);
          }
          const float2 y = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
          l += y.x + y.y;
          tmem_wait_st();
        }
        tc_fence_before();
        bar_arrive(b_p + 16 * s + 8 * (i & 1));
      }
      const bool whole = w.pieces == 1;
      if (SH && !waited) {
        waited = true;
        pdl_wait();
        pdl_trigger();
      }
      if (tid == 0 && !whole) {
        // all other pieces done: this one is joined as it is, without a way through memory
        s_last = !defer && *const_cast<volatile unsigned int*>(sc.ticket + w.first_cta) == static_cast<unsigned>(w.pieces - 1);
        __threadfence();
      }
      // (a stream without a block too: its issuing warp may not fall a piece behind)
      if (bar_wait_warp(b_o + 8 * s, no & 1, &s_abort)) tc_fence_after();
      ++no;
      slot0 += 2 * nb;
      if (NQ == 1) {
        s_x[(s * 128 + r) * 2] = m;
        s_x[(s * 128 + r) * 2 + 1] = l;
        tc_fence_before();
      }
      // (a thread that gave up a wait has set s_abort itself)
      if (soft_any(*const_cast<volatile int*>(&s_abort) != 0)) break;
      tc_fence_after();
      float w0 = 1.0f, w1 = 0.0f;                         // NQ = 1: the streams' weights
      if (NQ == 1) {
        const float m0 = s_x[r * 2], m1 = s_x[(128 + r) * 2], l0 = s_x[r * 2 + 1], l1 = s_x[(128 + r) * 2 + 1];
        m = fmaxf(m0, m1);
        w0 = m0 == -INFINITY ? 0.0f : ex2f((m0 - m) * c);
        w1 = m1 == -INFINITY ? 0.0f : ex2f((m1 - m) * c);
        l = l0 * w0 + l1 * w1;
      }
      const bool last = !whole && s_last;
      const int own = static_cast<int>(blockIdx.x) - w.first_cta;   // which piece this is
      const bool poison = *const_cast<volatile int*>(&s_poison) != 0;
      constexpr int COLS = NQ == 1 ? D / 2 : D;           // of this thread's row
      const int col0 = NQ == 1 ? s * (D / 2) : 0;
      const int xr = NQ == 1 ? r : s * 128 + r;           // row of the unit
      const int hq = w.h * p.g + x - t * p.g;
      const size_t place = 2 * static_cast<size_t>(blockIdx.x) + (w.lo == (SH ? w.pre / BN : 0) ? 1 : 0);
      if (live) {
#pragma unroll 1
        for (int q = 0; q < COLS; q += 32) {
          uint32_t o[32];
          float y[32];
          __syncwarp();
          tmem_ld32(o, to + (NQ == 1 ? 0 : s * 128) + col0 + q);
          tmem_wait_ld(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(o[i]);
          if (NQ == 1 && nb > 1) {
            tmem_ld32(o, to + 128 + col0 + q);
            tmem_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = y[i] * w0 + __uint_as_float(o[i]) * w1;
          }
          if (x < R) {
            if (poison) {
              const int32_t* table = a.bt.table + static_cast<size_t>(SH ? w.tb : w.b) * a.bt.max_blocks;
              int jb = all_seen / BN * BN;
              jb = jb < w.lo * BN ? w.lo * BN : jb;
              const int je = w.hi * BN < w.len ? w.hi * BN : w.len;
              for (int j = jb; j < je; ++j) {
                const int page = table[j >> p.ps_shift];
                if (page < 0 || page >= p.NP || !(seen_bits(a.bt, row, t, w.ctx, w.len, j) & 1u)) continue;
                const uint16_t* v = p.v + (((static_cast<size_t>(a.layer) * p.NP + page) * p.Hkv + w.h) * p.ps + (j & (p.ps - 1))) * D + col0 + q;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float z = to_f(v[i], BF);
                  if (!(fabsf(z) < INFINITY)) y[i] += z;
                }
              }
            }
            if (whole) {
              store_row<BF, SH>(a, p, static_cast<int>(row), hq, col0 + q, y, m, l, SH && w.pre);
            } else if (last) {
              float jm = m, jl = l;
              join_row<TM, D, 32, 1>(sc, w, xr, col0 + q, c, own, y, jm, jl);
              store_row<BF, SH>(a, p, static_cast<int>(row), hq, col0 + q, y, jm, jl, SH && w.pre);
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(acc_at<TM, D>(sc, place, xr, col0 + q + i)) =
                    make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
              if (col0 + q == 0) *reinterpret_cast<float2*>(sc.ml + (place * TM + xr) * 2) = make_float2(m, l);
            }
          }
        }
        tc_fence_before();
      }
      if (last) {
        if (tid == 0) sc.ticket[w.first_cta] = 0u;
        soft_sync();         // s_last and, NQ = 1, both streams' O are read before any thread goes on
      } else if (!whole && !defer) {
        __threadfence();
        soft_sync();
        if (tid == 0) {
          s_last = atomicAdd(sc.ticket + w.first_cta, 1u) == static_cast<unsigned>(w.pieces - 1);
          if (s_last) sc.ticket[w.first_cta] = 0u;
        }
        soft_sync();
        if (s_last) {
          __threadfence();
          // few rows: more threads to a row's channels
          const int rows = R - tile0 < TM ? R - tile0 : TM;
          const int pad = rows > 128 ? 256 : rows > 64 ? 128 : 64;
          const int jr = tid & (pad - 1), jx = tile0 + jr;
          constexpr int JN = 32;
          if (jr < rows) {
            const int jt = jx / p.g;
#pragma unroll 1
            for (int ch = (tid / pad) * JN; ch < D; ch += (kSoft / pad) * JN) {
              float y[JN] = {}, jm, jl;
              join_row<TM, D, JN, 2>(sc, w, jr, ch, c, -1, y, jm, jl);
              store_row<BF, SH>(a, p, w.row0 + jt, w.h * p.g + jx - jt * p.g, ch, y, jm, jl, SH && w.pre);
            }
          }
        }
      } else if (NQ == 1 || !whole) {
        soft_sync();
      }
      if (defer && tid == 0 && !whole && own == 0) cut = make_int4(w.pieces, w.b, w.h, w.mt);
      piece_done();
    }
    if (SH && !waited) pdl_wait();
    if (defer && tid == 0) sc.cut[blockIdx.x] = cut;
    tc_fence_before();
  }
  __syncthreads();
  if (s_abort && tid == 0) atomicOr(p.err, CONFKV_FLAG_TIMEOUT);
    if (warp == 10) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
  }
}

// The cut units of a deferring launch (tiles of 128 rows), joined on all SMs:
// blockIdx.x is the CTA that held a unit's first piece, a thread takes 8
// channels of a row.  (8 units of 65 rows in 19 pieces each: 20 us where 8
// CTAs join, 3 us here.)
constexpr int kJoinThreads = 128;
template <bool BF, int D, bool SH>
__global__ void __launch_bounds__(kJoinThreads)
k_join(const Pool p, const AttendArgs a, const Scratch sc) {
  pdl_wait();
  pdl_trigger();
  const int4 cut = sc.cut[blockIdx.x];
  if (cut.x < 2) return;
  Walk<128, BN, kOver, SH> w(p, a.bt, a.rows);
  int flag = 0;
  w.sequence(cut.y, flag);
  w.first_cta = blockIdx.x;
  w.pieces = cut.x;
  const int row = threadIdx.x, ch = 8 * blockIdx.y, x = cut.w * 128 + row;
  if (x >= w.T * p.g) return;
  float y[8] = {}, m, l;
  join_row<128, D, 8, 10>(sc, w, row, ch, a.scale * kL2E, -1, y, m, l);
  const int t = x / p.g;
  store_row<BF, SH>(a, p, w.row0 + t, cut.z * p.g + x - t * p.g, ch, y, m, l, SH && w.pre);
}

template <bool BF, int D, int NQ, bool SH>
cudaError_t go(const Pool& p, const AttendArgs& a, const Scratch& sc, const AttendMaps& m, int ctas, bool defer,
               cudaStream_t s) {
  const cudaError_t e = launch_pdl(k_attend_many<BF, D, NQ, SH>, dim3(ctas), dim3(kThreads), Many<D, NQ>::SMEM, s, p, a, sc,
                                   defer ? 1 : 0, m.k_many, m.v_many);
  if (e != cudaSuccess || !defer) return e;
  return launch_pdl(k_join<BF, D, SH>, dim3(ctas, D / 8), dim3(kJoinThreads), 0, s, p, a, sc);
}
template <bool BF, int D, int NQ>
cudaError_t set() {
  const cudaError_t e =
      cudaFuncSetAttribute(k_attend_many<BF, D, NQ, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Many<D, NQ>::SMEM);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(k_attend_many<BF, D, NQ, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Many<D, NQ>::SMEM);
}

template <bool SH>
cudaError_t launch_of(const Pool& p, const AttendArgs& a, const Scratch& sc, const AttendMaps& m, int ctas, bool two_tiles,
                      bool defer, cudaStream_t s) {
  if (two_tiles) {
    if (p.bf16) return p.d == 128 ? go<true, 128, 2, SH>(p, a, sc, m, ctas, defer, s) : go<true, 64, 2, SH>(p, a, sc, m, ctas, defer, s);
    return p.d == 128 ? go<false, 128, 2, SH>(p, a, sc, m, ctas, defer, s) : go<false, 64, 2, SH>(p, a, sc, m, ctas, defer, s);
  }
  if (p.bf16) return p.d == 128 ? go<true, 128, 1, SH>(p, a, sc, m, ctas, defer, s) : go<true, 64, 1, SH>(p, a, sc, m, ctas, defer, s);
  return p.d == 128 ? go<false, 128, 1, SH>(p, a, sc, m, ctas, defer, s) : go<false, 64, 1, SH>(p, a, sc, m, ctas, defer, s);
}

}  // namespace

cudaError_t launch_attend_many(const Pool& p, const AttendArgs& a, const Scratch& sc, const AttendMaps& m, int ctas,
                               bool two_tiles, bool defer, cudaStream_t s) {
  const cudaError_t e = a.bt.phase ? launch_of<true>(p, a, sc, m, ctas, two_tiles, defer, s)
                                   : launch_of<false>(p, a, sc, m, ctas, two_tiles, defer, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t setup_attend_many() {
  cudaError_t e = cudaSuccess;
  for (const cudaError_t r : {set<true, 128, 2>(), set<true, 64, 2>(), set<false, 128, 2>(), set<false, 64, 2>(),
                              set<true, 128, 1>(), set<true, 64, 1>(), set<false, 128, 1>(), set<false, 64, 1>()})
    if (e == cudaSuccess) e = r;
  return e;
}

}  // namespace paged
}  // namespace confkv
