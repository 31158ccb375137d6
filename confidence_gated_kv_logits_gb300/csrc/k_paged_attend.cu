// Attention of few new rows per sequence over a paged cache (single tokens,
// small trees): up to 16 query rows of a KV head at a time, streaming its
// cached K and V once.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(scale (q_r k_j) - max)
//
// The work is the cache's bytes, so everything serves the stream of tiles:
// each warp reads its own chunks of 8 KB (16 tokens at d = 128, 32 at d = 64;
// K and V boxes of the page, by TMA with the 128-byte swizzle) through a ring
// of its own, with no barrier between warps until the unit's end.  A chunk is
// 16 query rows x its tokens on mma.sync m16n8k16 (rows on M: the query
// fragments stay in registers, S's accumulators are P's A fragments as they
// are); these rows are too few for tcgen05's 64 or 128, and the matrix work is
// far below the memory's time.  Softmax statistics are fp32 per row and warp;
// P is rounded to the cache's type (fp16 by 2^-11 of its value at most, bf16 by
// 2^-8), which weighs as much as the output's own rounding.  Warps join through
// shared memory.  A unit is spread over CTAs in one of two ways: cut into equal
// shares (paged_sched.cuh), its pieces joined through the handle's scratch, which
// fills the GPU whatever the lengths are; or, where all units run at once and none
// can be long, shared by a cluster of two to eight CTAs that join it through
// distributed shared memory (the rule and its figures: paged_api.cu).
//
// Long caches are bound by HBM: 32 sequences of up to 16384 tokens, 64/8 heads of
// 64 channels (733 MB) take 119 us, 6.15 TB/s.  Short ones by the chain ctx_len ->
// page number -> tile -> product -> join.  Eight warps with rings of three chunks,
// one CTA per SM (192 KB in flight), against three CTAs of four warps with rings
// of two: 35 against 49 us for 1 x 32768 tokens of 40/8 x 128 heads.
//
// Chunks that reach past what every row sees are masked by bits per row; in
// them V's rows past the end are zeroed in shared memory, and so are
// non-finite elements (0 x NaN would reach rows that do not see them), which
// the rows that do see them get added by hand.
#include <climits>
#include <type_traits>

#include "paged_attend.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kRows = kFewRows;
// Chunks of a unit that one CTA takes whole, while every unit finds a CTA of its
// own and no cluster shares it. Cut against whole, one row: 1 x 128 tokens of
// 40/8 x 128 heads 11.1 against 8.4 us, 8 x 700 tokens of 12/12 x 64 13.9 against
// 9.0; at 16 chunks a warp (1 x 1024 tokens, d 128) 12.1 against 15.2.
constexpr int kUncut = 8 * kWarps;
constexpr int kChunkBytes = 4 * kFewChunk;
constexpr float kL2E = 1.4426950408889634f;

template <int D>
struct Few {
  static constexpr int CH = kFewChunk / D;             // tokens of a chunk
  static constexpr int NT = CH / 8;                // score column tiles
  static constexpr int KS = D / 16;                // k-steps of q k
  static constexpr int OT = D / 8;                 // output column tiles
  static constexpr int KV = CH * D * 2;            // bytes of K (of V) in a chunk
  static constexpr int HALF = CH * 128;            // bytes of one 64-channel half
  static constexpr int OVER = 2 * kWarps;          // a unit's fixed cost in chunks
};

// CL > 1: the CTAs of a cluster share each of their units, which are not cut
// otherwise, and join them through distributed shared memory.
template <bool BF, int D, int CL>
__global__ void __launch_bounds__(kThreads, 1)
k_attend_few(const Pool p, const AttendArgs a, const Scratch sc, const __grid_constant__ CUtensorMap mk,
             const __grid_constant__ CUtensorMap mv) {
  using F = Few<D>;
  extern __shared__ unsigned char s_raw[];
  __shared__ __align__(8) unsigned long long s_bar[kWarps * kStages];
  __shared__ float s_ml[kWarps][kRows][2];
  __shared__ Sched s_sched;
  __shared__ WalkState s_walk;
  __shared__ long long s_scan[kWarps];
  __shared__ float s_all[kRows][2];                 // CL > 1: the CTA's (maximum, sum) of each row
  __shared__ int s_abort, s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int STEP = kWarps * CL;                 // a warp's next chunk
  const int rank = CL > 1 ? blockIdx.x % CL : 0, wid = rank * kWarps + warp;
  const uint32_t ring0 = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t ring = ring0 + warp * (kStages * kChunkBytes);
  const uint32_t bar = smem_addr(&s_bar[warp * kStages]);
  if (lane == 0)
    for (int i = 0; i < kStages; ++i) bar_init(bar + 8 * i, 1);
  if (tid == 0) s_abort = 0;
  fence_bar_init();
  fence_async();
  pdl_wait();
  pdl_trigger();
  fence_async_global();

  // the walk stays in shared memory: its registers are the accumulators' between pieces
  using WalkF = Walk<kRows, F::CH, F::OVER>;
  if (a.bt.B > 32) {
    WalkF w(p, a.bt, a.rows);
    sched_init<kThreads>(w, &s_sched, s_scan, 2 * kWarps);
  }
  if (warp == 0) {
    WalkF w(p, a.bt, a.rows);
    if (a.bt.B > 32) {
      w.start(s_sched);
    } else {
      const Sched sh = sched_warp(w, 2 * kWarps, CL > 1 ? -1 : kUncut, blockIdx.x / CL, gridDim.x / CL);
      w.start(sh);
    }
    w.next();
    if (lane == 0) s_walk = w;
  }
  __syncthreads();
  const WalkState& w = s_walk;
  const uint64_t pol = stream_policy();
  const float c = a.scale * kL2E;
  unsigned turn = 0;                                // chunks this warp has taken so far
  const int r0 = lane >> 2, t4 = lane & 3;

  while (w.more) {
    const int b = w.b, h = w.h;
    const int32_t* table = a.bt.table + static_cast<size_t>(b) * a.bt.max_blocks;
    const int layer_row = (a.layer * p.NP) * p.Hkv;  // page of head h: (layer_row + page * Hkv + h) * ps
    int flag = 0;
    // boxes of 16 rows (or the whole chunk, where a page holds it); lane i asks
    // for box i (d = 128: half i & 1 of box i / 2)
    const int box = p.ps < F::CH ? p.ps : F::CH;
    const int my_box = D == 128 ? lane >> 1 : lane, my_half = D == 128 ? lane & 1 : 0;
    auto boxes = [&](int ci) {                        // those with tokens of the sequence
      const int live = (w.len - ci * F::CH + box - 1) / box;
      return live < F::CH / box ? live : F::CH / box;
    };
    // the lane's page of a chunk, read well before its boxes are asked for
    auto page_of = [&](int ci) { return ci < w.hi && my_box < boxes(ci) ? table[(ci * F::CH + my_box * box) >> p.ps_shift] : 0; };
    auto issue = [&](int ci, unsigned k, int page) {
      const int st = k % kStages;
      const uint32_t dst = ring + st * kChunkBytes, fb = bar + 8 * st;
      const int n = boxes(ci);
      if (lane == 0) bar_expect(fb, static_cast<unsigned>(n * box * D * 4));
      __syncwarp();
      if (my_box < n && lane < F::CH / box * (D / 64)) {
        const bool none = static_cast<unsigned>(page) >= static_cast<unsigned>(p.NP);
        if (none) flag = CONFKV_FLAG_BAD_PAGE;
        const int j = ci * F::CH + my_box * box;
        const int y = none ? kNoRows : ((layer_row + page * p.Hkv + h) << p.ps_shift) + (j & (p.ps - 1));
        const uint32_t o = dst + my_half * F::HALF + my_box * box * 128;
        tma_box(o, &mk, 64 * my_half, y, fb, pol);
        tma_box(o + F::KV, &mv, 64 * my_half, y, fb, pol);
      }
    };
    const int first = w.lo + wid;
    const unsigned turn0 = turn;
    unsigned issued = turn0;
    bool dead = false;
    int pages[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) pages[i] = page_of(first + i * STEP);
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      if (first + i * STEP < w.hi) issue(first + i * STEP, issued++, pages[i]);
    int page_next = page_of(first + kStages * STEP);

    // the tile's query rows as A fragments (zero behind the sequence's rows)
    const int R = w.T * p.g, base = w.mt * kRows;
    const int ra = base + r0, rb = ra + 8;            // this thread's rows
    const int ta = ra / p.g, tb = rb / p.g;
    uint32_t qf[F::KS][4];
    {
      const uint16_t* qa = a.q + (w.row0 + ta) * a.qs + (h * p.g + ra - ta * p.g) * D + 2 * t4;
      const uint16_t* qb = a.q + (w.row0 + tb) * a.qs + (h * p.g + rb - tb * p.g) * D + 2 * t4;
#pragma unroll
      for (int k = 0; k < F::KS; ++k) {
        qf[k][0] = ra < R ? *reinterpret_cast<const uint32_t*>(qa + 16 * k) : 0u;
        qf[k][1] = rb < R ? *reinterpret_cast<const uint32_t*>(qb + 16 * k) : 0u;
        qf[k][2] = ra < R ? *reinterpret_cast<const uint32_t*>(qa + 16 * k + 8) : 0u;
        qf[k][3] = rb < R ? *reinterpret_cast<const uint32_t*>(qb + 16 * k + 8) : 0u;
      }
    }
    // tokens that every row of the tile sees (a sequence may be longer than its table)
    const int all_seen = a.bt.mask ? w.ctx : min(w.ctx + base / p.g + 1, w.len);
    float o[F::OT][4];
#pragma unroll
    for (int i = 0; i < F::OT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    float ma = -INFINITY, mb = -INFINITY, la = 0.0f, lb = 0.0f;

    for (int ci = first; ci < w.hi; ci += STEP) {
      const unsigned st = turn % kStages;
      if (!bar_wait_warp(bar + 8 * st, (turn / kStages) & 1, &s_abort)) {
        dead = true;
        break;
      }
      const uint32_t kt = ring + st * kChunkBytes, vt = kt + F::KV;
      const int j0 = ci * F::CH;
      float s[F::NT][4];
#pragma unroll
      for (int i = 0; i < F::NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
      for (int k = 0; k < F::KS; ++k) {
#pragma unroll
        for (int i = 0; i < F::NT; i += 2) {
          uint32_t f[4];
          // matrices: tokens 8i.., channels 16k..; channels +8; tokens + 8; both
          const int row = 8 * i + ((lane >> 4) << 3) + (lane & 7), wd = 2 * k + ((lane >> 3) & 1);
          ldsm4(f, swz128(kt + (wd >> 3) * F::HALF, row, wd & 7));
          mma16816<BF>(s[i], qf[k], f[0], f[1]);
          mma16816<BF>(s[i + 1], qf[k], f[2], f[3]);
        }
      }
      if (j0 + F::CH > all_seen) {
        const uint32_t ba = ra < R ? seen_bits(a.bt, w.row0 + ta, ta, w.ctx, w.len, j0) : 0u;
        const uint32_t bb = rb < R ? seen_bits(a.bt, w.row0 + tb, tb, w.ctx, w.len, j0) : 0u;
#pragma unroll
        for (int i = 0; i < F::NT; ++i) {
          const int x = 8 * i + 2 * t4;
          if (!(ba >> x & 1u)) s[i][0] = -INFINITY;
          if (!(ba >> (x + 1) & 1u)) s[i][1] = -INFINITY;
          if (!(bb >> x & 1u)) s[i][2] = -INFINITY;
          if (!(bb >> (x + 1) & 1u)) s[i][3] = -INFINITY;
        }
        // V: zeroes past the end; non-finite elements by hand
        bool odd = false;
        for (int i = lane; i < F::KV / 16; i += 32) {
          const int row = (i >> 3) % F::CH;           // words in order: halves, rows, words
          const uint32_t ad = vt + i * 16;
          uint32_t x[4];
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(ad) : "memory");
          if (j0 + row >= w.len) {
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};\n" ::"r"(ad), "r"(0u) : "memory");
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) odd |= nonfinite2<BF>(x[e]) != 0u;
          }
        }
        if (__any_sync(0xffffffffu, odd)) {
          __syncwarp();
          for (int j = 0; j < F::CH && j0 + j < w.len; ++j) {
            const bool sa = ba >> j & 1u, sb = bb >> j & 1u;
#pragma unroll
            for (int i = 0; i < F::OT; ++i) {
              uint32_t x;
              const int ch = 8 * i + 2 * t4;
              asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(x)
                           : "r"(swz128(vt + (ch >> 6) * F::HALF, j, (ch & 63) >> 3) + 2 * (ch & 7)) : "memory");
              const uint32_t bad = nonfinite2<BF>(x);
              const float2 v = unpack2<BF>(x);
              if (bad & 0xffffu) {
                if (sa) o[i][0] += v.x;
                if (sb) o[i][2] += v.x;
              }
              if (bad >> 16) {
                if (sa) o[i][1] += v.y;
                if (sb) o[i][3] += v.y;
              }
            }
          }
          __syncwarp();
          for (int i = lane; i < F::KV / 4; i += 32) {
            uint32_t x;
            asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(x) : "r"(vt + 4 * i) : "memory");
            x &= ~nonfinite2<BF>(x);
            asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(vt + 4 * i), "r"(x) : "memory");
          }
        }
        fence_async();        // these writes before the next box in this stage
        __syncwarp();
      }
      // running maximum and sum of the two rows (4 lanes share a row)
      float xa = fmaxf(s[0][0], s[0][1]), xb = fmaxf(s[0][2], s[0][3]);
#pragma unroll
      for (int i = 1; i < F::NT; ++i) {
        xa = fmaxf(xa, fmaxf(s[i][0], s[i][1]));
        xb = fmaxf(xb, fmaxf(s[i][2], s[i][3]));
      }
      xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
      xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
      xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
      xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
      if (__any_sync(0xffffffffu, xa > ma || xb > mb)) {
        const float na = fmaxf(ma, xa), nb = fmaxf(mb, xb);
        // (nothing seen before: all sums are 0 but for infinities added by hand above, which stay)
        const float fa = ma == -INFINITY ? 1.0f : ex2f((ma - na) * c);
        const float fb = mb == -INFINITY ? 1.0f : ex2f((mb - nb) * c);
        if (turn != turn0) {
#pragma unroll
          for (int i = 0; i < F::OT; ++i) {
            o[i][0] *= fa;
            o[i][1] *= fa;
            o[i][2] *= fb;
            o[i][3] *= fb;
          }
        }
        la *= fa;
        lb *= fb;
        ma = na;
        mb = nb;
      }
      // the difference first: it is exact near the maximum, however large both are
      // (s c - max c by one fma is off by max c's rounding, a factor of 2^128 for scores of 2^31)
      const float sa = ma == -INFINITY ? 0.0f : ma, sb = mb == -INFINITY ? 0.0f : mb;
#pragma unroll
      for (int i = 0; i < F::NT; ++i) {
        s[i][0] = ex2f((s[i][0] - sa) * c);
        s[i][1] = ex2f((s[i][1] - sa) * c);
        s[i][2] = ex2f((s[i][2] - sb) * c);
        s[i][3] = ex2f((s[i][3] - sb) * c);
        la += s[i][0] + s[i][1];
        lb += s[i][2] + s[i][3];
      }
#pragma unroll
      for (int i = 0; i < F::NT; i += 2) {
        const uint32_t pf[4] = {pack2<BF>(s[i][0], s[i][1]), pack2<BF>(s[i][2], s[i][3]),
                                pack2<BF>(s[i + 1][0], s[i + 1][1]), pack2<BF>(s[i + 1][2], s[i + 1][3])};
#pragma unroll
        for (int n = 0; n < F::OT; n += 2) {
          uint32_t f[4];
          // matrices (transposed): tokens 8i.., channels 8n..; tokens +8; channels +8; both
          const int row = 8 * i + (((lane >> 3) & 1) << 3) + (lane & 7), wd = n + (lane >> 4);
          ldsm4t(f, swz128(vt + (wd >> 3) * F::HALF, row, wd & 7));
          mma16816<BF>(o[n], pf, f[0], f[1]);
          mma16816<BF>(o[n + 1], pf, f[2], f[3]);
        }
      }
      __syncwarp();           // every lane has read the stage
      if (ci + kStages * STEP < w.hi) {
        issue(ci + kStages * STEP, issued++, page_next);
        page_next = page_of(ci + (kStages + 1) * STEP);
      }
      ++turn;
    }
    if (dead)                 // no copy may land after the CTA has gone
      for (unsigned k = turn; k < issued; ++k) bar_drain(bar + 8 * (k % kStages), (k / kStages) & 1);
    if (flag) atomicOr(p.err, flag);
    la += __shfl_xor_sync(0xffffffffu, la, 1);
    lb += __shfl_xor_sync(0xffffffffu, lb, 1);
    la += __shfl_xor_sync(0xffffffffu, la, 2);
    lb += __shfl_xor_sync(0xffffffffu, lb, 2);

    // the warps' partials: each in its own ring (rows of D floats), then joined
    {
#pragma unroll
      for (int i = 0; i < F::OT; ++i) {
        const uint32_t ch = 8 * i + 2 * t4;
        asm volatile("st.shared.v2.f32 [%0], {%1,%2};\n" ::"r"(ring + (r0 * D + ch) * 4), "f"(o[i][0]), "f"(o[i][1]) : "memory");
        asm volatile("st.shared.v2.f32 [%0], {%1,%2};\n" ::"r"(ring + ((r0 + 8) * D + ch) * 4), "f"(o[i][2]), "f"(o[i][3]) : "memory");
      }
      if (t4 == 0) {
        s_ml[warp][r0][0] = ma;
        s_ml[warp][r0][1] = la;
        s_ml[warp][r0 + 8][0] = mb;
        s_ml[warp][r0 + 8][1] = lb;
      }
    }
    __syncthreads();
    // set before the barrier or not at all; a cluster's CTAs leave together, below
    if (CL == 1 && s_abort) break;
    constexpr int PER = kRows * D / kThreads;        // 16 or 8 channels of one row
    const int row = tid / (D / PER), ch0 = (tid % (D / PER)) * PER;
    const bool whole = w.pieces == 1;
    float m = -INFINITY, l = 0.0f, x[PER];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) m = fmaxf(m, s_ml[i][row][0]);
#pragma unroll
    for (int e = 0; e < PER; ++e) x[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const float li = s_ml[i][row][1];
      if (li == 0.0f) continue;                       // nothing seen (scores that are all NaN leave m at -inf, l NaN)
      const float f = ex2f((s_ml[i][row][0] - m) * c);
      l += f * li;
      const uint32_t src = ring0 + i * (kStages * kChunkBytes) + (row * D + ch0) * 4;
#pragma unroll
      for (int e = 0; e < PER; e += 4) {
        float v[4];
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];\n"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(src + 4 * e) : "memory");
#pragma unroll
        for (int y = 0; y < 4; ++y) x[e + y] = fmaf(f, v[y], x[e + y]);
      }
    }
    const int rr = base + row;
    if constexpr (CL > 1) {
      // the CTA's rows into its second chunk (nothing else lies there now), then
      // each CTA joins kRows / CL of them
      const uint32_t mine = ring0 + kChunkBytes;
#pragma unroll
      for (int e = 0; e < PER; e += 4)
        asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};\n" ::"r"(mine + (row * D + ch0 + e) * 4), "f"(x[e]), "f"(x[e + 1]),
                     "f"(x[e + 2]), "f"(x[e + 3]) : "memory");
      if (ch0 == 0) {
        s_all[row][0] = m;
        s_all[row][1] = l;
      }
      cluster_sync();
      bool dead_any = false;
#pragma unroll
      for (int i = 0; i < CL; ++i) dead_any |= ld_cluster_u32(cluster_addr(smem_addr(&s_abort), i)) != 0u;
      const int jr = rank * (kRows / CL) + tid / (D / 4), jc = tid % (D / 4) * 4, js = base + jr;
      if (!dead_any && tid < kRows / CL * (D / 4) && js < R) {
        float2 ml[CL];
        float4 v[CL];
#pragma unroll
        for (int i = 0; i < CL; ++i) {
          ml[i] = ld_cluster_f2(cluster_addr(smem_addr(&s_all[jr][0]), i));
          v[i] = ld_cluster_f4(cluster_addr(mine + (jr * D + jc) * 4, i));
        }
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < CL; ++i) m = fmaxf(m, ml[i].x);
#pragma unroll
        for (int i = 0; i < CL; ++i) {
          if (ml[i].y == 0.0f) continue;
          const float f = ex2f((ml[i].x - m) * c);
          l = fmaf(f, ml[i].y, l);
          y[0] = fmaf(f, v[i].x, y[0]);
          y[1] = fmaf(f, v[i].y, y[1]);
          y[2] = fmaf(f, v[i].z, y[2]);
          y[3] = fmaf(f, v[i].w, y[3]);
        }
        const int t = js / p.g;
        store_row<BF, 4>(a, p, w.row0 + t, h * p.g + js - t * p.g, jc, y, m, l);
      }
      cluster_sync();         // nobody leaves or goes on while its rows are read
      if (dead_any) break;
    } else if (whole) {
      if (rr < R) {
        const int t = rr / p.g;
        store_row<BF, PER>(a, p, w.row0 + t, h * p.g + rr - t * p.g, ch0, x, m, l);
      }
    } else {
      const size_t at = 2 * static_cast<size_t>(blockIdx.x) + (w.lo == 0 ? 1 : 0);
      if (rr < R) {
#pragma unroll
        for (int e = 0; e < PER; e += 4)
          *reinterpret_cast<float4*>(acc_at<kRows, D>(sc, at, row, ch0 + e)) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        if (ch0 == 0) *reinterpret_cast<float2*>(sc.ml + (at * kRows + row) * 2) = make_float2(m, l);
      }
      __syncthreads();
      if (tid == 0) {
        s_last = take_ticket(sc.ticket + w.first_cta) == static_cast<unsigned>(w.pieces - 1);
        if (s_last) sc.ticket[w.first_cta] = 0u;
      }
      __syncthreads();
      if (s_last) {
        // The pieces in their order, as many at a time as the rings hold: all of a
        // batch's words are asked for at once (a thread that walked its own words
        // through L2 one piece after another took 3 to 6 us for 9 pieces).
        const int live = R - base < kRows ? R - base : kRows;
        const int per_piece = live * (D / 4) + live / 2 + 1;            // 16-byte words, (maximum, sum) pairs behind
        const int batch = kWarps * kStages * kChunkBytes / (16 * per_piece);
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int e = 0; e < PER; ++e) x[e] = 0.0f;
        for (int i0 = 0; i0 < w.pieces; i0 += batch) {
          const int nb = w.pieces - i0 < batch ? w.pieces - i0 : batch;
          const int words = live * (D / 4);
          for (int it = tid; it < nb * words; it += kThreads) {
            const int i = it / words, y = it - i * words, ch = y / live, r = y - ch * live;
            cp_async16(ring0 + (i * per_piece + r * (D / 4) + ch) * 16, acc_at<kRows, D>(sc, piece_place(w, i0 + i), r, 4 * ch));
          }
          const int twos = (live + 1) / 2;                              // two rows' pairs are a word
          for (int it = tid; it < nb * twos; it += kThreads) {
            const int i = it / twos, r = it - i * twos;
            cp_async16(ring0 + (i * per_piece + words + r) * 16, sc.ml + (piece_place(w, i0 + i) * kRows + 2 * r) * 2);
          }
          cp_async_wait();
          __syncthreads();
          if (row < live) {
            float mn = m;
            for (int i = 0; i < nb; ++i) mn = fmaxf(mn, lds_f2(ring0 + (i * per_piece + words) * 16 + row * 8).x);
            const float f0 = m == -INFINITY ? 0.0f : ex2f((m - mn) * c);
            l *= f0;
#pragma unroll
            for (int e = 0; e < PER; ++e) x[e] *= f0;
            m = mn;
            for (int i = 0; i < nb; ++i) {
              const float2 ml = lds_f2(ring0 + (i * per_piece + words) * 16 + row * 8);
              if (ml.y == 0.0f) continue;
              const float f = ex2f((ml.x - m) * c);
              l = fmaf(f, ml.y, l);
#pragma unroll
              for (int e = 0; e < PER; e += 4) {
                float v[4];
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];\n"
                             : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                             : "r"(ring0 + (i * per_piece + row * (D / 4) + (ch0 + e) / 4) * 16) : "memory");
#pragma unroll
                for (int y = 0; y < 4; ++y) x[e + y] = fmaf(f, v[y], x[e + y]);
              }
            }
          }
          __syncthreads();
        }
        if (row < live) {
          const int t = rr / p.g;
          store_row<BF, PER>(a, p, w.row0 + t, h * p.g + rr - t * p.g, ch0, x, m, l);
        }
      }
    }
    fence_async();
    __syncthreads();          // the rings are free again, the piece has been read
    if (warp == 0) {
      WalkF on(p, a.bt, a.rows);
      static_cast<WalkState&>(on) = s_walk;
      on.next();
      __syncwarp();
      if (lane == 0) s_walk = on;
    }
    __syncthreads();
  }
  if (s_abort && tid == 0) atomicOr(p.err, CONFKV_FLAG_TIMEOUT);
}

// f of every instance, until one fails
template <typename F>
cudaError_t each_few(F&& f) {
  cudaError_t e = cudaSuccess;
  auto of = [&](auto bf, auto d) {
    auto one = [&](auto cl) {
      if (e == cudaSuccess) e = f(bf, d, cl, k_attend_few<decltype(bf)::value, decltype(d)::value, decltype(cl)::value>);
    };
    one(std::integral_constant<int, 1>{});
    one(std::integral_constant<int, 2>{});
    one(std::integral_constant<int, 4>{});
    one(std::integral_constant<int, 8>{});
  };
  of(std::false_type{}, std::integral_constant<int, 64>{});
  of(std::false_type{}, std::integral_constant<int, 128>{});
  of(std::true_type{}, std::integral_constant<int, 64>{});
  of(std::true_type{}, std::integral_constant<int, 128>{});
  return e;
}

}  // namespace

cudaError_t launch_attend_few(const Pool& p, const AttendArgs& a, const Scratch& sc, const AttendMaps& m,
                              int ctas, int cluster, cudaStream_t s) {
  const size_t smem = kWarps * kStages * kChunkBytes + 1024;
  return each_few([&](auto bf, auto d, auto cl, auto kernel) {
    if (bf != p.bf16 || d != p.d || cl != cluster) return cudaSuccess;
    cudaError_t e;
    if (cl > 1) e = launch_pdl_cluster(kernel, dim3(ctas), dim3(kThreads), cl, smem, s, p, a, sc, m.k_few, m.v_few);
    else e = launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem, s, p, a, sc, m.k_few, m.v_few);
    return e != cudaSuccess ? e : cudaGetLastError();
  });
}

cudaError_t few_clusters(int size, int* fit) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kWarps * kStages * kChunkBytes + 1024;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = size;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  *fit = INT_MAX;
  return each_few([&](auto, auto, auto cl, auto kernel) {
    int n = INT_MAX;
    const cudaError_t e = cl == size ? cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) : cudaSuccess;
    *fit = n < *fit ? n : *fit;
    return e;
  });
}

cudaError_t setup_attend_few() {
  return each_few([](auto, auto, auto, auto kernel) {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kWarps * kStages * kChunkBytes + 1024);
  });
}

}  // namespace paged
}  // namespace confkv
