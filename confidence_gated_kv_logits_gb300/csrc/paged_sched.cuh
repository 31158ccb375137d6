// How the paged attention's work is spread over its CTAs.
//
// A unit is one (sequence, KV head, tile of TM query rows); query row r of a
// sequence's KV head is new token r / g, head r % g of the group.  A unit's
// work is the blocks of KB tokens that its rows may see plus kOverhead blocks
// for its prologue and epilogue.  All units' work is laid end to end (sequence,
// head, tile) and cut into equal shares, one per CTA, so that the batch's
// lengths, known on the device alone, balance whatever they are.  A unit that
// is cut has its pieces' partial results joined by the CTA that finishes last,
// in the pieces' order, so results do not depend on timing.
#pragma once
#include "paged_internal.cuh"

namespace confkv {
namespace paged {

struct Sched {          // of one CTA: sched_warp, or for more than 32 sequences sched_init
  long long share;      // work per CTA
  long long cur, end;   // this CTA's range of the work
  // the sequence in which the range starts, and where its work does
  long long seq0, head;  // head: work of one of its heads
  int b, T, ctx, len, row0;
  int whole;             // units are not cut: each counts as 1, whatever its length
};

// 64-bit quotients of numbers that mostly fit 32 bits (a 64-bit division costs
// some 100 cycles of a launch that may last a few thousand)
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

struct Scratch {        // of the handle: partial results of cut units
  float* acc;           // [CTA][2][d / 4][TM][4]
  float* ml;            // [CTA][2][TM][2] (maximum, sum)
  unsigned int* ticket; // [CTA] of the unit whose first piece it holds: pieces done
  int4* cut;            // [CTA] that unit for the joining kernel: pieces, sequence, head, tile
};

struct WalkState {
  long long share, cur, end, ustart;
  int b, h, mt;
  int T, ctx, len, row0, m;     // of sequence b; m = tiles per head

  // a piece of a unit: blocks [lo, hi) of its n
  int lo, hi, n;
  int first_cta, pieces;        // CTAs that hold the unit's pieces
  int unit_done;                // the walk is behind the unit's last piece
  int more;                     // there is a piece
  int whole;                    // of Sched
};

template <int TM, int KB, int kOverhead>
struct Walk : WalkState {
  const Pool& p;
  const Batch& bt;
  int rows;

  __device__ __forceinline__ Walk(const Pool& p_, const Batch& b_, int rows_) : p(p_), bt(b_), rows(rows_) {}

  // what of sequence b's lengths is usable; `flag` collects what is not
  __device__ __forceinline__ void sequence(int b_, int& flag) {
    b = b_;
    int s0 = bt.q_start[b], s1 = bt.q_start[b + 1];
    ctx = bt.ctx[b];
    if (ctx < 0) {
      flag |= CONFKV_FLAG_BAD_INDEX;
      ctx = 0;
    }
    s0 = s0 < 0 ? 0 : s0 > rows ? rows : s0;
    s1 = s1 < s0 ? s0 : s1 > rows ? rows : s1;
    row0 = s0;
    T = s1 - s0;
    const long long cap = static_cast<long long>(bt.max_blocks) << p.ps_shift;
    long long l = static_cast<long long>(ctx) + T;
    if (l > cap) {
      if (T) flag |= CONFKV_FLAG_CAPACITY;
      l = cap;
    }
    if (l > 0x7fffff00ll) l = 0x7fffff00ll;         // (a block more still fits an int)
    len = static_cast<int>(l);
    if (ctx > len) ctx = len;
    m = static_cast<int>((static_cast<long long>(T) * p.g + TM - 1) / TM);
  }
  // tokens that some row of tile t may see
  __device__ __forceinline__ int tile_len(int t) const {
    if (bt.mask) return len;
    // new tokens up to the tile's last row (rows x heads fit 31 bits)
    uint32_t last = (static_cast<uint32_t>(t + 1) * TM - 1) / static_cast<uint32_t>(p.g) + 1;
    last = last > static_cast<uint32_t>(T) ? T : last;
    return last < static_cast<uint32_t>(len - ctx) ? ctx + static_cast<int>(last) : len;
  }
  __device__ __forceinline__ int blocks(int t) const { return (tile_len(t) + KB - 1) / KB; }
  // work of one head of the sequence
  __device__ __forceinline__ long long head_work() const {
    if (bt.mask || m <= 1) return static_cast<long long>(m) * (blocks(0 < m ? m - 1 : 0) + kOverhead);
    long long w = 0;
    for (int t = 0; t < m; ++t) w += blocks(t) + kOverhead;
    return w;
  }

  __device__ __forceinline__ int cost(int t) const { return whole ? 1 : blocks(t) + kOverhead; }
  __device__ __forceinline__ void start(const Sched& s) {
    unit_done = 0;
    whole = s.whole;
    share = s.share;
    cur = s.cur;
    end = s.end;
    if (cur >= end) return;
    b = s.b;
    T = s.T;
    ctx = s.ctx;
    len = s.len;
    row0 = s.row0;
    m = static_cast<int>((static_cast<long long>(T) * p.g + TM - 1) / TM);
    h = static_cast<int>(quotient(cur - s.seq0, s.head));
    ustart = s.seq0 + h * s.head;
    mt = 0;
    if (m == 1) {
    } else if (bt.mask) {
      const long long u = cost(0);
      mt = static_cast<int>(quotient(cur - ustart, u));
      ustart += mt * u;
    } else {
      for (long long u = cost(0); cur >= ustart + u; u = cost(mt)) {
        ustart += u;
        ++mt;
      }
    }
  }
  // goes to the range's next piece; false behind the last one
  __device__ __forceinline__ bool next() {
    for (;;) {
      if (unit_done) {
        unit_done = 0;
        ustart += whole ? 1 : n + kOverhead;
        if (++mt == m) {
          mt = 0;
          if (++h == p.Hkv) {
            h = 0;
            int flag = 0, nb = b;
            if (cur < end) {
              do sequence(++nb, flag); while (T <= 0);
            }
          }
        }
      }
      if (cur >= end) {
        more = 0;
        return false;
      }
      n = blocks(mt);
      if (whole) {
        lo = 0;
        hi = n;
        first_cta = blockIdx.x;
        pieces = 1;
        ++cur;
        unit_done = 1;
        more = 1;
        return true;
      }
      const long long uend = ustart + n + kOverhead;
      const long long x1 = end < uend ? end : uend;
      const long long a = cur - ustart - kOverhead, z = x1 - ustart - kOverhead;
      lo = a > 0 ? static_cast<int>(a) : 0;
      hi = z > 0 ? static_cast<int>(z) : 0;
      first_cta = static_cast<int>(quotient(ustart + kOverhead, share));
      pieces = static_cast<int>(quotient(uend - 1, share)) - first_cta + 1;
      cur = x1;
      unit_done = x1 == uend;
      if (hi > lo) {
        more = 1;
        return true;
      }
    }
  }
};

// The share of CTA `cta` of `ctas`, and the sequence that it starts in.
template <typename W>
__device__ __forceinline__ void sched_share(Sched* s, long long all, int cta, int ctas, long long min_share) {
  const long long even = quotient(all + ctas - 1, ctas);
  s->share = even < min_share ? min_share : even;
  s->cur = static_cast<long long>(cta) * s->share;
  s->end = s->cur + s->share < all ? s->cur + s->share : all;
}

// Up to 32 sequences: every warp works the schedule out by itself, a lane per
// sequence, without a barrier.
// Where no unit has more than `uncut` blocks and each finds a CTA of its own,
// none is cut (joining the pieces would take longer than the blocks); nor is
// any where uncut < 0.  (cta, ctas: a cluster and the clusters, if those share
// a unit.)
template <typename W>
__device__ __forceinline__ Sched sched_warp(W& w, long long min_share, int uncut, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  int flag = 0, most = 0;
  long long x = 0, head = 0, units = 0;
  w.whole = 0;
  if (lane < w.bt.B) {
    w.sequence(lane, flag);
    if (w.T > 0) {
      head = w.head_work();
      units = static_cast<long long>(w.m) * w.p.Hkv;
      most = w.blocks(w.m - 1);
    }
    x = head * w.p.Hkv;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  Sched s;
  s.whole = 0;
  if (uncut < 0 || most <= uncut) {
    long long all = units;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (uncut < 0 || all <= ctas) {
      s.whole = 1;
      min_share = 1;
      x = units;
      head = units ? w.m : 0;
    }
  }
  if (flag && blockIdx.x == 0) atomicOr(w.p.err, flag);
  long long incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  sched_share<W>(&s, __shfl_sync(0xffffffffu, incl, 31), cta, ctas, min_share);
  const unsigned in = __ballot_sync(0xffffffffu, x > 0 && s.cur >= incl - x && s.cur < incl);
  const int b = in ? __ffs(in) - 1 : 0;
  s.b = b;
  s.seq0 = __shfl_sync(0xffffffffu, incl - x, b);
  s.head = __shfl_sync(0xffffffffu, head, b);
  s.T = __shfl_sync(0xffffffffu, w.T, b);
  s.ctx = __shfl_sync(0xffffffffu, w.ctx, b);
  s.len = __shfl_sync(0xffffffffu, w.len, b);
  s.row0 = __shfl_sync(0xffffffffu, w.row0, b);
  return s;
}

// Every thread of the CTA calls it (kT threads).  s_scan holds kT / 32
// 64-bit words.
template <int kT, typename W>
__device__ __forceinline__ void sched_init(W& w, Sched* s, long long* s_scan, long long min_share) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kW = kT / 32;
  const int B = w.bt.B;
  int flag = 0;
  long long mine = 0, total = 0;
  // a thread's sequences: one each where the batch has no more than kT
  for (int b = tid; b < B; b += kT) {
    w.sequence(b, flag);
    mine = w.T > 0 ? w.head_work() * w.p.Hkv : 0;
    total += mine;
  }
  if (flag && blockIdx.x == 0) atomicOr(w.p.err, flag);
  // with one pass the scan of `total` is that of the sequences
  auto scan = [&](long long x, long long& sum) {       // exclusive, over the CTA
    long long incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long before = 0;
    sum = 0;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const long long y = s_scan[i];
      before += i < warp ? y : 0;
      sum += y;
    }
    __syncthreads();
    return before + incl - x;
  };
  long long all;
  long long pre = scan(total, all);
  Sched mine_of;
  sched_share<W>(&mine_of, all, blockIdx.x, gridDim.x, min_share);
  const long long cur = mine_of.cur;
  if (tid == 0) {
    s->share = mine_of.share;
    s->cur = cur;
    s->end = mine_of.end;
  }
  auto here = [&](long long at, long long x) {      // this thread's sequence (in w) is the one
    s->b = w.b;
    s->T = w.T;
    s->ctx = w.ctx;
    s->len = w.len;
    s->row0 = w.row0;
    s->seq0 = at;
    s->head = quotient(x, w.p.Hkv);
    s->whole = 0;
  };
  if (cur < all) {
    if (B <= kT) {
      if (mine > 0 && cur >= pre && cur < pre + mine) here(pre, mine);
    } else {
      long long base = 0;
      for (int b0 = 0; b0 < B; b0 += kT) {
        long long x = 0, sum;
        if (b0 + tid < B) {
          w.sequence(b0 + tid, flag);
          x = w.T > 0 ? w.head_work() * w.p.Hkv : 0;
        }
        const long long at = base + scan(x, sum);
        if (x > 0 && cur >= at && cur < at + x) here(at, x);
        base += sum;
      }
    }
  }
  __syncthreads();
}

// Which of 32 tokens from place j0 on query row `t` (new token) of a sequence
// sees: bit i is token j0 + i.
__device__ __forceinline__ uint32_t seen_bits(const Batch& bt, size_t row, int t, int ctx, int len, int j0) {
  const int left = len - j0;                       // tokens of the sequence from j0 on
  if (left <= 0) return 0u;
  uint32_t bits;
  if (!bt.mask) {
    const int nv = ctx + t + 1 - j0;
    bits = nv <= 0 ? 0u : nv >= 32 ? 0xffffffffu : (1u << nv) - 1u;
  } else {
    const int x = j0 - ctx;
    if (x <= -32) {
      bits = 0xffffffffu;
    } else {
      const int k = x >> 5;                        // floor
      const uint32_t* mw = bt.mask + row * bt.mask_words;
      const uint32_t a = k < 0 ? 0xffffffffu : k < bt.mask_words ? mw[k] : 0u;
      const uint32_t c = k + 1 < bt.mask_words ? mw[k + 1] : 0u;
      bits = __funnelshift_r(a, c, x & 31);
    }
  }
  return left >= 32 ? bits : bits & ((1u << left) - 1u);
}

}  // namespace paged
}  // namespace confkv
