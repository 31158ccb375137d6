// Beam selection: the best K of beams x vocabulary by summed log-probability.
//
//   score(w, v) = scores[w] + z_wv - lse_w,   lse_w = ln sum_u exp z_wu
//
// Within a beam the order is that of its logits, so only each row's best K
// can be among the best K of all.  One pass over the logits: a CTA holds one
// slice of one row in registers, reduces it to (max, sum of exponentials) and
// its best K logits; the CTA that takes a sequence's last ticket (no CTA
// waits) joins the slices and orders the candidates.
//
// Best K of a block's values: the K-th largest of the threads' own maxima is
// reached by K values at least and, on data in no particular order, by few
// more.  The 16-byte words that hold them are set aside in shared memory and
// taken apart there by a thread per value (33.5 -> 30.5 us against picking them
// up inside the sum's unrolled loop: 128 rows of 201088 bf16 logits, K = 16), and
// the values ranked by counting.  Should more be kept than the buffers hold
// (long runs of equal values, or an order that follows the lanes), K rounds of a
// block-wide maximum give the same answer.
//
// That takes 26.2 us now, 4 rows of 50257 fp32 logits 8.6.  What bounds it:
// neither the 35 MB (5.2 us) nor the issue slots (55% of the SMs' active cycles)
// but each slice's chain (load, maximum, bound, exponentials, ranking, ticket, with
// barriers between) in 896 CTAs, two per SM and so three waves, and the last
// sequence's join behind it: the SMs are active in 58% of the launch.
//
// Precision: exponentials and their sums per thread are fp32, relative to the
// slice's maximum (the largest terms are exact); sums over threads and slices
// are whole numbers of 2^-38 (exact in any order, and off the slow double
// pipe); the slices' weights and lse are 64-bit whole numbers and double, the
// candidates' scores double, rounded to fp32 once, at the end.  So lse's error is
// that of the exponentials and of a thread's sum: 1e-8 to 4e-8 measured (flat and
// peaked rows, normal logits of deviation 1 and 4, 50257 and 201088 tokens), and
// with |d| the weighted mean distance from the row's maximum at worst 2^-22
// (ex2.approx) + 2.25 2^-24 |d| (the argument's roundings, |d| <= ln V) + 12 2^-24
// (the sum), below 2^-18 for 2^18 tokens.  Candidates of different beams that are
// nearer than that may change places; equal scores go to the lower (beam, token).
#include <cmath>

#include "paged_internal.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCap = 1024;            // candidates ranked by counting
constexpr int kWords = 512;           // words of a slice that may hold them
constexpr int kMaxBeams = 32;
constexpr float kL2E = 1.4426950408889634f;

constexpr float kUnits = 274877906944.0f;     // 2^38: sums are whole numbers of 2^-38

// a slice's largest logit and sum of exp(z - max); sum ~0: a NaN or +inf was
// seen; 0: no finite logit
struct SlicePart {
  unsigned long long sum;
  float max;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// order-preserving integers (-0 counts as +0)
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ unsigned long long ordered(double x) {
  unsigned long long u = __double_as_longlong(x);
  u = u << 1 ? u : 0ull;
  return u ^ (static_cast<unsigned long long>(static_cast<long long>(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered(unsigned long long u) {
  return __longlong_as_double((u & 0x8000000000000000ull) ? u ^ 0x8000000000000000ull : ~u);
}

// (key, tie) pairs order by key, then by the larger tie
struct Cand {
  unsigned long long key, tie;
};
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
  return a.key > b.key || (a.key == b.key && a.tie > b.tie);
}

// the warp's 32 values in falling order over its lanes: a bitonic sort by shuffles
template <typename T>
__device__ __forceinline__ void warp_sort(T& x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int step = size >> 1; step > 0; step >>= 1) {
      const T y = __shfl_xor_sync(0xffffffffu, x, step);
      const bool desc = (lane & size) == 0;
      const bool low = (lane & step) == 0;
      x = (low == desc) ? (x > y ? x : y) : (x < y ? x : y);
    }
  }
}

// A value that at least K of the block's values reach, from each thread's
// largest (all threads call it, one barrier before and one behind): each warp
// gives its T largest of them, so that there are 16 T >= K; the bound is the K-th
// largest of these (K <= 32), or the smallest of the warps' T-th.  T = 2 from
// K = 9 on: with K = 16 of 16 values the bound is the weakest warp's and lets
// three times as many through (128 rows of 201088 bf16 logits, K = 16: 31.5
// against 30.5 us).  s_v: 32 values.
template <typename T>
__device__ __forceinline__ T block_bound(T mine, T lowest, int K, T* s_v) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = K <= kWarps / 2 ? 1 : K <= 2 * kWarps ? 2 : (K + kWarps - 1) / kWarps;
  T x = mine, top = lowest;
  for (int t = 0; t < per; ++t) {
    top = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const T y = __shfl_xor_sync(0xffffffffu, top, o);
      top = y > top ? y : top;
    }
    // one lane that holds it steps back
    const unsigned has = __ballot_sync(0xffffffffu, x == top);
    if (lane == __ffs(has) - 1) x = lowest;
    if (K <= 2 * kWarps && lane == 0) s_v[warp * per + t] = top;
  }
  if (K > 2 * kWarps && lane == 0) s_v[warp] = top;
  __syncthreads();
  // the one of the wanted rank, by counting what lies before each (a sort by
  // shuffles takes ten times as long)
  const int values = K > 2 * kWarps ? kWarps : kWarps * per;
  const T y = s_v[lane < values ? lane : 0];
  int rank = lane < values ? 0 : 32;
#pragma unroll 16
  for (int i = 0; i < values; ++i) {
    const T z = s_v[i];
    rank += z > y || (z == y && i < lane) ? 1 : 0;
  }
  const unsigned at = __ballot_sync(0xffffffffu, rank == (K > 2 * kWarps ? kWarps : K) - 1);
  __syncthreads();
  return __shfl_sync(0xffffffffu, y, at ? __ffs(at) - 1 : 0);     // (none: NaN among them, the row is left out)
}

// The K-th largest of the threads' largest itself (K <= 32; for more, the
// second best of the warps' (K / 2)-th), for values that are each the best of
// somewhere, so that the looser bound would keep most of them: the warps'
// sorted lanes merged pairwise.  s_v: 32 values per warp.
__device__ __forceinline__ uint32_t block_bound_tight(uint32_t x, int K, uint32_t* s_v) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  warp_sort(x);
  s_v[warp * 32 + lane] = x;
  __syncthreads();
  if (K > 32) {
    uint32_t w = s_v[(lane & (kWarps - 1)) * 32 + ((K + 1) >> 1) - 1];    // each warp's bound twice
    warp_sort(w);
    return __shfl_sync(0xffffffffu, w, 2);
  }
#pragma unroll
  for (int step = kWarps / 2; step > 0; step >>= 1) {
    if (warp < step) {
      // the larger of a falling and a rising list: the 32 largest, bitonic
      const uint32_t y = s_v[(warp + step) * 32 + 31 - lane];
      x = x > y ? x : y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const uint32_t z = __shfl_xor_sync(0xffffffffu, x, d);
        x = (lane & d) == 0 ? (x > z ? x : z) : (x < z ? x : z);
      }
      s_v[warp * 32 + lane] = x;
    }
    __syncthreads();
  }
  return s_v[K - 1];
}

// Powers of two in whole numbers, to a few 2^-60: the double pipe takes some 65
// cycles per dependent step, a 64-bit product 30.
__host__ __device__ constexpr unsigned long long inverse_factorial(int k) {      // 2^64 / k!
  unsigned long long f = 1;
  for (int i = 2; i <= k; ++i) f *= i;
  return ~0ull / f;
}
// 2^(f / 2^64) in units of 2^-63: e^r = 1 + r + r^2 (1/2! + r/3! + ..) with r =
// f ln 2 < 0.7 (up to r^17 / 17!, the even and the odd terms side by side)
__device__ __forceinline__ unsigned long long exp2_fraction(unsigned long long f) {
  const unsigned long long r = __umul64hi(f, 12786308645202655660ull);      // ln 2 * 2^64
  const unsigned long long r2 = __umul64hi(r, r);
  unsigned long long even = inverse_factorial(16), odd = inverse_factorial(17);
#pragma unroll
  for (int k = 14; k >= 2; k -= 2) {
    even = __umul64hi(even, r2) + inverse_factorial(k);
    odd = __umul64hi(odd, r2) + inverse_factorial(k + 1);
  }
  const unsigned long long s = even + __umul64hi(odd, r);
  return (1ull << 63) + ((r + __umul64hi(r2, s)) >> 1);
}
// 2^-a, 0 <= a < 1000, as fraction * 2^(n - 63)
struct Power {
  unsigned long long fraction;
  int n;
};
__device__ __forceinline__ Power exp2_neg(double a) {
  const long long t = -static_cast<long long>(a * 9007199254740992.0);      // 2^53
  return Power{exp2_fraction(static_cast<unsigned long long>(t) << 11), static_cast<int>(t >> 53)};
}
constexpr long long kNone = 0x7ff8000000000000ll;            // a NaN: the beam has no candidates of its logits
constexpr double kLog2E = 1.4426950408889634;
// sum * e^x, x <= 0, rounded down; sum < 2^63
__device__ __forceinline__ unsigned long long scaled(unsigned long long sum, double x) {
  const double a = -x * kLog2E;
  if (!(a < 63.0)) return 0ull;             // (below 1, and no shift by 64)
  const Power p = exp2_neg(a);
  return __umul64hi(sum << 1, p.fraction) >> -p.n;
}
// ln (sum / 2^38), sum >= 2^38: the fp32 logarithm y and one Newton step on e^y,
// for which sum * e^-y / 2^38 - 1 is taken in whole numbers (0 for sum = 2^38)
__device__ __forceinline__ double log_units(unsigned long long sum) {
  const float y = logf(static_cast<float>(sum) * (1.0f / kUnits));
  const Power p = exp2_neg(static_cast<double>(y) * kLog2E);
  const int s = __clzll(sum), k = 37 + s - p.n;             // one lies at 2^k
  const unsigned long long one = k < 64 ? 1ull << k : 0ull;
  const double d = static_cast<double>(static_cast<long long>(__umul64hi(sum << s, p.fraction) - one)) *
                   __longlong_as_double(static_cast<long long>(1023 - k) << 52);
  return static_cast<double>(y) + fma(-0.5 * d, d, d);
}

template <int DT>
__device__ __forceinline__ float elem(uint32_t w, int half) {
  if constexpr (DT == CONFKV_BF16) {
    return __uint_as_float(half ? (w & 0xffff0000u) : (w << 16));
  } else {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(half ? w >> 16 : w)));
  }
}

__device__ __forceinline__ Cand block_best(Cand c, Cand* s_best) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Cand d;
    d.key = __shfl_xor_sync(0xffffffffu, c.key, o);
    d.tie = __shfl_xor_sync(0xffffffffu, c.tie, o);
    if (before(d, c)) c = d;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_best[threadIdx.x >> 5] = c;
  __syncthreads();
  c = s_best[0];
  for (int w = 1; w < kWarps; ++w)
    if (before(s_best[w], c)) c = s_best[w];
  return c;
}

template <int DT, int EPT>
__global__ void __launch_bounds__(kThreads, 2)
k_beam_select(const BeamArgs a, int C, SlicePart* part, unsigned long long* cand, unsigned int* ticket) {
  constexpr int VEC = DT == CONFKV_FP32 ? 4 : 8;      // elements of a 16-byte word
  constexpr int NV = EPT / VEC;
  __shared__ Cand s_list[kCap];
  __shared__ unsigned long long s_sum[kWarps];
  __shared__ float s_f[kWarps];
  __shared__ unsigned long long s_v[kThreads];
  __shared__ Cand s_best[kWarps];
  __shared__ double s_base[kMaxBeams];
  __shared__ int s_cnt, s_words, s_bad, s_last;
  __shared__ uint4 s_word[kWords];
  __shared__ int s_place[kWords];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.y, b = row / a.W;
  const size_t slice = static_cast<size_t>(row) * C + blockIdx.x;
  if (tid == 0) s_cnt = s_words = s_bad = 0;
  pdl_wait();
  pdl_trigger();
  const float score = a.scores[row];
  const bool skip = (a.finished && a.finished[row]) || !(score > -INFINITY) || !(score < INFINITY);
  if (!skip) {
    uint4 x[NV];
    // 16-byte words counted from the aligned address at or before the row
    const int size = DT == CONFKV_FP32 ? 4 : 2;
    const char* base = static_cast<const char*>(a.logits) + static_cast<size_t>(row) * a.stride * size;
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / size);
    const long long w0 = static_cast<long long>(blockIdx.x) * (kThreads * NV);
    const uint32_t ninf = DT == CONFKV_FP32 ? 0xff800000u : DT == CONFKV_BF16 ? 0xff80ff80u : 0xfc00fc00u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const long long v = (w0 + i * kThreads + tid) * VEC - lead;   // token of the word's first element
      if (v >= 0 && v + VEC <= a.V) {
        x[i] = __ldcs(reinterpret_cast<const uint4*>(base + v * size));
      } else {
        uint32_t w[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if (v + e < 0 || v + e >= a.V) continue;
          if constexpr (DT == CONFKV_FP32) {
            w[e] = reinterpret_cast<const uint32_t*>(base)[v + e];
          } else {
            const uint32_t h = reinterpret_cast<const uint16_t*>(base)[v + e];
            w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | (h << 16) : (w[e >> 1] & 0xffff0000u) | h;
          }
        }
        x[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    auto value = [&](int i, int e) -> float {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i]);
      if constexpr (DT == CONFKV_FP32) return __uint_as_float(w[e]);
      else return elem<DT>(w[e >> 1], e & 1);
    };
    // largest value of a word; of all words (16-bit types two at a time; NaN is passed over)
    auto top_of = [&](uint32_t a0, uint32_t a1) -> uint32_t {
      uint32_t r;
      if constexpr (DT == CONFKV_BF16) asm("max.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a0), "r"(a1));
      else if constexpr (DT == CONFKV_FP16) asm("max.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a0), "r"(a1));
      else r = __float_as_uint(fmaxf(__uint_as_float(a0), __uint_as_float(a1)));
      return r;
    };
    auto word_top = [&](const uint4& w) { return top_of(top_of(w.x, w.y), top_of(w.z, w.w)); };
    auto top_value = [&](uint32_t t) {
      if constexpr (DT == CONFKV_FP32) return __uint_as_float(t);
      else return fmaxf(elem<DT>(t, 0), elem<DT>(t, 1));
    };
    uint32_t mw = word_top(x[0]);
#pragma unroll
    for (int i = 1; i < NV; ++i) mw = top_of(mw, word_top(x[i]));
    const float m = top_value(mw);
    // the passes unpack the values anew instead of holding all of them as floats
    auto again = [&] {
#pragma unroll
      for (int i = 0; i < NV; ++i) asm volatile("" : "+r"(x[i].x), "+r"(x[i].y), "+r"(x[i].z), "+r"(x[i].w));
    };
    again();
    float bm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
    if (lane == 0) s_f[warp] = bm;
    const float bound = block_bound(m, -INFINITY, a.K, reinterpret_cast<float*>(s_v));    // (its barriers publish s_f)
    bm = s_f[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) bm = fmaxf(bm, s_f[w]);
    float sum = 0.0f;
    if (bm > -INFINITY && bm < INFINITY) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float part4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        // (z - max) first, which is exact for what weighs: z's product alone would lose digits
#pragma unroll
        for (int e = 0; e < VEC; ++e) part4[e & 3] += ex2((value(i, e) - bm) * kL2E);
        sum += (part4[0] + part4[1]) + (part4[2] + part4[3]);
        // words that hold a candidate: taken apart below, by other threads
        if (top_value(word_top(x[i])) >= bound) {
          const int at = atomicAdd(&s_words, 1);
          if (at < kWords) {
            s_word[at] = x[i];
            s_place[at] = i * kThreads + tid;
          }
        }
      }
    } else if (!(bm >= INFINITY)) {         // no finite logit, but perhaps a NaN (the maxima pass over it)
      again();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum = value(i, e) == value(i, e) ? sum : NAN;
    }
    // NaN anywhere in the slice makes its sum NaN, +inf its maximum
    if (!(sum < INFINITY) || bm == INFINITY) s_bad = 1;
    // the sum goes on in whole units: exact, in any order, and off the double pipe
    const unsigned long long mine = sum < 65536.0f ? static_cast<unsigned long long>(sum * kUnits) : 0ull;   // (NaN: 0)
    const unsigned lo = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(mine) & 0x7ffffffu);
    const unsigned hi = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(mine >> 27));
    if (lane == 0) s_sum[warp] = (static_cast<unsigned long long>(hi) << 27) + lo;
    __syncthreads();
    const int words = s_words;
    if (words <= kWords) {
      for (int i = tid; i < words * VEC; i += kThreads) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&s_word[i / VEC]);
        const int e = i % VEC;
        float z;
        if constexpr (DT == CONFKV_FP32) z = __uint_as_float(w[e]);
        else z = elem<DT>(w[e >> 1], e & 1);
        if (z >= bound && z > -INFINITY) {
          const uint32_t v = static_cast<uint32_t>((w0 + s_place[i / VEC]) * VEC - lead + e);
          const int at = atomicAdd(&s_cnt, 1);
          if (at < kCap) s_list[at].key = (static_cast<unsigned long long>(ordered(z)) << 32) | (0xffffffffu - v);
        }
      }
      __syncthreads();
    }
    const int cnt = words <= kWords ? s_cnt : kCap + 1;
    unsigned long long* out = cand + slice * a.K;
    if (tid == 0) {
      unsigned long long t = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += s_sum[w];
      part[slice] = SlicePart{s_bad ? ~0ull : t, bm};
    }
    if (cnt <= kCap) {
      for (int i = tid; i < cnt; i += kThreads) {
        const unsigned long long k = s_list[i].key;
        int rank = 0;
        for (int j = 0; j < cnt; ++j) rank += s_list[j].key > k;
        if (rank < a.K) out[rank] = k;
      }
      for (int i = cnt + tid; i < a.K; i += kThreads) out[i] = 0;
    } else {
      Cand last{~0ull, 0};
#pragma unroll 1
      for (int r = 0; r < a.K; ++r) {
        Cand c{0, 0};
        again();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float z = value(i, e);
            const uint32_t v = static_cast<uint32_t>((w0 + i * kThreads + tid) * VEC - lead + e);
            const unsigned long long k = (static_cast<unsigned long long>(ordered(z)) << 32) | (0xffffffffu - v);
            if (z > -INFINITY && k < last.key && k > c.key) c.key = k;
          }
        last = block_best(c, s_best);
        if (tid == 0) out[r] = last.key;
        if (last.key == 0) {        // nothing left: the rest is empty
          for (int i = r + 1 + tid; i < a.K; i += kThreads) out[i] = 0;
          break;
        }
      }
    }
  }
  // the sequence's last CTA goes on
  __syncthreads();
  if (tid == 0) {
    s_last = take_ticket(&ticket[b]) == static_cast<unsigned>(C * a.W - 1);
    s_cnt = 0;
  }
  __syncthreads();
  if (!s_last) return;
  if (tid == 0) ticket[b] = 0u;

  // everything that the last stage reads is asked for at once
  const int per = C * a.K, n = a.W * per;
  constexpr int kHeld = 4;                  // candidates of a thread that stay in registers
  unsigned long long raw[kHeld];
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    raw[u] = tid + u * kThreads < n ? __ldcg(cand + static_cast<size_t>(b) * n + tid + u * kThreads) : 0ull;

  // Each beam's score minus lse (NaN: no candidates of its logits).  The slices'
  // sums relative to the row's maximum are whole units again, exact in any order;
  // the slice that holds it counts as it is, so a row of one token gives exactly 0.
  const SlicePart* pp = part + static_cast<size_t>(b) * a.W * C;
  auto part_of = [&](int i) {
    const ulonglong2 v = __ldcg(reinterpret_cast<const ulonglong2*>(pp + i));
    return SlicePart{v.x, v.x ? __uint_as_float(static_cast<unsigned>(v.y)) : -INFINITY};
  };
  auto units = [&](const SlicePart& y, float m) {
    return scaled(y.sum, static_cast<double>(y.max) - static_cast<double>(m));
  };
  // of beam w, whose slices' maximum and sum are given
  auto finish = [&](int w, float sc, bool done, float m, bool bad, unsigned long long sum) {
    const int r = b * a.W + w;
    int flag = 0;
    double base = __longlong_as_double(kNone);
    if (!(sc < INFINITY)) {
      flag = CONFKV_FLAG_NONFINITE;
    } else if (sc > -INFINITY && !done) {
      if (bad || !(m > -INFINITY)) flag = CONFKV_FLAG_NONFINITE;
      else base = static_cast<double>(sc) -
                  (static_cast<double>(m) + log_units(sum));
    }
    s_base[w] = base;
    if (a.flags_out) a.flags_out[r] = flag;
  };
  const int pairs = a.W * C;
  if (pairs <= kThreads) {
    // a thread per slice, then one per beam: few warps come to the double pipe (2
    // results a cycle: with a warp per beam, four of them, this took a quarter of
    // the call for 4 beams of 50257)
    float* s_top = reinterpret_cast<float*>(s_list);
    const float sc = tid < a.W ? a.scores[b * a.W + tid] : 0.0f;     // (asked for ahead)
    const bool done = tid < a.W && a.finished && a.finished[b * a.W + tid];
    SlicePart q{0ull, -INFINITY};
    if (tid < pairs) {
      q = part_of(tid);
      s_top[tid] = q.sum == ~0ull ? NAN : q.max;
    }
    __syncthreads();
    auto top_of_beam = [&](int w, bool& bad) {
      float m = -INFINITY;
      for (int c = 0; c < C; ++c) {
        const float y = s_top[w * C + c];
        bad |= y != y;
        m = fmaxf(m, y);
      }
      return m;
    };
    if (tid < pairs) {
      bool bad = false;
      const float m = top_of_beam(tid / C, bad);
      s_v[tid] = q.sum && !bad ? units(q, m) : 0ull;
    }
    __syncthreads();
    if (tid < a.W) {
      bool bad = false;
      const float m = top_of_beam(tid, bad);
      unsigned long long sum = 0;
      for (int c = 0; c < C; ++c) sum += s_v[tid * C + c];
      finish(tid, sc, done, m, bad, sum);
    }
  } else {
    for (int w = warp; w < a.W; w += kWarps) {        // a warp per beam, its lanes over the slices
      float m = -INFINITY;
      bool bad = false;
      for (int c = lane; c < C; c += 32) {
        const SlicePart y = part_of(w * C + c);
        m = fmaxf(m, y.max);
        bad |= y.sum == ~0ull;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      bad = __any_sync(0xffffffffu, bad);
      unsigned long long sum = 0;
      for (int c = lane; c < C; c += 32) {
        const SlicePart y = part_of(w * C + c);
        if (y.sum && !bad) sum += units(y, m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const int r = b * a.W + w;
      if (lane == 0) finish(w, a.scores[r], a.finished && a.finished[r], m, bad, sum);
    }
  }
  __syncthreads();

  // candidate i of the sequence: slice lists, then one of each finished beam
  auto candidate = [&](int i, unsigned long long k) -> Cand {
    Cand c{0, 0};
    if (i < n) {
      const int w = i / per;
      const double base = s_base[w];
      if (__double_as_longlong(base) != kNone) {
        if (k) {
          c.key = ordered(base + static_cast<double>(unordered(static_cast<uint32_t>(k >> 32))));
          c.tie = ~((static_cast<unsigned long long>(w) << 32) | (0xffffffffu - static_cast<uint32_t>(k)));
        }
      }
    } else {
      const int w = i - n;
      const float sc = a.scores[b * a.W + w];
      if (a.finished && a.finished[b * a.W + w] && sc > -INFINITY && sc < INFINITY) {
        c.key = ordered(static_cast<double>(sc));
        c.tie = ~((static_cast<unsigned long long>(w) << 32) | static_cast<unsigned>(a.pad));
      }
    }
    return c;
  };
  auto fetched = [&](int i) { return candidate(i, i < n ? __ldcg(cand + static_cast<size_t>(b) * n + i) : 0ull); };
  Cand held[kHeld];
  uint32_t top = 0;           // the scores' upper halves bound them well enough (and sort twice as fast)
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    held[u] = Cand{0, 0};
    if (tid + u * kThreads < n + a.W) held[u] = candidate(tid + u * kThreads, raw[u]);
    const uint32_t k = static_cast<uint32_t>(held[u].key >> 32);
    top = k > top ? k : top;
  }
  for (int i = tid + kHeld * kThreads; i < n + a.W; i += kThreads) {
    const uint32_t k = static_cast<uint32_t>(fetched(i).key >> 32);
    top = k > top ? k : top;
  }
  const uint32_t bound = block_bound_tight(top, a.K, reinterpret_cast<uint32_t*>(s_v));
  auto keep = [&](const Cand& c) {
    if (c.key && (c.key >> 32) >= bound) {
      const int at = atomicAdd(&s_cnt, 1);
      if (at < kCap) s_list[at] = c;
    }
  };
#pragma unroll
  for (int u = 0; u < kHeld; ++u) keep(held[u]);
  for (int i = tid + kHeld * kThreads; i < n + a.W; i += kThreads) keep(fetched(i));
  __syncthreads();
  const int cnt = s_cnt;
  auto put = [&](int r, const Cand& c) {
    const size_t o = static_cast<size_t>(b) * a.K + r;
    const unsigned long long at = ~c.tie;
    a.score_out[o] = c.key ? static_cast<float>(unordered(c.key)) : -INFINITY;
    a.parent_out[o] = c.key ? static_cast<int>(at >> 32) : -1;
    a.token_out[o] = c.key ? static_cast<int>(at & 0xffffffffull) : -1;
  };
  if (cnt <= kCap) {
    for (int i = tid; i < cnt; i += kThreads) {
      const Cand c = s_list[i];
      int rank = 0;
      for (int j = 0; j < cnt; ++j) rank += before(s_list[j], c);
      if (rank < a.K) put(rank, c);
    }
    for (int i = cnt + tid; i < a.K; i += kThreads) put(i, Cand{0, 0});
  } else {
    Cand last{~0ull, ~0ull};
    for (int r = 0; r < a.K; ++r) {
      Cand best{0, 0};
      for (int i = tid; i < n + a.W; i += kThreads) {
        const Cand c = fetched(i);
        if (c.key && before(last, c) && before(c, best)) best = c;
      }
      last = block_best(best, s_best);
      if (tid == 0) put(r, last);
      if (!last.key) {
        for (int i = r + 1 + tid; i < a.K; i += kThreads) put(i, Cand{0, 0});
        break;
      }
    }
  }
}

// Elements per thread: short slices while they do not fill the GPU twice (a
// slice's fixed cost is then latency), long ones where there are many rows.
int beam_ept(long long rows, int V, int dtype) {
  const long long short_slices = rows * ((V + kThreads * 8 - 1) / (kThreads * 8));
  if (short_slices <= 2 * 152) return 8;
  return dtype == CONFKV_FP32 ? 32 : 64;
}
int beam_slices(long long rows, int V, int dtype) {
  const int per = kThreads * beam_ept(rows, V, dtype);
  const int lead = dtype == CONFKV_FP32 ? 3 : 7;     // a row may start inside a 16-byte word
  return static_cast<int>((static_cast<long long>(V) + lead + per - 1) / per);
}
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

template <int DT>
cudaError_t launch_dt(const BeamArgs& a, int C, SlicePart* part, unsigned long long* cand,
                      unsigned int* ticket, cudaStream_t s) {
  const dim3 grid(C, a.B * a.W);
  constexpr int kLong = DT == CONFKV_FP32 ? 32 : 64;
  if (beam_ept(static_cast<long long>(a.B) * a.W, a.V, DT) == 8)
    return launch_pdl(k_beam_select<DT, 8>, grid, dim3(kThreads), 0, s, a, C, part, cand, ticket);
  return launch_pdl(k_beam_select<DT, kLong>, grid, dim3(kThreads), 0, s, a, C, part, cand, ticket);
}

}  // namespace

// [tickets][parts: rows x slices][candidates: rows x slices x K].  The tickets,
// which every call leaves zero, have a place of their own whatever a call's
// sizes are (one for each sequence that a call can have): calls of several sizes
// may share a workspace.
constexpr size_t kTicketBytes = sizeof(unsigned int) * 65536;

size_t beam_workspace(int B, int W, int V, int K, int dtype) {
  const size_t n = static_cast<size_t>(B) * W * beam_slices(static_cast<long long>(B) * W, V, dtype);
  return kTicketBytes + round256(sizeof(SlicePart) * n) + sizeof(unsigned long long) * n * K;
}

cudaError_t launch_beam(const BeamArgs& a, cudaStream_t s) {
  const int C = beam_slices(static_cast<long long>(a.B) * a.W, a.V, a.dtype);
  const size_t n = static_cast<size_t>(a.B) * a.W * C;
  char* w = static_cast<char*>(a.ws);
  unsigned int* ticket = reinterpret_cast<unsigned int*>(w);
  w += kTicketBytes;
  SlicePart* part = reinterpret_cast<SlicePart*>(w);
  w += round256(sizeof(SlicePart) * n);
  unsigned long long* cand = reinterpret_cast<unsigned long long*>(w);
  cudaError_t e;
  if (a.dtype == CONFKV_FP32) e = launch_dt<CONFKV_FP32>(a, C, part, cand, ticket, s);
  else if (a.dtype == CONFKV_BF16) e = launch_dt<CONFKV_BF16>(a, C, part, cand, ticket, s);
  else e = launch_dt<CONFKV_FP16>(a, C, part, cand, ticket, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
