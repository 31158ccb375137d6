// Eviction from a paged cache: each KV head of each sequence and layer keeps N of
// its n tokens; those behind the budget move into the places of evicted ones.
//
// Order: the sequence's first places, then its newest positions, then the larger
// mass; equal ones by the lower place.  Classes and masses are one 32-bit key
// (masses in an order-preserving form); the N-th largest key is found by four
// rounds of counting one byte each, and of the keys equal to it the lowest places
// stay.  Evicted places below N (holes) and kept places from N on (movers) are
// equally many; the r-th hole takes the r-th mover's rows, which no other move
// reads or writes, so all moves are independent.  Up to eight evicted places are
// found one by one instead, as minima, while the rows behind the budget, which
// may have to move, are on their way.
//
// The work is bytes: masses and positions once, moved rows twice.  64 layers x 8 x 8 heads
// of 2049 tokens that lose one, out of place (137 MB): 33 us, 61% of the copy rate,
// bound by each CTA's chain (length -> masses -> newest position -> minimum -> page) at
// four CTAs per SM; 97.6 by counting bytes.  16 layers x 4 x 8 heads of 8192 that come down to 1024
// or 2048 (665 MB): 148 us, 66%, rows of 256 bytes scattered over the pools; 203 with
// the r-th set bit searched for by each lane, 207 with positions in shared memory (three CTAs per SM instead of four).
#include <type_traits>

#include "paged_internal.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kU = 8;                   // loads of a thread in flight
constexpr uint32_t kFirst = 0xffffffffu, kNewest = 0xfffffffeu;
constexpr int kKeysShared = 40960;      // keys up to here stay in shared memory
constexpr int kPosShared = 4096;        // positions too up to here
constexpr int kList = 8192;             // moves at a time beyond
constexpr int kFew = 8;                 // evicted places that are found one by one, a warp each
// Places (of the mass's rows) from which on units that leave SMs idle are worth 1024 threads instead of 256.  us, 256 and
// 1024: 8 units of 1500 places, 1000 kept, 14.9, 16.6; of 4000, 1000 kept, 24.8, 22.7; of 16000, 2000 kept, 66.6, 44.0; 64
// of 4000 42.3, 27.5; 152 of 10000, 5000 kept, 137.5, 89.8; 64 of 2049, one evicted, 4.2, 5.3.  With more units than SMs
// four CTAs of 256 do more than one of 1024 while shared memory holds them: 160 of 4000, 1000 kept, 51.4, 65.4; of 10000,
// 5000 kept, 143, 156; 304 of 16000, 2000 kept, 182, 150.  From some 20000 places on it holds two at most, and 256 are the
// slower ones (160 of 30000, half kept, 674, 398; 608 of 45000, 4000 kept, 1833, 689) but for rows that are far longer
// than their sequences (160 of 1000 in 30000 20, 27; 304 in 100000 17, 29), which the host cannot tell: left as it is.
constexpr int kWide = 2500;

// A mass as an unsigned number in the same order; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// What the threads before give, and the CTA's sum.
template <int kWarps>
__device__ __forceinline__ int scan(int x, int* s_warp, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    before += i < warp ? s_warp[i] : 0;
    all += s_warp[i];
  }
  return before + incl - x;
}

// n places as they are (out of line: the kernel's registers are the other paths')
__device__ __noinline__ void pass_on(const float* mass, const int32_t* pos, float* mass_out, int32_t* pos_out, int n) {
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    mass_out[j] = mass[j];
    pos_out[j] = pos[j];
  }
}

// One CTA: a KV head of a sequence in a layer.  KEYS: its keys lie in shared memory, and its positions too
// where that leaves room for as many CTAs (else they are read again wherever they are needed).
// T: threads, 256 or, where there are fewer units than SMs, 1024.
template <bool KEYS, int D, int T>
__global__ void __launch_bounds__(T, 1024 / T)
k_evict(const Pool p, const EvictArgs a) {
  constexpr int kThreads = T, kWarps = T / 32;
  extern __shared__ uint32_t s_dyn[];
  __shared__ unsigned s_count[256];
  __shared__ int s_warp[kWarps];
  __shared__ int s_top;
  __shared__ unsigned s_key, s_want;
  __shared__ unsigned long long s_min[2][kWarps];
  __shared__ int s_gone[kFew];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t unit = blockIdx.x;
  const int h = static_cast<int>(unit % p.Hkv), b = static_cast<int>(unit / p.Hkv % a.B), l = static_cast<int>(unit / p.Hkv / a.B);
  const int seq = a.per_layer ? l * a.B + b : b;
  const int n = a.len[seq], budget = a.keep[seq], first = a.first ? a.first[b] : 0;
  int flag = 0;
  if (n < 0 || budget < 0 || first < 0) flag = CONFKV_FLAG_BAD_INDEX;
  if (n > a.cap || n > static_cast<long long>(a.max_blocks) << p.ps_shift) flag |= CONFKV_FLAG_CAPACITY;
  const int N = flag ? n : budget < n ? budget : n, gone = n - N;
  if (tid == 0) {
    if (flag) atomicOr(p.err, flag);
    if (h == 0 && (a.per_layer || l == 0)) a.new_len[seq] = N;
    s_top = INT32_MIN;
  }
  if (flag) {                           // such a sequence stays as it is, its masses in the outputs too
    if (a.mass_out != a.mass) pass_on(a.mass + unit * a.cap, a.pos + unit * a.cap, a.mass_out + unit * a.cap, a.pos_out + unit * a.cap, min(n, a.cap));
    return;
  }
  const float* mass = a.mass + unit * a.cap;
  const int32_t* pos = a.pos + unit * a.cap;
  float* mass_out = a.mass_out + unit * a.cap;
  int32_t* pos_out = a.pos_out + unit * a.cap;
  const bool copy = mass_out != mass;
  const int32_t* table = a.table + static_cast<size_t>(b) * a.max_blocks;
  const int layer = l * p.NP;           // (rows of a pool stay below 2^31)
  constexpr int LR = D / 8;             // lanes of a row, K's and then V's
  const int half = lane % (2 * LR) < LR ? 0 : 1, ch = lane % LR * 8;
  uint16_t* pool = half ? p.v : p.k;
  auto row_of = [&](int page, int j) { return (((layer + page) * p.Hkv + h) << p.ps_shift) + (j & (p.ps - 1)); };
  uint32_t* s_keys = s_dyn;
  const bool with_pos = KEYS && a.cap <= kPosShared;
  int* s_pos = reinterpret_cast<int*>(s_dyn + a.cap);

  // Few evicted places: a warp takes each place from N on, whose rows may have to move, and fetches them while
  // the keys come.
  const bool few = gone <= kFew;
  uint4 row = {};
  float row_mass = 0.0f;
  int row_pos = 0, row_page = 0;
  if (few && warp < gone && N > 0) {
    const int j = N + warp;
    row_page = table[j >> p.ps_shift];
    row_mass = mass[j];
    row_pos = pos[j];
    if (row_page >= 0 && row_page < p.NP && lane < 2 * LR)
      row = *reinterpret_cast<const uint4*>(pool + static_cast<size_t>(row_of(row_page, j)) * D + ch);
  }
  // masses and positions once: the kept part's copy, the newest position, keys without classes
  int top = INT32_MIN;
  for (int j0 = tid; j0 < n; j0 += kU * kThreads) {
    float x[kU];
    int y[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int j = j0 + u * kThreads;
      if (j < n) {
        x[u] = mass[j];
        y[u] = pos[j];
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int j = j0 + u * kThreads;
      if (j < n) {
        top = max(top, y[u]);
        if (KEYS) {
          s_keys[j] = order_of(x[u]);
          if (with_pos) s_pos[j] = y[u];
        }
        if (copy && j < N) {
          mass_out[j] = x[u];
          pos_out[j] = y[u];
        }
      }
    }
  }
  if (gone == 0 || N == 0) return;
  top = __reduce_max_sync(0xffffffffu, top);
  __syncthreads();
  if (lane == 0) atomicMax(&s_top, top);
  __syncthreads();
  const long long edge = static_cast<long long>(s_top) - a.protect;     // positions above it are the newest
  auto fresh_key = [&](int j) {
    return j < first ? kFirst : (with_pos ? s_pos[j] : pos[j]) > edge ? kNewest : KEYS ? s_keys[j] : order_of(mass[j]);
  };
  if (few) {
    // rounds of a minimum over (key, last place first), each thread's own beforehand
    auto least = [&](int skip) {        // of the thread's places but those that have gone in rounds before `skip`
      unsigned long long m = ~0ull;
      for (int j = tid; j < n; j += kThreads) {
        bool out = false;
        for (int i = 0; i < skip; ++i) out |= s_gone[i] == j;
        const unsigned long long x = static_cast<unsigned long long>(fresh_key(j)) << 32 | static_cast<unsigned>(INT32_MAX - j);
        if (!out && x < m) m = x;
      }
      return m;
    };
    unsigned long long mine = least(0);
    for (int i = 0; i < gone; ++i) {
      const unsigned hi = __reduce_min_sync(0xffffffffu, static_cast<unsigned>(mine >> 32));
      const unsigned lo = __reduce_min_sync(0xffffffffu, static_cast<unsigned>(mine >> 32) == hi ? static_cast<unsigned>(mine) : ~0u);
      if (lane == 0) s_min[i & 1][warp] = static_cast<unsigned long long>(hi) << 32 | lo;
      __syncthreads();
      unsigned long long m = s_min[i & 1][0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = min(m, s_min[i & 1][w]);
      if (m == mine) {                  // (one thread: places differ)
        s_gone[i] = INT32_MAX - static_cast<int>(static_cast<unsigned>(m));
        mine = i + 1 < gone ? least(i + 1) : ~0ull;
      }
    }
    __syncthreads();
    if (warp >= gone) return;
    // this warp's place from N on: kept, and the how manieth of those; the hole of that rank
    const int j = N + warp, g = lane < gone ? s_gone[lane] : INT32_MAX;
    if (__any_sync(0xffffffffu, g == j)) return;
    const int rank = warp - __popc(__ballot_sync(0xffffffffu, g >= N && g < j));
    int below = 0;
#pragma unroll
    for (int i = 0; i < kFew; ++i) below += __shfl_sync(0xffffffffu, g, i) < g;
    const unsigned at = __ballot_sync(0xffffffffu, g < N && below == rank);
    const int to = __shfl_sync(0xffffffffu, g, __ffs(at) - 1), page = table[to >> p.ps_shift];
    if (page < 0 || page >= p.NP || row_page < 0 || row_page >= p.NP) {
      if (lane == 0) atomicOr(p.err, CONFKV_FLAG_BAD_PAGE);
      return;
    }
    if (lane < 2 * LR)
      *reinterpret_cast<uint4*>(pool + static_cast<size_t>(row_of(page, to)) * D + ch) = row;
    if (lane == 0) {
      mass_out[to] = row_mass;
      pos_out[to] = row_pos;
    }
    return;
  }
  if (KEYS) {
#pragma unroll 8
    for (int j = tid; j < n; j += kThreads) {
      const bool newest = (with_pos ? s_pos[j] : pos[j]) > edge;
      if (j < first || newest) s_keys[j] = j < first ? kFirst : kNewest;
    }
    __syncthreads();
  }
  auto key = [&](int j) { return KEYS ? s_keys[j] : fresh_key(j); };
  // what stays, a bit for each place, by the N-th largest key, found byte by byte: of the keys equal to it the first
  // `want` stay
  const int words = (n + 31) >> 5;
  uint32_t* s_kept = s_dyn + (KEYS ? (with_pos ? 2 : 1) * a.cap : 2 * kList);   // [words]
  int* s_before = reinterpret_cast<int*>(s_kept + ((a.cap + 31) >> 5));         // [words + 1]: as below
  // (each thread takes a run of words, so that its sums go on from word to word)
  const int per = (words + kThreads - 1) / kThreads, w_lo = min(words, tid * per), w_hi = min(words, w_lo + per);
  int all;
  unsigned prefix = 0, want = N;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) s_count[tid] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kThreads) {
      const unsigned k = key(j);
      if (shift == 24 || k >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&s_count[k >> shift & 255u], 1u);
    }
    __syncthreads();
    // thread t: byte 255 - t, the keys above it
    int all;
    const unsigned mine = tid < 256 ? s_count[255 - tid] : 0u;
    const unsigned above = scan<kWarps>(static_cast<int>(mine), s_warp, all);
    if (tid < 256 && above < want && want <= above + mine) {
      s_key = prefix | static_cast<unsigned>(255 - tid) << shift;
      s_want = want - above;
    }
    __syncthreads();
    prefix = s_key;
    want = s_want;
  }
  for (int w0 = 0; w0 < words; w0 += kWarps) {
    const int j = 32 * (w0 + warp) + lane;
    const unsigned k = j < n ? key(j) : 0u;
    const unsigned more = __ballot_sync(0xffffffffu, j < n && k > prefix), same = __ballot_sync(0xffffffffu, j < n && k == prefix);
    if (lane == 0 && w0 + warp < words) {
      s_kept[w0 + warp] = more;
      s_before[w0 + warp] = static_cast<int>(same);
    }
  }
  __syncthreads();
  int equal = 0;
  for (int w = w_lo; w < w_hi; ++w) equal += __popc(s_before[w]);
  int eq = scan<kWarps>(equal, s_warp, all);
  for (int w = w_lo; w < w_hi; ++w) {
    unsigned same = s_before[w];
    const int left = static_cast<int>(want) - eq, here = __popc(same);
    eq += here;
    if (left < here) same = left <= 0 ? 0u : same & ((2u << __fns(same, 0, left)) - 1u);
    s_kept[w] |= same;
  }
  const int wn = N >> 5;                // holds the last holes' places and the first movers'
  const uint32_t low = (1u << (N & 31)) - 1u, tail = n & 31 ? (1u << (n & 31)) - 1u : 0xffffffffu;
  auto hole_word = [&](int w) { return ~s_kept[w] & (w < wn ? 0xffffffffu : w == wn ? low : 0u); };
  auto mover_word = [&](int w) { return s_kept[w] & (w > wn ? 0xffffffffu : w == wn ? ~low : 0u) & (w == words - 1 ? tail : 0xffffffffu); };
  int holes = 0, movers = 0;
  for (int w = w_lo; w < w_hi; ++w) {
    holes += __popc(hole_word(w));
    movers += __popc(mover_word(w));
  }
  int moves;
  holes = scan<kWarps>(holes, s_warp, all);
  movers = scan<kWarps>(movers, s_warp, moves);
  __syncthreads();                      // s_before's bits have been read
  // holes in the words before a word up to N's; from N's on, one place further, movers in those before
  for (int w = w_lo; w < w_hi; ++w) {
    if (w <= wn) s_before[w] = holes;
    holes += __popc(hole_word(w));
    if (w >= wn) s_before[w + 1] = movers;
    movers += __popc(mover_word(w));
  }
  // The moves' places, as many as the lists hold at a time (all, where the keys were in shared memory: they make
  // room, and there are no more moves than half the places), then the moves: a lane works one out, the warp copies its rows.
  int* s_to = reinterpret_cast<int*>(s_dyn);
  const int room = KEYS ? a.cap >> 1 : kList;
  int* s_from = s_to + room;
  constexpr int PER = 32 / (2 * LR);    // moves of a warp at once, K and V
  constexpr int kM = 8;                 // and so many in flight
  for (int c0 = 0; c0 < moves; c0 += room) {
    __syncthreads();
    for (int w = warp; w < words; w += kWarps) {
      const uint32_t hole = hole_word(w), mover = mover_word(w), lower = (1u << lane) - 1u;
      if (hole >> lane & 1u) {
        const int r = s_before[w] + __popc(hole & lower) - c0;
        if (r >= 0 && r < room) s_to[r] = 32 * w + lane;
      }
      if (mover >> lane & 1u) {
        const int r = s_before[w + 1] + __popc(mover & lower) - c0;
        if (r >= 0 && r < room) s_from[r] = 32 * w + lane;
      }
    }
    __syncthreads();
    const int here = min(room, moves - c0);
    for (int r0 = 32 * warp; r0 < here; r0 += kThreads) {
      int from = -1, to = -1;           // rows of the pool
      if (r0 + lane < here) {
        const int jt = s_to[r0 + lane], jf = s_from[r0 + lane];
        const int pt = table[jt >> p.ps_shift], pf = table[jf >> p.ps_shift];
        if (pt < 0 || pt >= p.NP || pf < 0 || pf >= p.NP) {
          flag = CONFKV_FLAG_BAD_PAGE;
        } else {
          to = row_of(pt, jt);
          from = row_of(pf, jf);
          mass_out[jt] = mass[jf];
          pos_out[jt] = pos[jf];
        }
      }
      const int live = min(32, here - r0), slot = lane / (2 * LR);
      for (int i0 = 0; i0 < live; i0 += PER * kM) {
        uint4 v[kM];
        int t[kM];
#pragma unroll
        for (int u = 0; u < kM; ++u) {
          const int i = i0 + u * PER + slot;
          const int f = __shfl_sync(0xffffffffu, from, i & 31);
          t[u] = __shfl_sync(0xffffffffu, to, i & 31);
          if (i >= live || f < 0) t[u] = -1;
          else v[u] = *reinterpret_cast<const uint4*>(pool + static_cast<size_t>(f) * D + ch);
        }
#pragma unroll
        for (int u = 0; u < kM; ++u)
          if (t[u] >= 0) *reinterpret_cast<uint4*>(pool + static_cast<size_t>(t[u]) * D + ch) = v[u];
      }
    }
  }
  if (flag) atomicOr(p.err, flag);
}

size_t shared_bytes(int cap, bool keys) {
  return (2 * static_cast<size_t>((cap + 31) >> 5) + 1 + (!keys ? 2 * kList : cap <= kPosShared ? 2 * cap : cap)) * 4;
}
template <typename F>
cudaError_t each_evict(F&& f) {
  cudaError_t e = cudaSuccess;
  auto of = [&](auto d, auto t) {
    constexpr int D = decltype(d)::value, T = decltype(t)::value;
    if (e == cudaSuccess) e = f(k_evict<true, D, T>, true, D, T);
    if (e == cudaSuccess) e = f(k_evict<false, D, T>, false, D, T);
  };
  using std::integral_constant;
  of(integral_constant<int, 64>{}, integral_constant<int, 256>{});
  of(integral_constant<int, 128>{}, integral_constant<int, 256>{});
  of(integral_constant<int, 64>{}, integral_constant<int, 1024>{});
  of(integral_constant<int, 128>{}, integral_constant<int, 1024>{});
  return e;
}

}  // namespace

cudaError_t setup_evict() {
  return each_evict([](auto kernel, bool keys, int, int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(shared_bytes(keys ? kKeysShared : kMaxEvictTokens, keys)));
  });
}

cudaError_t launch_evict(const Pool& p, const EvictArgs& a, int sms, cudaStream_t s) {
  const bool in_shared = a.cap <= kKeysShared;
  const unsigned units = static_cast<unsigned>(p.L) * a.B * p.Hkv;
  const int threads = units <= static_cast<unsigned>(sms) && a.cap > kWide ? 1024 : 256;
  const cudaError_t e = each_evict([&](auto kernel, bool keys, int d, int t) {
    if (keys != in_shared || d != p.d || t != threads) return cudaSuccess;
    return launch_pdl(kernel, dim3(units), dim3(t), shared_bytes(a.cap, keys), s, p, a);
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
