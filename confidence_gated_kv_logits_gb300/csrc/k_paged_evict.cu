// Eviction from a paged cache: each KV head of each sequence and layer keeps N of
// its n tokens; those behind the budget move into the places of evicted ones.
//
// Order: the sequence's first places, then its newest positions, then the larger
// mass; equal ones by the lower place.  Classes and masses are one 32-bit key
// (masses in an order-preserving form); the N-th largest key is found by four
// rounds of counting one byte each, and of the keys equal to it the lowest places
// stay.  Evicted places below N (holes) and kept places from N on (movers) are
// equally many; the r-th hole takes the r-th mover's rows, which no other move
// reads or writes, so all moves are independent.
#include "paged_internal.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kU = 8;                   // loads of a thread in flight
constexpr uint32_t kFirst = 0xffffffffu, kNewest = 0xfffffffeu;
constexpr int kKeysShared = 40960;      // keys up to here stay in shared memory

// A mass as an unsigned number in the same order; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// What the threads before give, and the CTA's sum.
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

// The place of the r-th one among words [lo, hi) with `before` ones before each.
template <typename Word>
__device__ __forceinline__ int place_of(const int* before, int lo, int hi, int r, Word&& word) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= r) lo = mid;
    else hi = mid;
  }
  return 32 * lo + static_cast<int>(__fns(word(lo), 0, r - before[lo] + 1));
}

// One CTA: a KV head of a sequence in a layer.  KEYS: its keys lie in shared memory
// (else they are made again from mass and position wherever they are needed).
template <bool KEYS, int D>
__global__ void __launch_bounds__(kThreads)
k_evict(const Pool p, const EvictArgs a) {
  extern __shared__ uint32_t s_dyn[];
  __shared__ unsigned s_count[256];
  __shared__ int s_warp[kWarps];
  __shared__ int s_top;
  __shared__ unsigned s_key, s_want;
  const int words_cap = (a.cap + 31) >> 5;
  uint32_t* s_kept = s_dyn;                                   // [words]
  // [words + 1]: holes in the words before; from the word of place N on, one place further, movers
  int* s_before = reinterpret_cast<int*>(s_dyn + words_cap);
  uint32_t* s_keys = s_dyn + 2 * words_cap + 1;
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
  const int N = flag ? n : budget < n ? budget : n;
  if (tid == 0) {
    if (flag) atomicOr(p.err, flag);
    if (h == 0 && (a.per_layer || l == 0)) a.new_len[seq] = N;
    s_top = INT32_MIN;
  }
  if (flag) return;                     // such a sequence stays as it is
  const float* mass = a.mass + unit * a.cap;
  const int32_t* pos = a.pos + unit * a.cap;
  float* mass_out = a.mass_out + unit * a.cap;
  int32_t* pos_out = a.pos_out + unit * a.cap;
  const bool copy = mass_out != mass;
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
        if (KEYS) s_keys[j] = order_of(x[u]);
        if (copy && j < N) {
          mass_out[j] = x[u];
          pos_out[j] = y[u];
        }
      }
    }
  }
  if (N == n || N == 0) return;
  top = __reduce_max_sync(0xffffffffu, top);
  __syncthreads();
  if (lane == 0) atomicMax(&s_top, top);
  __syncthreads();
  const long long edge = static_cast<long long>(s_top) - a.protect;     // positions above it are the newest
  auto fresh_key = [&](int j) {
    return j < first ? kFirst : pos[j] > edge ? kNewest : KEYS ? s_keys[j] : order_of(mass[j]);
  };
  if (KEYS) {
    for (int j = tid; j < n; j += kThreads) s_keys[j] = fresh_key(j);
    __syncthreads();
  }
  auto key = [&](int j) { return KEYS ? s_keys[j] : fresh_key(j); };
  // the N-th largest key, byte by byte
  unsigned prefix = 0, want = N;
  for (int shift = 24; shift >= 0; shift -= 8) {
    s_count[tid] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kThreads) {
      const unsigned k = key(j);
      if (shift == 24 || k >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&s_count[k >> shift & 255u], 1u);
    }
    __syncthreads();
    // thread t: byte 255 - t, the keys above it
    int all;
    const unsigned mine = s_count[255 - tid];
    const unsigned above = scan(static_cast<int>(mine), s_warp, all);
    if (above < want && want <= above + mine) {
      s_key = prefix | static_cast<unsigned>(255 - tid) << shift;
      s_want = want - above;
    }
    __syncthreads();
    prefix = s_key;
    want = s_want;
  }
  // what stays, a bit for each place; of the keys equal to the N-th the first `want`
  const int words = (n + 31) >> 5;
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
  // (each thread takes a run of words, so that its sums go on from word to word)
  const int per = (words + kThreads - 1) / kThreads, w_lo = min(words, tid * per), w_hi = min(words, w_lo + per);
  int all, equal = 0;
  for (int w = w_lo; w < w_hi; ++w) equal += __popc(s_before[w]);
  int eq = scan(equal, s_warp, all);
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
  holes = scan(holes, s_warp, all);
  movers = scan(movers, s_warp, moves);
  __syncthreads();                      // s_before's bits have been read
  for (int w = w_lo; w < w_hi; ++w) {
    if (w <= wn) s_before[w] = holes;
    holes += __popc(hole_word(w));
    if (w >= wn) s_before[w + 1] = movers;
    movers += __popc(mover_word(w));
  }
  __syncthreads();
  // the moves: a lane finds one, the warp copies its rows
  const int32_t* table = a.table + static_cast<size_t>(b) * a.max_blocks;
  const size_t layer = static_cast<size_t>(l) * p.NP;
  constexpr int LR = D / 8;             // lanes of a row
  constexpr int PER = 32 / (2 * LR);    // moves of a warp at once, K and V
  constexpr int kM = 8;                 // and so many in flight
  flag = 0;
  for (int r0 = 32 * warp; r0 < moves; r0 += kThreads) {
    long long from = -1, to = -1;       // rows in head h's pool
    if (r0 + lane < moves) {
      const int jt = place_of(s_before, 0, wn + 1, r0 + lane, hole_word);
      const int jf = place_of(s_before + 1, wn, words, r0 + lane, mover_word);
      const int pt = table[jt >> p.ps_shift], pf = table[jf >> p.ps_shift];
      if (pt < 0 || pt >= p.NP || pf < 0 || pf >= p.NP) {
        flag = CONFKV_FLAG_BAD_PAGE;
      } else {
        to = ((layer + pt) * p.Hkv + h) * p.ps + (jt & (p.ps - 1));
        from = ((layer + pf) * p.Hkv + h) * p.ps + (jf & (p.ps - 1));
        mass_out[jt] = mass[jf];
        pos_out[jt] = pos[jf];
      }
    }
    const int live = min(32, moves - r0);
    const int slot = lane / (2 * LR), x = lane % (2 * LR);
    uint16_t* pool = x < LR ? p.k : p.v;
    const int ch = (x % LR) * 8;
    for (int i0 = 0; i0 < live; i0 += PER * kM) {
      uint4 v[kM];
      long long t[kM];
#pragma unroll
      for (int u = 0; u < kM; ++u) {
        const int i = i0 + u * PER + slot;
        const long long f = __shfl_sync(0xffffffffu, from, i & 31);
        t[u] = __shfl_sync(0xffffffffu, to, i & 31);
        if (i >= live || f < 0) t[u] = -1;
        else v[u] = *reinterpret_cast<const uint4*>(pool + f * D + ch);
      }
#pragma unroll
      for (int u = 0; u < kM; ++u)
        if (t[u] >= 0) *reinterpret_cast<uint4*>(pool + t[u] * D + ch) = v[u];
    }
  }
  if (flag) atomicOr(p.err, flag);
}

size_t shared_bytes(int cap, bool keys) {
  return (2 * static_cast<size_t>((cap + 31) >> 5) + 1 + (keys ? cap : 0)) * 4;
}
template <typename F>
cudaError_t each_evict(F&& f) {
  cudaError_t e = f(k_evict<true, 64>, true, 64);
  if (e == cudaSuccess) e = f(k_evict<true, 128>, true, 128);
  if (e == cudaSuccess) e = f(k_evict<false, 64>, false, 64);
  return e == cudaSuccess ? f(k_evict<false, 128>, false, 128) : e;
}

}  // namespace

cudaError_t setup_evict() {
  return each_evict([](auto kernel, bool keys, int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(shared_bytes(keys ? kKeysShared : kMaxEvictTokens, keys)));
  });
}

cudaError_t launch_evict(const Pool& p, const EvictArgs& a, cudaStream_t s) {
  const bool in_shared = a.cap <= kKeysShared;
  const cudaError_t e = each_evict([&](auto kernel, bool keys, int d) {
    if (keys != in_shared || d != p.d) return cudaSuccess;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(p.L) * a.B * p.Hkv), dim3(kThreads), shared_bytes(a.cap, keys), s, p, a);
  });
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
