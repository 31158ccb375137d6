// Moving rows within a paged cache: an accepted path of drafted tokens to its
// places (commit), and the part-filled last pages of reordered beams (fork),
// both in every layer at once.
//
// Both are copies, bound by the bytes read and written: nothing is computed
// but addresses, which are worked out once per CTA.  Fork of 8 x 4 beams' half
// pages in 64 layers (755 MB): 99 us, 7.6 TB/s (part of what is written stays in
// L2).  Commit of 9 rows of 32 sequences in 64 layers (82 MB): 17.2 us, 4.7 TB/s,
// with rows of 256 bytes scattered over the pools; 18.8 us with K and V in CTAs of
// their own, 16.9 with a thread's column in both, which takes 2.9 us instead of 2.6
// for one sequence of a small model.
#include "paged_internal.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 256;       // of fork
constexpr int kCommitThreads = 256; // 8 KV heads of 128 channels are 128 columns of K and of V
constexpr int kCommitBatch = 8;     // rows in flight per thread
constexpr int kMaxPath = 1024;      // path_cap limit (confkv_paged.h)

// One CTA: sequence blockIdx.x, layer blockIdx.y.  A thread owns a 16-byte
// column of one head of K or V and moves it along the whole path, several rows
// loaded before they are stored.  In place this is safe: the path rises,
// so path[j] >= j, and a row that is overwritten (place j) can only be the
// source of a move j' <= j, which has been loaded by then.
__global__ void __launch_bounds__(kCommitThreads)
k_commit(const Pool p, const CommitArgs a) {
  __shared__ int s_src[kMaxPath], s_dst[kMaxPath];   // row numbers in the layer's head 0: page * Hkv * ps + slot
  __shared__ int s_bad;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, tid = threadIdx.x;
  const int ctx = a.ctx[b];
  const int n = a.path_len[b];
  const int32_t* path = a.path + static_cast<size_t>(b) * a.cap;
  const int32_t* table = a.table + static_cast<size_t>(b) * a.max_blocks;
  // asked for before the length is known: a step less in the chain (19.3 -> 17.2 us)
  const int x0 = tid < a.cap ? path[tid] : 0, prev0 = tid && tid <= a.cap ? path[tid - 1] : -1;
  const bool sane = n >= 0 && n <= a.cap && ctx >= 0;
  if (tid == 0) s_bad = sane ? 0 : CONFKV_FLAG_BAD_INDEX;
  __syncthreads();
  if (sane) {
    for (int j = tid; j < n; j += kCommitThreads) {
      const int x = j == tid ? x0 : path[j];
      const int prev = j == tid ? prev0 : path[j - 1];
      if (x <= prev) {
        atomicOr(&s_bad, CONFKV_FLAG_BAD_INDEX);
        continue;
      }
      const long long from = static_cast<long long>(ctx) + x, to = static_cast<long long>(ctx) + j;
      if ((from >> p.ps_shift) >= a.max_blocks) {
        atomicOr(&s_bad, CONFKV_FLAG_CAPACITY);
        continue;
      }
      if (x == j) {
        s_src[j] = -1;
        continue;
      }
      const int pf = table[from >> p.ps_shift], pt = table[to >> p.ps_shift];
      if (pf < 0 || pf >= p.NP || pt < 0 || pt >= p.NP) {
        atomicOr(&s_bad, CONFKV_FLAG_BAD_PAGE);
        continue;
      }
      s_src[j] = pf * p.Hkv * p.ps + static_cast<int>(from & (p.ps - 1));
      s_dst[j] = pt * p.Hkv * p.ps + static_cast<int>(to & (p.ps - 1));
    }
  }
  __syncthreads();
  const int bad = s_bad;
  if (blockIdx.y == 0 && tid == 0) {
    a.new_len[b] = bad ? ctx : ctx + n;
    if (bad) atomicOr(p.err, bad);
  }
  if (bad) return;
  // the path rises, so once a row moves every later one does
  int first = 0;
  while (first < n && s_src[first] < 0) ++first;
  if (first == n) return;
  const int cols = p.Hkv * (p.d >> 3);
  const size_t layer = static_cast<size_t>(blockIdx.y) * p.NP * p.Hkv * p.ps * p.d;
  for (int c = tid; c < 2 * cols; c += kCommitThreads) {
    uint16_t* pool = c < cols ? p.k : p.v;
    const int y = c < cols ? c : c - cols;
    const int h = y / (p.d >> 3), x = y - h * (p.d >> 3);
    uint16_t* col = pool + layer + static_cast<size_t>(h) * p.ps * p.d + 8 * x;
    for (int j = first; j < n; j += kCommitBatch) {
      uint4 r[kCommitBatch];
#pragma unroll
      for (int i = 0; i < kCommitBatch; ++i)
        if (j + i < n) r[i] = *reinterpret_cast<const uint4*>(col + static_cast<size_t>(s_src[j + i]) * p.d);
#pragma unroll
      for (int i = 0; i < kCommitBatch; ++i)
        if (j + i < n) *reinterpret_cast<uint4*>(col + static_cast<size_t>(s_dst[j + i]) * p.d) = r[i];
    }
  }
}

// One CTA: beam row blockIdx.x, layer blockIdx.y / 2, K or V.  The CTA of the
// first layer's K also writes the row's table and length.
__global__ void __launch_bounds__(kThreads)
k_fork(const Pool p, const ForkArgs a) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, tid = threadIdx.x;
  int flag = 0;
  int par = a.parent[r];
  if (par < -1 || par >= a.beams) flag = CONFKV_FLAG_BAD_INDEX;
  const int src = (par < 0 || par >= a.beams) ? r : r / a.beams * a.beams + par;
  const int len = a.len_in[src];
  const bool fits = len >= 0 && static_cast<long long>(len) <= static_cast<long long>(a.max_blocks) * p.ps;
  if (!fits) flag |= len < 0 ? CONFKV_FLAG_BAD_INDEX : CONFKV_FLAG_CAPACITY;
  const int full = fits ? len >> p.ps_shift : 0, fill = fits ? len & (p.ps - 1) : 0;
  const int32_t* tin = a.table_in + static_cast<size_t>(src) * a.max_blocks;
  const int to = fill ? a.tail[r] : 0;
  const int from = fill ? tin[full] : 0;
  const bool pages = to >= 0 && to < p.NP && from >= 0 && from < p.NP;
  if (!pages) flag |= CONFKV_FLAG_BAD_PAGE;
  if (blockIdx.y == 0) {
    int32_t* tout = a.table_out + static_cast<size_t>(r) * a.max_blocks;
    for (int i = tid; i < full; i += kThreads) tout[i] = tin[i];
    if (tid == 0) {
      if (fill) tout[full] = to;
      a.len_out[r] = len;
      if (flag) atomicOr(p.err, flag);
    }
  }
  if (!fill || !pages || from == to) return;
  const size_t head = static_cast<size_t>(p.ps) * p.d;     // elements of a page of one head
  uint16_t* base = ((blockIdx.y & 1) ? p.v : p.k) + static_cast<size_t>(blockIdx.y >> 1) * p.NP * p.Hkv * head;
  const uint16_t* s = base + static_cast<size_t>(from) * p.Hkv * head;
  uint16_t* t = base + static_cast<size_t>(to) * p.Hkv * head;
  const int per = fill * (p.d >> 3);                        // 16-byte words of one head
  const int n = per * p.Hkv;
  constexpr int kU = 8;
  for (int i0 = tid; i0 < n; i0 += kThreads * kU) {
    uint4 x[kU];
    size_t o[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + u * kThreads;
      if (i < n) {
        const int h = i / per;
        o[u] = h * head + 8 * static_cast<size_t>(i - h * per);
        x[u] = *reinterpret_cast<const uint4*>(s + o[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (i0 + u * kThreads < n) *reinterpret_cast<uint4*>(t + o[u]) = x[u];
  }
}

}  // namespace

cudaError_t launch_commit(const Pool& p, const CommitArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(k_commit, dim3(a.B, p.L), dim3(kCommitThreads), 0, s, p, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_fork(const Pool& p, const ForkArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(k_fork, dim3(a.rows, 2 * p.L), dim3(kThreads), 0, s, p, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
