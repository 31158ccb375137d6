// Attention of new rows (single tokens, prompt chunks, trees of drafted
// tokens) over a paged cache.
//
// One warp per (row, query head): each lane scores one key of a 32-key block
// (fp32), the block joins the running softmax (maximum and sum in fp32), and
// the lanes then add up their channels of the visible V rows.  Keys that the
// row does not see are never read into the sums.
#include <cfloat>

#include "paged_internal.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kWarps = 4;
constexpr float kL2E = 1.4426950408889634f;

template <bool BF, int D>
__global__ void __launch_bounds__(kWarps * 32)
k_attend_rows(const Pool p, const AttendArgs a) {
  __shared__ float s_q[kWarps][D];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int row = static_cast<int>(item / p.Hq), hq = static_cast<int>(item - static_cast<long long>(row) * p.Hq);
  if (row >= a.rows) return;
  const int b = sequence_of(a.bt.q_start, a.bt.B, row);
  if (b >= a.bt.B) return;
  const int first = a.bt.q_start[b], last = a.bt.q_start[b + 1];
  if (row < first) return;
  int ctx = a.bt.ctx[b];
  if (ctx < 0) {
    if (lane == 0) atomicOr(p.err, CONFKV_FLAG_BAD_INDEX);
    ctx = 0;
  }
  const int t = row - first;
  long long len = static_cast<long long>(ctx) + (last - first);
  const long long cap = static_cast<long long>(a.bt.max_blocks) * p.ps;
  if (len > cap) {
    if (lane == 0) atomicOr(p.err, CONFKV_FLAG_CAPACITY);
    len = cap;
  }
  const uint16_t* q = a.q + row * a.qs + hq * D;
  constexpr int C = D / 32;
  for (int i = lane; i < D; i += 32) s_q[warp][i] = to_f(q[i], BF) * a.scale;
  __syncwarp();
  const int h = hq / p.g;
  float m = -INFINITY, l = 0.0f, acc[C] = {};
  for (long long base = 0; base < len; base += 32) {
    const long long j = base + lane;
    bool seen = j < len;
    const uint16_t* kr = nullptr;
    const uint16_t* vr = nullptr;
    if (seen && j >= ctx) {
      const int x = static_cast<int>(j - ctx);
      if (a.bt.mask)
        seen = x < 32 * a.bt.mask_words &&
               ((a.bt.mask[static_cast<size_t>(row) * a.bt.mask_words + (x >> 5)] >> (x & 31)) & 1u);
      else
        seen = x <= t;
    }
    if (seen) {
      const int page = a.bt.table[static_cast<size_t>(b) * a.bt.max_blocks + (j >> p.ps_shift)];
      if (page < 0 || page >= p.NP) {
        atomicOr(p.err, CONFKV_FLAG_BAD_PAGE);
        seen = false;
      } else {
        const size_t off = (((static_cast<size_t>(a.layer) * p.NP + page) * p.Hkv + h) * p.ps + (j & (p.ps - 1))) * D;
        kr = p.k + off;
        vr = p.v + off;
      }
    }
    float s = -INFINITY;
    if (seen) {
      s = 0.0f;
#pragma unroll 4
      for (int i = 0; i < D; i += 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(kr + i);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = unpack2<BF>(ww[e]);
          s = fmaf(x.x, s_q[warp][i + 2 * e], s);
          s = fmaf(x.y, s_q[warp][i + 2 * e + 1], s);
        }
      }
    }
    float bm = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
    const float mn = fmaxf(m, bm);
    if (mn == -INFINITY) continue;
    const float f = m == -INFINITY ? 0.0f : exp2f((m - mn) * kL2E);
    const float pr = s == -INFINITY ? 0.0f : exp2f((s - mn) * kL2E);
    m = mn;
    float ps = pr;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
    l = l * f + ps;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] *= f;
    for (int jj = 0; jj < 32; ++jj) {
      const float w = __shfl_sync(0xffffffffu, pr, jj);
      const uint16_t* r = reinterpret_cast<const uint16_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vr), jj));
      if (!r) continue;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = fmaf(w, to_f(r[lane * C + c], BF), acc[c]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  uint16_t* out = a.out + (static_cast<size_t>(row) * p.Hq + hq) * D + lane * C;
#pragma unroll
  for (int c = 0; c < C; c += 2) *reinterpret_cast<uint32_t*>(out + c) = pack2<BF>(acc[c] * inv, acc[c + 1] * inv);
  if (a.lse && lane == 0) a.lse[static_cast<size_t>(row) * p.Hq + hq] = m + logf(l);
}

}  // namespace

cudaError_t launch_attend(const Pool& p, const AttendArgs& a, cudaStream_t s) {
  const long long items = static_cast<long long>(a.rows) * p.Hq;
  const dim3 grid(static_cast<unsigned>((items + kWarps - 1) / kWarps)), block(kWarps * 32);
  cudaError_t e;
  if (p.bf16)
    e = launch_pdl(p.d == 128 ? k_attend_rows<true, 128> : k_attend_rows<true, 64>, grid, block, 0, s, p, a);
  else
    e = launch_pdl(p.d == 128 ? k_attend_rows<false, 128> : k_attend_rows<false, 64>, grid, block, 0, s, p, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
