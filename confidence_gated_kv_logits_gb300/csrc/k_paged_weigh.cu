// Accumulated attention weight of each cached token and KV head:
//
//   mass_out_t = decay mass_t + gain sum_r exp(scale q_r k_t - lse_r)
//
// over the rows r (new tokens x the group's query heads) that see token t, with
// the rows' lse as attend gave it: the weights are final at once, nothing is
// rescaled, and each token's sum is one thread's, in one order.
#include "paged_attend.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 128;
constexpr float kL2E = 1.4426950408889634f;

// A CTA takes 128 tokens of one KV head of one sequence at a time, a thread each.
template <bool BF, int D>
__global__ void __launch_bounds__(kThreads)
k_weigh(const Pool p, const WeighArgs a) {
  __shared__ float s_q[D];
  pdl_wait();
  pdl_trigger();
  Walk<128, 128, 0> w(p, a.bt, a.rows);
  for (int b = blockIdx.z; b < a.bt.B; b += gridDim.z) {
    int flag = 0;
    w.sequence(b, flag);
    const int h = blockIdx.y, j = blockIdx.x * kThreads + threadIdx.x;
    if (flag && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) atomicOr(p.err, flag);
    if (w.T <= 0 || static_cast<int>(blockIdx.x * kThreads) >= w.len) continue;
    const bool live = j < w.len;
    const int32_t* table = a.bt.table + static_cast<size_t>(w.b) * a.bt.max_blocks;
    const int page = live ? table[j >> p.ps_shift] : 0;
    const bool none = page < 0 || page >= p.NP;
    float k[D], sum = 0.0f;
    const uint16_t* src = p.k + (((static_cast<size_t>(a.layer) * p.NP + (none ? 0 : page)) * p.Hkv + h) * p.ps + (j & (p.ps - 1))) * D;
#pragma unroll
    for (int i = 0; i < D; ++i) k[i] = live ? none ? NAN : to_f(src[i], BF) : 0.0f;
    for (int r = 0; r < w.T * p.g; ++r) {
      const int t = r / p.g, hq = h * p.g + r - t * p.g;
      const size_t row = w.row0 + t;
      __syncthreads();
      for (int i = threadIdx.x; i < D; i += kThreads) s_q[i] = to_f(a.q[row * a.qs + hq * D + i], BF);
      __syncthreads();
      if (!live || !(seen_bits(a.bt, row, t, w.ctx, w.len, j) & 1u)) continue;
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < D; ++i) z = fmaf(k[i], s_q[i], z);
      const float lse = a.lse[row * p.Hq + hq];
      if (lse != -INFINITY) sum += exp2f((z * a.scale - lse) * kL2E);
    }
    if (!live) continue;
    if (j >= a.cap) {
      atomicOr(p.err, CONFKV_FLAG_CAPACITY);
      continue;
    }
    const size_t at = (static_cast<size_t>(w.b) * p.Hkv + h) * a.cap + j;
    if (none) atomicOr(p.err, CONFKV_FLAG_BAD_PAGE);
    a.mass_out[at] = (j < w.ctx ? a.decay * a.mass[at] : 0.0f) + a.gain * sum;
    if (j >= w.ctx && a.pos) a.pos[at] = a.positions ? a.positions[w.row0 + j - w.ctx] : j;
  }
}

}  // namespace

cudaError_t launch_weigh(const Pool& p, const WeighArgs& a, cudaStream_t s) {
  const long long tokens = static_cast<long long>(a.bt.max_blocks) * p.ps;
  const dim3 grid(static_cast<unsigned>((tokens + kThreads - 1) / kThreads), p.Hkv, a.bt.B < 65535 ? a.bt.B : 65535);
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) { e = launch_pdl(kernel, grid, dim3(kThreads), 0, s, p, a); };
  if (p.bf16) p.d == 128 ? go(k_weigh<true, 128>) : go(k_weigh<true, 64>);
  else p.d == 128 ? go(k_weigh<false, 128>) : go(k_weigh<false, 64>);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
