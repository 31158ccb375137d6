// Appending new rows' K and V to a paged cache, K (and Q) rotated by their
// positions on the way.
//
// Channel pair i of the first `rot` channels turns by the angle pos * f_i:
//   (a, b) -> (a cos - b sin, b cos + a sin).
// In whole turns the angle is pos * f_i / 2 pi, of which only the fraction
// counts.  That fraction is kept in 64-bit fixed point: F_i = frac(f_i / 2 pi)
// * 2^64 from one double product, and the wrapped 64-bit product pos * F_i,
// so the reduction is exact for every position (F_i itself is good to 2^-53
// relative); sincospi then sees an fp32 fraction in [-1, 1).  A double-
// precision sincos per angle would keep GB300's slow FP64 pipe busy for longer
// than the memory.
//
// The work is traffic: each row is read once and written once, 16 bytes per
// access.  One CTA takes `tpc` rows (4 where there are enough to fill the
// GPU, else 1), computes their rot / 2 sines once into shared memory for all
// heads, and then moves (row, head, 8-channel chunk) items, a rotated item
// being the two chunks of eight pairs.
#include "paged_internal.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTpc = 4;

template <bool BF>
__device__ __forceinline__ void rotate8(uint4& lo, uint4& hi, const float2* cs, bool interleaved) {
  // half-split: lo = channels c .. c+7, hi = their partners, cs[0..7]
  // interleaved: lo, hi = 16 channels in order = pairs 0..7
  uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
  uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? a[i] : b[i - 4];
      const float2 x = unpack2<BF>(w);
      const float2 t = cs[i];
      w = pack2<BF>(x.x * t.x - x.y * t.y, x.y * t.x + x.x * t.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2<BF>(a[i]), y = unpack2<BF>(b[i]);
      const float2 t = cs[2 * i], u = cs[2 * i + 1];
      a[i] = pack2<BF>(x.x * t.x - y.x * t.y, x.y * u.x - y.y * u.y);
      b[i] = pack2<BF>(y.x * t.x + x.x * t.y, y.y * u.x + x.y * u.y);
    }
  }
}

template <bool BF>
__global__ void __launch_bounds__(kThreads)
k_append(const Pool p, const AppendArgs a, int tpc) {
  __shared__ float2 s_cs[kMaxTpc * 64];      // (cos, sin) per row and pair
  __shared__ long long s_row[kMaxTpc];       // element offset of (layer, page, head 0, slot), -1: no store
  __shared__ int s_pos[kMaxTpc];             // position
  __shared__ int s_live[kMaxTpc];            // the row belongs to a sequence
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = blockIdx.x * tpc;
  if (warp < tpc) {
    const int row = row0 + warp;
    int b = a.bt.B;
    if (row < a.rows) b = sequence_of(a.bt.q_start, a.bt.B, row);
    if (lane == 0) {
      long long off = -1;
      int pos = 0, live = 0;
      if (b < a.bt.B) {
        const int first = a.bt.q_start[b], ctx = a.bt.ctx[b];
        if (row >= first) {
          live = 1;
          const long long place = static_cast<long long>(ctx) + (row - first);
          pos = a.pos ? a.pos[row] : static_cast<int>(place);
          const long long blk = place >> p.ps_shift;
          if (ctx < 0) {
            atomicOr(p.err, CONFKV_FLAG_BAD_INDEX);
          } else if (blk >= a.bt.max_blocks) {
            atomicOr(p.err, CONFKV_FLAG_CAPACITY);
          } else {
            const int page = a.bt.table[static_cast<size_t>(b) * a.bt.max_blocks + blk];
            if (page < 0 || page >= p.NP) {
              atomicOr(p.err, CONFKV_FLAG_BAD_PAGE);
            } else {
              const int slot = static_cast<int>(place & (p.ps - 1));
              off = ((static_cast<long long>(a.layer) * p.NP + page) * p.Hkv * p.ps + slot) * p.d;
            }
          }
        }
      }
      s_row[warp] = off;
      s_pos[warp] = pos;
      s_live[warp] = live;
    }
  }
  __syncthreads();
  const int half = a.rot >> 1;
  for (int i = tid; i < tpc * half; i += kThreads) {
    const int t = i / half, c = i - t * half;
    double turns = static_cast<double>(a.inv_freq[c]) * 0.15915494309189535;   // 1 / (2 pi)
    turns -= floor(turns);
    const unsigned long long F = static_cast<unsigned long long>(turns * 18446744073709551616.0);
    const unsigned long long ang = static_cast<unsigned long long>(static_cast<long long>(s_pos[t])) * F;
    const int h = static_cast<int>((ang + 0x80000000ull) >> 32);   // fraction of a half turn, 2^-31 units
    float sn, cn;
    sincospif(static_cast<float>(h) * 4.656612873077393e-10f, &sn, &cn);
    s_cs[t * 64 + c] = make_float2(cn, sn);
  }
  __syncthreads();

  // items of one row: rotated chunks of the q and k heads (two 16-byte
  // accesses each), then their other channels, then v (one access each)
  const int rc = a.rot >> 4;                       // rotated items per head
  const int pc = (p.d - a.rot) >> 3;               // plain items per head
  const int heads = (a.q ? p.Hq : 0) + p.Hkv;
  const int nrot = heads * rc, npl = heads * pc, nv = p.Hkv * (p.d >> 3);
  const int per_row = nrot + npl + nv;
  const int q0 = a.q ? p.Hq : 0;
  const long long hs = static_cast<long long>(p.ps) * p.d;   // head stride in a page
  for (int i = blockIdx.y * kThreads + tid; i < tpc * per_row; i += gridDim.y * kThreads) {
    const int t = i / per_row;
    int j = i - t * per_row;
    if (!s_live[t]) continue;
    const int row = row0 + t;
    const long long dst = s_row[t];
    if (j < nrot) {
      const int h = j / rc, c = j - h * rc;
      const int c0 = a.interleaved ? 16 * c : 8 * c;
      const int c1 = a.interleaved ? c0 + 8 : c0 + half;
      const uint16_t* src = h < q0 ? a.q + row * a.qs + h * p.d : a.k + row * a.ks + (h - q0) * p.d;
      uint16_t* out = h < q0 ? a.q_out + row * a.qos + h * p.d : p.k + dst + (h - q0) * hs;
      uint4 lo = *reinterpret_cast<const uint4*>(src + c0);
      uint4 hi = *reinterpret_cast<const uint4*>(src + c1);
      rotate8<BF>(lo, hi, s_cs + t * 64 + 8 * c, a.interleaved);
      if (h < q0 || dst >= 0) {
        *reinterpret_cast<uint4*>(out + c0) = lo;
        *reinterpret_cast<uint4*>(out + c1) = hi;
      }
    } else {
      j -= nrot;
      const uint16_t* src;
      uint16_t* out;
      bool st = dst >= 0;
      if (j < npl) {
        const int h = j / pc, c = a.rot + 8 * (j - h * pc);
        src = (h < q0 ? a.q + row * a.qs + h * p.d : a.k + row * a.ks + (h - q0) * p.d) + c;
        out = (h < q0 ? a.q_out + row * a.qos + h * p.d : p.k + dst + (h - q0) * hs) + c;
        st = st || h < q0;
      } else {
        j -= npl;
        const int h = j / (p.d >> 3), c = 8 * (j - h * (p.d >> 3));
        src = a.v + row * a.vs + h * p.d + c;
        out = p.v + dst + h * hs + c;
      }
      if (st) *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(src);
    }
  }
}

}  // namespace

cudaError_t launch_append(const Pool& p, const AppendArgs& a, cudaStream_t s) {
  const int tpc = a.rows >= 4 * 152 ? kMaxTpc : 1;
  const int heads = (a.q ? p.Hq : 0) + p.Hkv;
  const int items = tpc * (heads * ((a.rot >> 4) + ((p.d - a.rot) >> 3)) + p.Hkv * (p.d >> 3));
  const int gx = (a.rows + tpc - 1) / tpc;
  // few rows: their items over several CTAs, one item per thread
  const int split = gx >= 152 ? 1 : (items + kThreads - 1) / kThreads;
  const cudaError_t e = launch_pdl(p.bf16 ? k_append<true> : k_append<false>, dim3(gx, split),
                                   dim3(kThreads), 0, s, p, a, tpc);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
