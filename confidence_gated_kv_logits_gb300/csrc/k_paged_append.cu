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
// access, one CTA per row.  What a row costs besides is a chain of small reads
// (its sequence, length, page) before anything can be stored, so every thread
// asks for its part of the row first and the chain runs meanwhile, in the two
// warps that take the row's sines, which lie in shared memory as the lanes read
// them.  (4 prompts' chunks, 40 + 2 x 8 heads, d = 128, bf16, 116 MB, 17.1 us at
// the copy rate: 30.0 us with four rows per CTA and loads behind the chain, 25.8
// with one row and one item of a thread in flight, 22.0 with the sines read without
// bank conflicts and one barrier instead of two; then 22.8 with two items in
// flight and 5 CTAs per SM instead of 8, 23.5 with CTAs of 512 threads.  A row's
// chain, the turnover of CTAs and the issue slots bound it: these are used in 68% of
// the SMs' active cycles, which are 79% of the launch.)
#include "paged_internal.cuh"

namespace confkv {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kU = 1;             // items of a thread in flight (8 CTAs per SM hide more than 2 items in 5)

// Sines of a row: pairs 8c + 2i and 8c + 2i + 1 (cos, sin, cos, sin) at [i][c], so
// that a warp's lanes, which have neighbouring c, read whole lines.
constexpr int kChunks = 8;        // of 8 pairs: 64 pairs at most

template <bool BF>
__device__ __forceinline__ void rotate8(uint4& lo, uint4& hi, const float4* cs, bool interleaved) {
  // half-split: lo = channels c .. c+7, hi = their partners, cs: their pairs
  // interleaved: lo, hi = 16 channels in order = pairs 0..7
  uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
  uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = cs[i * kChunks];
      uint32_t& w0 = i < 2 ? a[2 * i] : b[2 * i - 4];
      uint32_t& w1 = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
      const float2 x = unpack2<BF>(w0), y = unpack2<BF>(w1);
      w0 = pack2<BF>(x.x * t.x - x.y * t.y, x.y * t.x + x.x * t.y);
      w1 = pack2<BF>(y.x * t.z - y.y * t.w, y.y * t.z + y.x * t.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = cs[i * kChunks];
      const float2 x = unpack2<BF>(a[i]), y = unpack2<BF>(b[i]);
      a[i] = pack2<BF>(x.x * t.x - y.x * t.y, x.y * t.z - y.y * t.w);
      b[i] = pack2<BF>(y.x * t.x + x.x * t.y, y.y * t.z + x.y * t.w);
    }
  }
}

// A row's items: first the rotated chunks of the q and k heads (two 16-byte
// accesses each), then those heads' other channels, then v (one access each).
struct Item {
  const uint16_t* src;
  int to;            // channel offset in q_out's row, or in the page of k or v: head * head stride + channel
  int second;        // channels from the first access to the second, 0: none
  int chunk;         // its 8 rotated pairs
  int dst;           // 0 q_out, 1 k, 2 v, -1 none
};

template <bool BF>
__global__ void __launch_bounds__(kThreads, 8)
k_append(const Pool p, const AppendArgs a) {
  __shared__ float4 s_cs[4 * kChunks];
  __shared__ long long s_row;      // element offset of (layer, page, head 0, slot), -1: no store
  __shared__ int s_live;           // the row belongs to a sequence
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5;
  const int row = blockIdx.x;
  const int half = a.rot >> 1, rc = a.rot >> 4, pc = (p.d - a.rot) >> 3, vc = p.d >> 3;
  const int q0 = a.q ? p.Hq : 0, heads = q0 + p.Hkv;
  const int nrot = heads * rc, nplain = heads * pc, items = nrot + nplain + p.Hkv * vc;
  const int hs = p.ps * p.d;       // head stride in a page
  auto item = [&](int j) {
    Item t{nullptr, 0, 0, 0, -1};
    if (j >= items) return t;
    int h, c;
    if (j < nrot) {
      h = j / rc;
      c = j - h * rc;
      t.chunk = c;
      t.second = a.interleaved ? 8 : half;
      c *= a.interleaved ? 16 : 8;
    } else if (j < nrot + nplain) {
      j -= nrot;
      h = j / pc;
      c = a.rot + 8 * (j - h * pc);
    } else {
      j -= nrot + nplain;
      h = j / vc;
      c = 8 * (j - h * vc);
      t.src = a.v + row * a.vs + h * p.d + c;
      t.to = h * hs + c;
      t.dst = 2;
      return t;
    }
    if (h < q0) {
      t.src = a.q + row * a.qs + h * p.d + c;
      t.to = h * p.d + c;
      t.dst = 0;
    } else {
      h -= q0;
      t.src = a.k + row * a.ks + h * p.d + c;
      t.to = h * hs + c;
      t.dst = 1;
    }
    return t;
  };
  for (int j0 = tid; j0 - tid < items; j0 += kU * kThreads) {
    Item t[kU];
    uint4 lo[kU], hi[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      t[u] = item(j0 + u * kThreads);
      if (t[u].dst >= 0) {
        lo[u] = *reinterpret_cast<const uint4*>(t[u].src);
        if (t[u].second) hi[u] = *reinterpret_cast<const uint4*>(t[u].src + t[u].second);
      }
    }
    if (j0 == tid) {               // the first time round: where the row goes, and its sines
      if (warp < 2) {              // (64 pairs at most; both find the row's place)
        unsigned long long F = 0;
        if (tid < half) {
          double turns = static_cast<double>(a.inv_freq[tid]) * 0.15915494309189535;   // 1 / (2 pi)
          turns -= floor(turns);
          F = static_cast<unsigned long long>(turns * 18446744073709551616.0);
        }
        const int given = a.pos ? a.pos[row] : 0;
        const int b = sequence_of(a.bt.q_start, a.bt.B, row);
        long long off = -1;
        int pos = given, live = 0;
        if (b < a.bt.B) {
          const int first = a.bt.q_start[b], ctx = a.bt.ctx[b];
          if (row >= first) {
            live = 1;
            const long long place = static_cast<long long>(ctx) + (row - first);
            if (!a.pos) pos = static_cast<int>(place);
            const long long blk = place >> p.ps_shift;
            int flag = 0;
            if (ctx < 0) {
              flag = CONFKV_FLAG_BAD_INDEX;
            } else if (blk >= a.bt.max_blocks) {
              flag = CONFKV_FLAG_CAPACITY;
            } else {
              const int page = a.bt.table[static_cast<size_t>(b) * a.bt.max_blocks + blk];
              if (page < 0 || page >= p.NP) flag = CONFKV_FLAG_BAD_PAGE;
              else off = ((static_cast<long long>(a.layer) * p.NP + page) * p.Hkv * p.ps + (place & (p.ps - 1))) * p.d;
            }
            if (flag && tid == 0) atomicOr(p.err, flag);
          }
        }
        if (tid == 0) {
          s_row = off;
          s_live = live;
        }
        if (tid < half) {
          const unsigned long long ang = static_cast<unsigned long long>(static_cast<long long>(pos)) * F;
          const int h = static_cast<int>((ang + 0x80000000ull) >> 32);   // fraction of a half turn, 2^-31 units
          float2 t;
          sincospif(static_cast<float>(h) * 4.656612873077393e-10f, &t.y, &t.x);
          reinterpret_cast<float2*>(s_cs)[(((tid & 7) >> 1) * kChunks + (tid >> 3)) * 2 + (tid & 1)] = t;
        }
      }
      __syncthreads();
      if (!s_live) return;
    }
    const long long at = s_row;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (t[u].dst < 0 || (t[u].dst > 0 && at < 0)) continue;
      uint16_t* out = t[u].dst == 0 ? a.q_out + row * a.qos : (t[u].dst == 1 ? p.k : p.v) + at;
      out += t[u].to;
      if (t[u].second) {
        rotate8<BF>(lo[u], hi[u], s_cs + t[u].chunk, a.interleaved);
        *reinterpret_cast<uint4*>(out + t[u].second) = hi[u];
      }
      *reinterpret_cast<uint4*>(out) = lo[u];
    }
  }
}

}  // namespace

cudaError_t launch_append(const Pool& p, const AppendArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(p.bf16 ? k_append<true> : k_append<false>, dim3(a.rows), dim3(kThreads), 0, s, p, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
