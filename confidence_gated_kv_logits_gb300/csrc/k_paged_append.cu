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
#include <type_traits>

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

// Where a row goes and its sines, by the CTA's first two warps (64 pairs at most;
// both find the row's place).  AXES: pair i turns by the row's position axis[i].
template <bool AXES>
__device__ __forceinline__ void place_row(const Pool& p, const AppendArgs& a, int row, int half, float4* s_cs,
                                          long long* s_row, int* s_live) {
  const int tid = threadIdx.x;
  unsigned long long F = 0;
  int axis = 0, flag = 0;
  if (tid < half) {
    if constexpr (AXES) axis = a.axis[tid];
    double turns = static_cast<double>(a.inv_freq[tid]) * 0.15915494309189535;   // 1 / (2 pi)
    turns -= floor(turns);
    F = static_cast<unsigned long long>(turns * 18446744073709551616.0);
  }
  int given = 0;
  if constexpr (AXES) {
    if (axis < 0 || axis >= a.axes) flag = CONFKV_FLAG_BAD_INDEX;      // (such a pair is not turned)
    else if (tid < half) given = a.pos[static_cast<size_t>(row) * a.axes + axis];
    flag = __any_sync(0xffffffffu, flag) ? CONFKV_FLAG_BAD_INDEX : 0;
  } else {
    given = a.pos ? a.pos[row] : 0;
  }
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
      if (ctx < 0) {
        flag |= CONFKV_FLAG_BAD_INDEX;
      } else if (blk >= a.bt.max_blocks) {
        flag |= CONFKV_FLAG_CAPACITY;
      } else {
        const int page = a.bt.table[static_cast<size_t>(b) * a.bt.max_blocks + blk];
        if (page < 0 || page >= p.NP) flag |= CONFKV_FLAG_BAD_PAGE;
        else off = ((static_cast<long long>(a.layer) * p.NP + page) * p.Hkv * p.ps + (place & (p.ps - 1))) * p.d;
      }
      if (flag && (tid & 31) == 0) atomicOr(p.err, flag);
    }
  }
  if (tid == 0) {
    *s_row = off;
    *s_live = live;
  }
  if (tid < half) {
    const unsigned long long ang = static_cast<unsigned long long>(static_cast<long long>(pos)) * F;
    const int h = static_cast<int>((ang + 0x80000000ull) >> 32);   // fraction of a half turn, 2^-31 units
    float2 t;
    sincospif(static_cast<float>(h) * 4.656612873077393e-10f, &t.y, &t.x);
    reinterpret_cast<float2*>(s_cs)[(((tid & 7) >> 1) * kChunks + (tid >> 3)) * 2 + (tid & 1)] = t;
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
      if (warp < 2) place_row<false>(p, a, row, half, s_cs, &s_row, &s_live);
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

// The same with each head of q and k normed on the way,
//   y_c = x_c w_c / sqrt(sum_c x_c^2 / d + eps),
// and with a position of its own for each channel pair (axis).  A head is d / 16
// neighbouring lanes with 16 channels each, both channels of its 8 pairs among them,
// so that the sum of squares is a few shuffles and the rotation needs none; x is
// read once, kept in fp32 through norm and rotation, and rounded once.  Squares of
// values from 2^59 on can leave fp32's range: such heads' sums are taken again
// with x 2^-100 (eps does not count there).
//
// 4 prompts' chunks, 40 + 2 x 8 heads of 128 channels, three axes, bf16, 116 MB: 28.5 us,
// 60% of the copy rate (append without norms 22.0).  Bound by issue slots (63% of active
// cycles used) and the row's chain before its barrier; without axis 30.6 (64 registers, 48 with it).  Slower: paired arithmetic (31.3),
// 40 registers for six CTAs per SM (29.4), CTAs that take row after row with the next
// one's place and sines found by two warps of their own (33.0).
constexpr float kTiny = 7.888609052210118e-31f;      // 2^-100

template <bool BF, int D, bool AXES>
__global__ void __launch_bounds__(kThreads)
k_append_normed(const Pool p, const AppendArgs a) {
  __shared__ float4 s_cs[4 * kChunks];
  __shared__ __align__(16) float s_w[2][D];        // weights of q and k
  __shared__ long long s_row;
  __shared__ int s_live;
  constexpr int LP = D / 16;       // lanes of a head
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, row = blockIdx.x;
  const int half = a.rot >> 1, rc = a.rot >> 4;
  const int q0 = a.q ? p.Hq : 0, heads = q0 + 2 * p.Hkv, items = heads * LP;
  const int c = tid % LP;          // this thread's channels, in every head that it takes
  const bool turned = c < rc;
  const int lo_at = turned && !a.interleaved ? 8 * c : 16 * c, hi_at = turned && !a.interleaved ? lo_at + half : lo_at + 8;
  for (int j0 = tid; j0 - tid < items; j0 += kThreads) {
    const int head = j0 / LP;
    const bool is = head < heads;
    const int kind = head < q0 ? 0 : head < q0 + p.Hkv ? 1 : 2;       // q, k, v
    const int h = head - (kind == 0 ? 0 : kind == 1 ? q0 : q0 + p.Hkv);
    const uint16_t* src = (kind == 0 ? a.q + row * a.qs : kind == 1 ? a.k + row * a.ks : a.v + row * a.vs) + h * D;
    const int lo = kind == 2 ? 16 * c : lo_at, hi = kind == 2 ? 16 * c + 8 : hi_at;
    uint4 raw[2] = {};
    if (is) {
      raw[0] = *reinterpret_cast<const uint4*>(src + lo);
      raw[1] = *reinterpret_cast<const uint4*>(src + hi);
    }
    if (j0 == tid) {               // the first time round: where the row goes, its sines, the weights
      if (tid < 64) {
        place_row<AXES>(p, a, row, half, s_cs, &s_row, &s_live);
      } else {
        for (int i = tid - 64; i < 2 * D; i += kThreads - 64) {
          const void* w = i < D ? a.q_norm : a.k_norm;
          const int ch = i < D ? i : i - D;
          s_w[i < D ? 0 : 1][ch] = !w ? 1.0f : a.norm_fp32 ? static_cast<const float*>(w)[ch] : to_f(static_cast<const uint16_t*>(w)[ch], BF);
        }
      }
      __syncthreads();
      if (!s_live) return;
    }
    const long long at = s_row;
    // (whole warps: a head's lanes need each other, and a warp can hold heads of all kinds)
    float x[16], ss = 0.0f;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = unpack2<BF>(words[i]);
      x[2 * i] = t.x;
      x[2 * i + 1] = t.y;
      ss = fmaf(t.x, t.x, ss);
      ss = fmaf(t.y, t.y, ss);
    }
#pragma unroll
    for (int o = 1; o < LP; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    float inv = rsqrtf(ss * (1.0f / D) + a.eps);
    if (__any_sync(0xffffffffu, !(ss < INFINITY))) {
      float big = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) big = fmaf(x[i] * kTiny, x[i] * kTiny, big);
#pragma unroll
      for (int o = 1; o < LP; o <<= 1) big += __shfl_xor_sync(0xffffffffu, big, o);
      // (from 2^126 on a subnormal number, good to 2^-21 of itself at least, and x inv with it)
      if (!(ss < INFINITY)) inv = kTiny * rsqrtf(big * (1.0f / D));
    }
    if (kind != 2) {
      if (kind == 0 ? a.q_norm != nullptr : a.k_norm != nullptr) {
        const float4* w = reinterpret_cast<const float4*>(s_w[kind]);
        const float4 w4[4] = {w[lo >> 2], w[(lo >> 2) + 1], w[hi >> 2], w[(hi >> 2) + 1]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {      // (inv * w first could leave fp32's range where the row's values do not)
          x[4 * i] = x[4 * i] * inv * w4[i].x;
          x[4 * i + 1] = x[4 * i + 1] * inv * w4[i].y;
          x[4 * i + 2] = x[4 * i + 2] * inv * w4[i].z;
          x[4 * i + 3] = x[4 * i + 3] * inv * w4[i].w;
        }
      }
      if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 t = s_cs[i * kChunks + c];
          // half-split: pair e is x[e], x[8 + e]; interleaved: x[2 e], x[2 e + 1]
          if (a.interleaved) {
            const float x0 = x[4 * i], y0 = x[4 * i + 1], x1 = x[4 * i + 2], y1 = x[4 * i + 3];
            x[4 * i] = x0 * t.x - y0 * t.y;
            x[4 * i + 1] = y0 * t.x + x0 * t.y;
            x[4 * i + 2] = x1 * t.z - y1 * t.w;
            x[4 * i + 3] = y1 * t.z + x1 * t.w;
          } else {
            const float x0 = x[2 * i], y0 = x[8 + 2 * i], x1 = x[2 * i + 1], y1 = x[9 + 2 * i];
            x[2 * i] = x0 * t.x - y0 * t.y;
            x[8 + 2 * i] = y0 * t.x + x0 * t.y;
            x[2 * i + 1] = x1 * t.z - y1 * t.w;
            x[9 + 2 * i] = y1 * t.z + x1 * t.w;
          }
        }
      }
      uint32_t* out = reinterpret_cast<uint32_t*>(raw);
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = pack2<BF>(x[2 * i], x[2 * i + 1]);
    }
    if (!is || (kind > 0 && at < 0)) continue;
    uint16_t* out = kind == 0 ? a.q_out + row * a.qos + h * D
                              : (kind == 1 ? p.k : p.v) + at + static_cast<long long>(h) * p.ps * D;
    *reinterpret_cast<uint4*>(out + lo) = raw[0];
    *reinterpret_cast<uint4*>(out + hi) = raw[1];
  }
}

}  // namespace

cudaError_t launch_append(const Pool& p, const AppendArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_pdl(p.bf16 ? k_append<true> : k_append<false>, dim3(a.rows), dim3(kThreads), 0, s, p, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_append_normed(const Pool& p, const AppendArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  auto go = [&](auto kernel) { e = launch_pdl(kernel, dim3(a.rows), dim3(kThreads), 0, s, p, a); };
  auto of = [&](auto bf) {
    constexpr bool BF = decltype(bf)::value;
    if (p.d == 128) a.axis ? go(k_append_normed<BF, 128, true>) : go(k_append_normed<BF, 128, false>);
    else a.axis ? go(k_append_normed<BF, 64, true>) : go(k_append_normed<BF, 64, false>);
  };
  p.bf16 ? of(std::true_type{}) : of(std::false_type{});
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace paged
}  // namespace confkv
