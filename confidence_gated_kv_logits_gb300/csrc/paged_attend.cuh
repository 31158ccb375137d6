// Parts shared by the two paged attention kernels (k_paged_attend.cu: few rows
// per sequence, k_paged_attend_many.cu: many).
#pragma once
#include "paged_internal.cuh"
#include "paged_ptx.cuh"
#include "paged_sched.cuh"

namespace confkv {
namespace paged {

struct AttendMaps {                    // pools as rows of d elements, boxes of 64 channels
  CUtensorMap k_few, v_few;            // x min(page_size, chunk) rows
  CUtensorMap k_many, v_many;          // x min(page_size, 128) rows
};

constexpr int kFewRows = 16;           // query rows of a tile
constexpr int kFewChunk = 2048;        // elements of K in a chunk (tokens x d)
constexpr int kManyRows = 256;         // two tiles of 128
constexpr int kManyBlock = 128;        // tokens of a block

// Where the boxes of a page that is not in the pool are asked for: rows before the
// pool.  TMA gives NaN for K there and zeroes for V, so that the scores of such a
// page's tokens, and with them the rows that see one, are NaN.
constexpr int kNoRows = -kManyBlock;

// CTAs of a launch: one per SM
constexpr int kFewCtasPerSm = 1;

cudaError_t launch_attend_few(const Pool& p, const AttendArgs& a, const Scratch& sc, const AttendMaps& m,
                              int ctas, int cluster, cudaStream_t s);
cudaError_t launch_attend_many(const Pool& p, const AttendArgs& a, const Scratch& sc, const AttendMaps& m,
                               int ctas, bool two_tiles, bool defer, cudaStream_t s);
cudaError_t setup_attend_few();
cudaError_t few_clusters(int size, int* fit);       // clusters of `size` CTAs that run at once
cudaError_t setup_attend_many();

// 0xffff in each half of a word whose element is NaN or infinite
template <bool BF>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x) {
  constexpr uint32_t E = BF ? 0x7f80u : 0x7c00u;
  return ((x & E) == E ? 0xffffu : 0u) | (((x >> 16) & E) == E ? 0xffff0000u : 0u);
}

// N channels of an output row: acc / l (0 where nothing was seen), rounded once
template <bool BF, int N>
__device__ __forceinline__ void store_row(const AttendArgs& a, const Pool& p, int row, int hq, int ch, const float (&x)[N],
                                          float m, float l) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const size_t at = static_cast<size_t>(row) * p.Hq + hq;
  uint16_t* out = a.out + at * p.d + ch;
  static_assert(N % 4 == 0, "whole 8-byte words");
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int e = 0; e < N; e += 8)
      *reinterpret_cast<uint4*>(out + e) =
          make_uint4(pack2<BF>(x[e] * inv, x[e + 1] * inv), pack2<BF>(x[e + 2] * inv, x[e + 3] * inv),
                     pack2<BF>(x[e + 4] * inv, x[e + 5] * inv), pack2<BF>(x[e + 6] * inv, x[e + 7] * inv));
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 4)
      *reinterpret_cast<uint2*>(out + e) =
          make_uint2(pack2<BF>(x[e] * inv, x[e + 1] * inv), pack2<BF>(x[e + 2] * inv, x[e + 3] * inv));
  }
  if (a.lse && ch == 0) a.lse[at] = l == 0.0f ? -INFINITY : m * a.scale + logf(l);
}

// Where the pieces' partial results of the walk's current unit lie: piece i of
// it, of CTA first + i, in that CTA's second place if it is the unit's first.
template <typename W>
__device__ __forceinline__ size_t piece_place(const W& w, int i) {
  return 2 * static_cast<size_t>(w.first_cta + i) + (i == 0 ? 1 : 0);
}

// Partial accumulators lie as [place][d / 4][row][4]: both the threads of a
// warp that hold one row each and those that join them touch whole lines.
template <int TM, int D>
__device__ __forceinline__ float* acc_at(const Scratch& sc, size_t place, int row, int ch) {
  return sc.acc + (place * (D / 4) + (ch >> 2)) * (TM * 4) + 4 * row;
}

// N channels of one row joined over a unit's pieces, in their order (so that
// the sum does not depend on who joins), U pieces' loads in flight: what this
// costs is round trips to L2.  A piece in which the row saw nothing has the sum
// 0 and is left out; one whose scores were all NaN has the maximum -inf too, but
// the sum NaN, which has to reach the row.  `own` >= 0: that piece is this thread's, in x
// with maximum m and sum l, and is not read.
template <int TM, int D, int N, int U, typename W>
__device__ __forceinline__ void join_row(const Scratch& sc, const W& w, int row, int ch, float c, int own, float (&x)[N],
                                         float& m, float& l) {
  float z[N];
  const float om = m, ol = l;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    z[e] = x[e];
    x[e] = 0.0f;
  }
  m = own >= 0 ? om : -INFINITY;
  l = 0.0f;
  if (w.pieces > U) {       // else the one round below brings all maxima
#pragma unroll 8
    for (int i = 0; i < w.pieces; ++i)
      if (i != own) m = fmaxf(m, __ldcg(sc.ml + (piece_place(w, i) * TM + row) * 2));
  }
#pragma unroll 1
  for (int i0 = 0; i0 < w.pieces; i0 += U) {
    float2 ml[U];
    float4 v[U][N / 4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i < w.pieces && i != own) {
        const size_t at = piece_place(w, i);
        ml[u] = __ldcg(reinterpret_cast<const float2*>(sc.ml + (at * TM + row) * 2));
#pragma unroll
        for (int e = 0; e < N / 4; ++e)
          v[u][e] = __ldcg(reinterpret_cast<const float4*>(acc_at<TM, D>(sc, at, row, ch + 4 * e)));
      }
    }
    if (w.pieces <= U) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < w.pieces && u != own) m = fmaxf(m, ml[u].x);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i >= w.pieces) break;
      const float li = i == own ? ol : ml[u].y;
      if (li == 0.0f) continue;
      const float f = ex2f(((i == own ? om : ml[u].x) - m) * c);
      l = fmaf(f, li, l);
      if (i == own) {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = fmaf(f, z[e], x[e]);
      } else {
#pragma unroll
        for (int e = 0; e < N / 4; ++e) {
          x[4 * e] = fmaf(f, v[u][e].x, x[4 * e]);
          x[4 * e + 1] = fmaf(f, v[u][e].y, x[4 * e + 1]);
          x[4 * e + 2] = fmaf(f, v[u][e].z, x[4 * e + 2]);
          x[4 * e + 3] = fmaf(f, v[u][e].w, x[4 * e + 3]);
        }
      }
    }
  }
}

}  // namespace paged
}  // namespace confkv
