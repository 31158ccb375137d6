// Internal layout of the paged cache and launch wrappers of its operators
// (include/confkv_paged.h).
//
// Pools k, v: [L][num_pages][Hkv][page_size][d], fp16 or bf16.  A page of one
// head is page_size * d contiguous elements, so one TMA box reads a page's
// (or a tile's) rows.  Element offsets are 64-bit, rows of a pool fit 31 bits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/confkv_paged.h"
#include "confkv_internal.cuh"

namespace confkv {
namespace paged {

struct Pool {
  uint16_t* k;
  uint16_t* v;
  int L, NP, Hq, Hkv, g, d, ps, ps_shift;   // ps = 1 << ps_shift
  int bf16;
  int32_t* err;                             // latched CONFKV_FLAG_* bits
};

struct Batch {
  int B, max_blocks;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* q_start;
  const uint32_t* mask;
  int mask_words;
};

struct AppendArgs {
  Batch bt;
  int layer, rows;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;
  uint16_t* q_out;
  long long ks, vs, qs, qos;    // row strides in elements
  const int32_t* pos;
  const float* inv_freq;
  int rot, interleaved;
};

struct AttendArgs {
  Batch bt;
  int layer, rows;
  const uint16_t* q;
  long long qs;
  uint16_t* out;
  float* lse;
  float scale;
};

struct CommitArgs {
  int B, max_blocks, cap;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* path;
  const int32_t* path_len;
  int32_t* new_len;
};

struct ForkArgs {
  int rows, beams, max_blocks;
  const int32_t* parent;
  const int32_t* table_in;
  const int32_t* len_in;
  const int32_t* tail;
  int32_t* table_out;
  int32_t* len_out;
};

struct BeamArgs {
  const void* logits;
  int dtype;
  long long stride;
  int B, W, V, K;
  const float* scores;
  const uint8_t* finished;
  int pad;
  float* score_out;
  int32_t* parent_out;
  int32_t* token_out;
  int32_t* flags_out;
  void* ws;
};

cudaError_t launch_append(const Pool& p, const AppendArgs& a, cudaStream_t s);
cudaError_t launch_commit(const Pool& p, const CommitArgs& a, cudaStream_t s);
cudaError_t launch_fork(const Pool& p, const ForkArgs& a, cudaStream_t s);
cudaError_t launch_beam(const BeamArgs& a, cudaStream_t s);
size_t beam_workspace(int B, int W, int V, int K, int dtype);

// ---- device helpers ----
__device__ __forceinline__ float to_f(uint16_t x, bool bf) {
  return bf ? __uint_as_float(static_cast<uint32_t>(x) << 16) : __half2float(__ushort_as_half(x));
}
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}
// two floats rounded to the cache's type (round to nearest even)
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  uint32_t r;
  if constexpr (BF)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(y), "f"(x));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

// The sequence that a row belongs to: how many sequences end at or before it
// (every lane of the warp gets it; B where the row is behind the last one).
__device__ __forceinline__ int sequence_of(const int32_t* q_start, int B, int row) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  for (int b = lane; b < B; b += 32) n += (q_start[b + 1] <= row) ? 1 : 0;
  return __reduce_add_sync(0xffffffffu, n);
}

// Takes a ticket: behind a barrier of the CTA one thread's call orders what all of
// its threads wrote before what the CTAs that take later tickets read (after a
// barrier of their own).  A fence of every thread on both sides costs 0.3 to
// 0.6 us more.
__device__ __forceinline__ unsigned take_ticket(unsigned* ticket) {
  unsigned n;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;\n" : "=r"(n) : "l"(ticket) : "memory");
  return n;
}

// launch_pdl, the grid in clusters of `cluster` CTAs
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, int cluster, size_t smem, cudaStream_t s,
                               Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace paged
}  // namespace confkv
