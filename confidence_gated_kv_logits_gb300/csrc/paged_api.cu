// Host side of the paged-cache and beam operators (include/confkv_paged.h):
// handle lifetime, argument checks and launches.  No call but create, free
// and status synchronises or allocates.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <mutex>
#include <new>

#include "paged_attend.cuh"

using namespace confkv::paged;

namespace confkv {
namespace paged {

cudaError_t encode_map(CUtensorMap* map, bool bf16, int rank, void* at, const cuuint64_t* dims, const cuuint64_t* strides,
                       const cuuint32_t* box, bool nan_outside) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<Encode> known{nullptr};
  Encode enc = known.load();
  if (!enc) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    enc = reinterpret_cast<Encode>(fn);
    known.store(enc);
  }
  const cuuint32_t steps[3] = {1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, at, dims, strides, box, steps,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             nan_outside ? CU_TENSOR_MAP_FLOAT_OOB_FILL_NAN_REQUEST_ZERO_FMA : CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

}  // namespace paged
}  // namespace confkv

namespace {

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (dev < 0 || dev == prev) prev = -1;
    else cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
bool good_stride(int64_t s, int64_t width) { return s >= width && s % 8 == 0 && s < (1ll << 40); }
// [a, a + na) and [b, b + nb) share a byte
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
// rows of wa / wb elements of 2 bytes, sa / sb elements apart, share a byte
// (rows of one buffer with one stride may lie side by side; with two strides
// any common range counts as shared)
bool rows_overlap(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int rows) {
  const size_t na = (static_cast<size_t>(rows - 1) * sa + wa) * 2, nb = (static_cast<size_t>(rows - 1) * sb + wb) * 2;
  if (!overlap(a, na, b, nb)) return false;
  if (sa != sb) return true;
  const int64_t step = 2 * sa;
  int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) % step;
  if (d < 0) d += step;
  return d < 2 * wa || d + 2 * wb > step;
}

struct Limits {         // what a device runs at once: CTAs of the big kernels, clusters of two, four and eight
  int sms, clusters2, clusters4, clusters8;
};

}  // namespace

struct confkv_paged {
  Pool pool{};
  AttendMaps maps;
  Scratch scratch{};
  Limits limits = {};
  int device = 0;
  const char* msg = "ok";     // static texts only: no allocation, so nothing can throw
};

namespace {

int fail(confkv_paged* kv, int code, const char* msg) {
  kv->msg = msg;
  return code;
}

int launched(confkv_paged* kv, cudaError_t e) {
  if (e == cudaSuccess) return CONFKV_OK;
  return fail(kv, CONFKV_ERR_CUDA, cudaGetErrorString(e));
}

const char* check_batch(const confkv_paged_batch* b, bool masked) {
  if (!b) return "null batch";
  if (b->batch < 1 || b->batch > 65536) return "batch must be in 1 .. 65536";
  if (b->max_blocks < 1) return "max_blocks must be positive";
  if (!b->page_table || !b->ctx_len || !b->q_start) return "null page_table, ctx_len or q_start";
  if (!aligned4(b->page_table) || !aligned4(b->ctx_len) || !aligned4(b->q_start) || !aligned4(b->mask))
    return "page_table, ctx_len, q_start and mask must be 4-byte aligned";
  if (masked && b->mask && b->mask_words < 1) return "mask_words must be positive";
  return nullptr;
}

// An output shares a byte with the batch's own tensors.  (CTAs plan for themselves from what these hold: were they
// to change while a kernel runs, one could look for sequences behind the last.)
bool in_batch(const confkv_paged_batch* b, int rows, const void* out, size_t n) {
  const size_t seqs = static_cast<size_t>(b->batch);
  return overlap(out, n, b->page_table, seqs * b->max_blocks * 4) || overlap(out, n, b->ctx_len, seqs * 4) ||
         overlap(out, n, b->q_start, (seqs + 1) * 4) ||
         (b->mask && b->mask_words > 0 && overlap(out, n, b->mask, static_cast<size_t>(rows) * b->mask_words * 4));
}

// Tensor maps of both pools for both kernels: rows of d elements in boxes of 64
// channels (128 bytes, swizzled) x as many rows as a page and the kernel's tile share.
// Rows outside the pool (kNoRows) read as NaN from K's maps and as zero from V's.
cudaError_t encode_maps(const Pool& p, AttendMaps* m) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.d),
                              static_cast<cuuint64_t>(p.L) * p.NP * p.Hkv * p.ps};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.d) * 2};
  const int few = std::min(p.ps, kFewChunk / p.d), many = std::min(p.ps, kManyBlock);
  struct {
    CUtensorMap* map;
    uint16_t* pool;
    int rows;
    bool nan_outside;
  } const all[] = {{&m->k_few, p.k, few, true}, {&m->v_few, p.v, few, false}, {&m->k_many, p.k, many, true}, {&m->v_many, p.v, many, false}};
  for (const auto& x : all) {
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(x.rows)};
    const cudaError_t e = encode_map(x.map, p.bf16, 2, x.pool, dims, strides, box, x.nan_outside);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// What the device runs at once and, the first time, the kernels' shared-memory
// limits (function attributes hold per device).
cudaError_t device_ready(int dev, Limits* limits) {
  constexpr int kDevices = 64;
  static std::mutex mu;
  static Limits known[kDevices] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  if (!known[dev].sms) {
    Limits n = {};
    cudaError_t e = cudaDeviceGetAttribute(&n.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = setup_attend_few();
    if (e == cudaSuccess) e = setup_attend_many();
    if (e == cudaSuccess) e = setup_evict();
    if (e == cudaSuccess) e = setup_weigh();
    if (e == cudaSuccess) e = few_clusters(2, &n.clusters2);
    if (e == cudaSuccess) e = few_clusters(4, &n.clusters4);
    if (e == cudaSuccess) e = few_clusters(8, &n.clusters8);
    if (e != cudaSuccess) return e;
    known[dev] = n;
  }
  *limits = known[dev];
  return cudaSuccess;
}

// CTAs that share a unit of the few rows' kernel as a cluster, or 1 to cut the
// units into equal shares. A cluster joins its pieces in 1 us where tickets and
// the scratch take 3 to 4, but holds 96 of 152 SMs at worst, so it is for units
// that all run at once and sequences that cannot be long (a table's width is
// what the host knows): from 9 chunks (below, one CTA does) to 16 a warp.
// Behind a shared prefix the width holds the prefix too, which says little of the tokens that phase 2 has left; us, cut
// against clusters: 12/12 heads of 64, 4 x 300 own tokens behind 1000 10.6, 15.6; 3000 own 24.6, 21.7; 40/8 heads of 128,
// 2 x 300 behind 300 12.0, 12.8; 1500 own 22.3, 13.3; 1 x 300 behind 4000 14.7, 19.5; 3000 own 25.9, 21.6.
// One row, us, cut against clusters: 12/12 heads of 64, 1 x 512 tokens 8.5, 7.6;
// 1 x 2048 10.6, 8.5; 1 x 16384 18.5, 16.7; 2 x 4000 13.6, 11.1; 40/8 heads of 128,
// 1 x 1024 12.1, 9.1; 1 x 8192 19.0, 17.0; 1 x 16384 24.9, 24.9; 4 x 2000 18.3,
// 13.3; 8 x 4000 31.6, 27.4.  More clusters than run at once (16 of eight): 2 x 1500
// 12.9, 18.2.
int few_cluster(const confkv_paged& kv, int batch, int64_t units, int64_t tokens) {
  const int64_t chunks = (tokens * kv.pool.d + kFewChunk - 1) / kFewChunk;
  if (batch > 32 || chunks <= 8) return 1;
  if (units <= kv.limits.clusters8) return chunks <= 16 * 64 ? 8 : 1;
  if (units <= kv.limits.clusters4) return chunks <= 16 * 32 ? 4 : 1;
  if (units <= kv.limits.clusters2) return chunks <= 16 * 16 ? 2 : 1;
  return 1;
}

// [flags][tickets][cut units] (zeroed by the caller) [(maximum, sum)][accumulators]: two
// places per CTA, as a CTA's share cuts at most the unit it starts in and the
// one it ends in
constexpr size_t kTicketsAt = 256;
size_t scratch_rows(int sms) { return 2 * static_cast<size_t>(sms) * std::max(kFewCtasMost * kFewRows, kManyRows); }
size_t scratch_bytes_of(int sms, int d) { return CONFKV_PAGED_ZEROED + scratch_rows(sms) * (2 + d) * sizeof(float); }
constexpr size_t kCutAt = 8192;
bool tickets_fit(int sms) {
  return kTicketsAt + sizeof(unsigned int) * kFewCtasMost * sms <= kCutAt && kCutAt + sizeof(int4) * sms <= CONFKV_PAGED_ZEROED;
}

Batch batch_of(const confkv_paged_batch* b) {
  return Batch{b->batch, b->max_blocks, b->page_table, b->ctx_len, b->q_start, b->mask, b->mask ? b->mask_words : 0,
               0, 0, b->batch, nullptr, nullptr};
}

// The checks that both appends share; null and *a filled where there is nothing to refuse.
const char* append_args(const Pool& p, const confkv_paged_batch* batch, int layer, int rows, const void* k, int64_t k_stride,
                        const void* v, int64_t v_stride, const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                        const int32_t* positions, const float* inv_freq, int rotary_dim, int interleaved, AppendArgs* a) {
  if (const char* m = check_batch(batch, false)) return m;
  if (layer < 0 || layer >= p.L) return "no such layer";
  if (rows < 0) return "rows < 0";
  if (rows == 0) return nullptr;
  if (!k || !v) return "null k or v";
  if ((q == nullptr) != (q_out == nullptr)) return "q and q_out go together";
  const int64_t wk = static_cast<int64_t>(p.Hkv) * p.d, wq = static_cast<int64_t>(p.Hq) * p.d;
  if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out)) return "k, v, q and q_out must be 16-byte aligned";
  if (!good_stride(k_stride, wk) || !good_stride(v_stride, wk) ||
      (q && (!good_stride(q_stride, wq) || !good_stride(q_out_stride, wq))))
    return "a row stride is below the row's width or no multiple of 8";
  if (!inv_freq) rotary_dim = 0;
  else if (rotary_dim < 16 || rotary_dim % 16 || rotary_dim > p.d) return "rotary_dim must be a multiple of 16 up to head_dim";
  if (interleaved < 0 || interleaved > 1) return "interleaved must be 0 or 1";
  if (!aligned4(positions) || !aligned4(inv_freq)) return "positions and inv_freq must be 4-byte aligned";
  if (q && !(q == q_out && q_stride == q_out_stride) && rows_overlap(q, q_stride, wq, q_out, q_out_stride, wq, rows))
    return "q_out overlaps q and is not q itself";
  if (q && (rows_overlap(k, k_stride, wk, q_out, q_out_stride, wq, rows) ||
            rows_overlap(v, v_stride, wk, q_out, q_out_stride, wq, rows)))
    return "q_out overlaps k or v";
  if (q && in_batch(batch, rows, q_out, (static_cast<size_t>(rows - 1) * q_out_stride + wq) * 2))
    return "q_out overlaps the batch's tensors";
  *a = AppendArgs{};
  a->bt = batch_of(batch);
  a->layer = layer;
  a->rows = rows;
  a->k = static_cast<const uint16_t*>(k);
  a->v = static_cast<const uint16_t*>(v);
  a->q = static_cast<const uint16_t*>(q);
  a->q_out = static_cast<uint16_t*>(q_out);
  a->ks = k_stride;
  a->vs = v_stride;
  a->qs = q_stride;
  a->qos = q_out_stride;
  a->pos = positions;
  a->inv_freq = inv_freq;
  a->rot = rotary_dim;
  a->interleaved = interleaved;
  return nullptr;
}

// The checks that both attends share; null and *a filled where there is nothing to refuse.
const char* attend_args(const Pool& p, const confkv_paged_batch* batch, int layer, int rows, const void* q, int64_t q_stride,
                        void* out, float* lse, float scale, AttendArgs* a) {
  if (const char* m = check_batch(batch, true)) return m;
  if (layer < 0 || layer >= p.L) return "no such layer";
  if (rows < 0) return "rows < 0";
  if (static_cast<int64_t>(rows) * p.Hq >= (1ll << 31)) return "rows x heads must be below 2^31";
  if (rows == 0) return nullptr;
  if (!q || !out) return "null q or out";
  const int64_t wq = static_cast<int64_t>(p.Hq) * p.d;
  if (!aligned16(q) || !aligned16(out) || !aligned4(lse)) return "q and out must be 16-byte aligned, lse 4-byte";
  if (!good_stride(q_stride, wq)) return "q_stride is below the row's width or no multiple of 8";
  if (!(scale >= 0.0f && std::isfinite(scale))) return "scale must be finite and not negative";
  if (rows_overlap(q, q_stride, wq, out, wq, wq, rows)) return "out overlaps q";
  const size_t nr = static_cast<size_t>(rows);
  if (lse && (overlap(lse, nr * p.Hq * 4, out, nr * wq * 2) || overlap(lse, nr * p.Hq * 4, q, ((nr - 1) * q_stride + wq) * 2)))
    return "lse overlaps q or out";
  if (in_batch(batch, rows, out, nr * wq * 2) || (lse && in_batch(batch, rows, lse, nr * p.Hq * 4)))
    return "out or lse overlaps the batch's tensors";
  *a = AttendArgs{batch_of(batch), layer, rows, static_cast<const uint16_t*>(q), q_stride, static_cast<uint16_t*>(out), lse,
                  scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(p.d)), nullptr, nullptr};
  return nullptr;
}

// Launches the attention of `batch` sequences (groups, over a shared prefix).
cudaError_t attend(const confkv_paged& kv, const AttendArgs& a, int batch, cudaStream_t s) {
  const Pool& p = kv.pool;
  // By the query rows of a sequence's (a group's) KV head, on average (measured on GB300, us):
  //  - up to 16 the streaming kernel (1 x 32768 tokens, 40/8 heads, d = 128: 10 rows 37
  //    streamed, 42 with the padded tiles of 128; 20 rows 62 in two streamed tiles, 42)
  //  - from 257 on units of two tiles, which share each K and V block, if they fill half
  //    the GPU (8 x 8192 tokens: 385 rows 152, 194 in units of one tile; 1 x 32768 tokens,
  //    whose 16 units do not: 260 rows 110, 87 in units of one)
  //  - one kernel for the whole batch, so that chunks beside single tokens go with the
  //    average: 128 rows over 2048 tokens and 64 x 1 row over 2048 (40/8 heads, d =
  //    128) take 135 together, 32 and 88 in a call each; 512 rows over 2048 and 255 x 1
  //    row 504, 62 and 310
  //  - far fewer units of one tile than CTAs are cut into many pieces each, which a
  //    kernel of its own joins on all SMs (1 x 32768 tokens, 65 rows: 58 joined by the
  //    last CTA of each unit, 42)
  const int64_t heads = static_cast<int64_t>(a.rows) * p.g, per = heads / batch;
  //  - behind a shared prefix, where sequences have few tokens of their own, the streaming kernel up to 40 rows in its tiles
  //    of 16.  Neither is the faster one throughout: few or ragged units leave the prompt kernel's SMs idle, many or long
  //    ones are faster there from 20 to 30 rows on.  Streamed and in padded tiles: 32/4 heads of 64, 11 ragged sequences of
  //    up to 400 own tokens, 32 rows 28.1, 40.1; 40/8 of 128, 5 ragged of up to 1000, 25 rows 43.5, 53.1; 3, 23 rows 27.9,
  //    45.9; 64/8 of 64, two groups of 4 of 300 own behind 6000, 18 rows 27.7, 32.2, 40 rows 43.0, 40.4; two of 8, 18 rows
  //    43.2, 39.1, 32 rows 51.5, 38.8; two of 32, 18 rows 70.4, 83.4, 40 rows 116, 114; two of 8 of 2000 own, 32 rows 66.4,
  //    57.1; 72 rows 52, 48
  if (per <= (a.bt.phase == 2 ? 40 : kFewRows)) {
    // at most (a row's heads fill one tile, or its sequence's last is part-filled)
    const int64_t units = p.Hkv * std::min<int64_t>(static_cast<int64_t>(a.rows) * ((p.g + kFewRows - 1) / kFewRows),
                                                    heads / kFewRows + batch);
    const int cl = few_cluster(kv, batch, units, static_cast<int64_t>(a.bt.max_blocks) * p.ps);
    // Behind a shared prefix many sequences have few tokens of their own: from 32 on CTAs of four warps, two per SM, so
    // that one's joins run beside another's tiles (40/8 heads of 128, one row each, us, of eight warps and of four: 32
    // sequences of 200 own tokens 45.0, 35.3; 64 of 700 76.3, 68.8; 128 of 2000 151, 142; 32 of 8000 134.6, 134.8; 16 of
    // 300 33.2, 36.1)
    if (a.bt.phase == 2 && cl == 1 && batch >= 32) return launch_attend_few(p, a, kv.scratch, kv.maps, kFewCtasMost * kv.limits.sms, 1, 4, s);
    const int ctas = cl > 1 ? cl * static_cast<int>(units) : kFewCtasPerSm * kv.limits.sms;
    return launch_attend_few(p, a, kv.scratch, kv.maps, ctas, cl, 8, s);
  }
  const int sms = kv.limits.sms;
  const int64_t ones = p.Hkv * (heads / 128 + batch), twos = p.Hkv * (heads / kManyRows + batch);
  const bool two = per > kManyRows && 2 * twos >= sms;
  return launch_attend_many(p, a, kv.scratch, kv.maps, sms, two, !two && 4 * ones <= sms, s);
}

// [rows][heads][d] accumulators, [rows][heads] (maximum, sum)
size_t partial_bytes(int rows, int heads, int d) { return static_cast<size_t>(rows) * heads * (d + 2) * sizeof(float); }

}  // namespace

extern "C" {

size_t confkv_paged_scratch(int head_dim, int device) {
  int dev = device, sms = 0;
  if ((head_dim != 64 && head_dim != 128) || (dev < 0 && cudaGetDevice(&dev) != cudaSuccess) ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || !tickets_fit(sms)) {
    cudaGetLastError();
    return 0;
  }
  return scratch_bytes_of(sms, head_dim);
}

int confkv_paged_create(int layers, int heads, int kv_heads, int head_dim, int num_pages, int page_size,
                        int dtype, int device, void* k_pages, void* v_pages, void* scratch, size_t scratch_bytes,
                        confkv_paged** out) {
  if (!out) return CONFKV_ERR_INVALID_ARG;
  *out = nullptr;
  if (layers < 1 || layers > 32767 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 ||
      heads / kv_heads > confkv::kMaxGroup || (head_dim != 64 && head_dim != 128) || num_pages < 1 ||
      (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256) ||
      (dtype != CONFKV_FP16 && dtype != CONFKV_BF16) || !k_pages || !v_pages || !scratch ||
      (reinterpret_cast<uintptr_t>(scratch) & 255) || ((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 127))
    return CONFKV_ERR_INVALID_ARG;
  // rows of a pool stay below 2^31 (checked factor by factor: no overflow)
  long long n = layers;
  for (const long long f : {static_cast<long long>(num_pages), static_cast<long long>(kv_heads),
                            static_cast<long long>(page_size)}) {
    n *= f;
    if (n >= (1ll << 31)) return CONFKV_ERR_INVALID_ARG;
  }
  int dev = device;
  if (dev < 0 && cudaGetDevice(&dev) != cudaSuccess) return CONFKV_ERR_CUDA;
  DeviceGuard guard(dev);
  confkv_paged* kv = new (std::nothrow) confkv_paged();
  if (!kv) return CONFKV_ERR_OOM;
  kv->device = dev;
  Pool& p = kv->pool;
  p.k = static_cast<uint16_t*>(k_pages);
  p.v = static_cast<uint16_t*>(v_pages);
  p.L = layers;
  p.NP = num_pages;
  p.Hq = heads;
  p.Hkv = kv_heads;
  p.g = heads / kv_heads;
  p.d = head_dim;
  p.ps = page_size;
  while ((1 << p.ps_shift) < page_size) ++p.ps_shift;
  p.bf16 = dtype == CONFKV_BF16;
  cudaError_t e = device_ready(dev, &kv->limits);
  if (e == cudaSuccess) e = encode_maps(p, &kv->maps);
  if (e != cudaSuccess || !tickets_fit(kv->limits.sms) || scratch_bytes < scratch_bytes_of(kv->limits.sms, head_dim)) {
    cudaGetLastError();
    delete kv;
    return e != cudaSuccess ? CONFKV_ERR_CUDA : CONFKV_ERR_CAPACITY;
  }
  char* at = static_cast<char*>(scratch);
  p.err = reinterpret_cast<int32_t*>(at);
  kv->scratch.ticket = reinterpret_cast<unsigned int*>(at + kTicketsAt);
  kv->scratch.cut = reinterpret_cast<int4*>(at + kCutAt);
  kv->scratch.ml = reinterpret_cast<float*>(at + CONFKV_PAGED_ZEROED);
  kv->scratch.acc = kv->scratch.ml + 2 * scratch_rows(kv->limits.sms);
  *out = kv;
  return CONFKV_OK;
}

void confkv_paged_free(confkv_paged* kv) { delete kv; }

const char* confkv_paged_last_error(const confkv_paged* kv) { return kv ? kv->msg : "null handle"; }

int confkv_paged_status(confkv_paged* kv, int32_t* flags) {
  if (!kv) return CONFKV_ERR_INVALID_ARG;
  DeviceGuard guard(kv->device);
  int32_t f = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&f, kv->pool.err, sizeof(f), cudaMemcpyDeviceToHost);
  // with the flags the tickets: a launch that gave up (CONFKV_FLAG_TIMEOUT) may have left some
  if (e == cudaSuccess && f) e = cudaMemset(kv->pool.err, 0, CONFKV_PAGED_ZEROED);
  if (e == cudaSuccess && f) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return launched(kv, e);
  if (flags) *flags = f;
  return f ? fail(kv, CONFKV_ERR_DEVICE, "the GPU latched CONFKV_FLAG_* bits") : CONFKV_OK;
}

int confkv_paged_append(confkv_paged* kv, const confkv_paged_batch* batch, int layer, int rows, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, const void* q, int64_t q_stride,
                        void* q_out, int64_t q_out_stride, const int32_t* positions, const float* inv_freq,
                        int rotary_dim, int interleaved, void* stream) {
  if (!kv) return CONFKV_ERR_INVALID_ARG;
  AppendArgs a{};
  const char* m = append_args(kv->pool, batch, layer, rows, k, k_stride, v, v_stride, q, q_stride, q_out, q_out_stride,
                              positions, inv_freq, rotary_dim, interleaved, &a);
  if (m) return fail(kv, CONFKV_ERR_INVALID_ARG, m);
  if (rows == 0) return CONFKV_OK;
  DeviceGuard guard(kv->device);
  return launched(kv, launch_append(kv->pool, a, static_cast<cudaStream_t>(stream)));
}

int confkv_paged_append_normed(confkv_paged* kv, const confkv_paged_batch* batch, int layer, int rows, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride, const void* q, int64_t q_stride,
                               void* q_out, int64_t q_out_stride, const int32_t* positions, const float* inv_freq,
                               int rotary_dim, int interleaved, const confkv_paged_norm* norm, void* stream) {
  if (!kv) return CONFKV_ERR_INVALID_ARG;
  const Pool& p = kv->pool;
  if (!norm) return fail(kv, CONFKV_ERR_INVALID_ARG, "null norm");
  AppendArgs a{};
  const char* m = append_args(p, batch, layer, rows, k, k_stride, v, v_stride, q, q_stride, q_out, q_out_stride,
                              positions, inv_freq, rotary_dim, interleaved, &a);
  if (m) return fail(kv, CONFKV_ERR_INVALID_ARG, m);
  if (rows > 0 && norm->q_norm && !q) return fail(kv, CONFKV_ERR_INVALID_ARG, "q_norm without q");
  if (norm->q_norm || norm->k_norm) {
    if (norm->norm_dtype != CONFKV_FP32 && norm->norm_dtype != (p.bf16 ? CONFKV_BF16 : CONFKV_FP16))
      return fail(kv, CONFKV_ERR_INVALID_ARG, "norm weights must be fp32 or of the cache's type");
    if (!(norm->eps >= 1e-12f && std::isfinite(norm->eps)))
      return fail(kv, CONFKV_ERR_INVALID_ARG, "eps must be finite and 1e-12 or more");
  }
  const bool wide = norm->norm_dtype == CONFKV_FP32;
  const uintptr_t elem = wide ? 3 : 1;
  if (((reinterpret_cast<uintptr_t>(norm->q_norm) | reinterpret_cast<uintptr_t>(norm->k_norm)) & elem) || !aligned4(norm->axis))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "q_norm and k_norm must be aligned to their type, axis 4-byte");
  if (norm->axis && (norm->axes < 1 || norm->axes > 8 || !positions || !inv_freq))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "axis needs positions, inv_freq and 1 .. 8 axes");
  if (q_out && rows > 0) {
    const size_t n = (static_cast<size_t>(rows - 1) * q_out_stride + static_cast<size_t>(p.Hq) * p.d) * 2;
    const size_t nw = static_cast<size_t>(p.d) * (elem + 1), nf = static_cast<size_t>(a.rot) * 2;
    if ((norm->q_norm && overlap(q_out, n, norm->q_norm, nw)) || (norm->k_norm && overlap(q_out, n, norm->k_norm, nw)) ||
        (positions && overlap(q_out, n, positions, static_cast<size_t>(rows) * (norm->axis ? norm->axes : 1) * 4)) ||
        (inv_freq && overlap(q_out, n, inv_freq, nf)) || (norm->axis && overlap(q_out, n, norm->axis, nf)))
      return fail(kv, CONFKV_ERR_INVALID_ARG, "q_out overlaps an input");
  }
  if (rows == 0) return CONFKV_OK;
  a.q_norm = norm->q_norm;
  a.k_norm = norm->k_norm;
  a.norm_fp32 = wide;
  a.eps = norm->eps;
  a.axis = norm->axis;
  a.axes = norm->axis ? norm->axes : 1;
  DeviceGuard guard(kv->device);
  return launched(kv, launch_append_normed(p, a, static_cast<cudaStream_t>(stream)));
}

int confkv_paged_attend(confkv_paged* kv, const confkv_paged_batch* batch, int layer, int rows, const void* q,
                        int64_t q_stride, void* out, float* lse, float scale, void* stream) {
  if (!kv) return CONFKV_ERR_INVALID_ARG;
  AttendArgs a{};
  if (const char* m = attend_args(kv->pool, batch, layer, rows, q, q_stride, out, lse, scale, &a))
    return fail(kv, CONFKV_ERR_INVALID_ARG, m);
  if (rows == 0) return CONFKV_OK;
  DeviceGuard guard(kv->device);
  return launched(kv, attend(*kv, a, batch->batch, static_cast<cudaStream_t>(stream)));
}

size_t confkv_paged_partial(int rows, int heads, int head_dim) {
  if (rows < 0 || heads < 1 || (head_dim != 64 && head_dim != 128) || static_cast<int64_t>(rows) * heads >= (1ll << 31)) return 0;
  return partial_bytes(rows > 0 ? rows : 1, heads, head_dim);
}

int confkv_paged_attend_shared(confkv_paged* kv, const confkv_paged_batch* batch, const confkv_paged_prefix* prefix,
                               int layer, int rows, const void* q, int64_t q_stride, void* out, float* lse, float scale,
                               void* stream) {
  if (!kv) return CONFKV_ERR_INVALID_ARG;
  const Pool& p = kv->pool;
  if (!prefix) return fail(kv, CONFKV_ERR_INVALID_ARG, "null prefix");
  AttendArgs a{};
  if (const char* m = attend_args(p, batch, layer, rows, q, q_stride, out, lse, scale, &a))
    return fail(kv, CONFKV_ERR_INVALID_ARG, m);
  if (prefix->groups < 1 || prefix->groups > batch->batch)
    return fail(kv, CONFKV_ERR_INVALID_ARG, "groups must be in 1 .. batch");
  if (!prefix->group_start || !prefix->prefix_len || !prefix->partial)
    return fail(kv, CONFKV_ERR_INVALID_ARG, "null group_start, prefix_len or partial");
  if (!aligned4(prefix->group_start) || !aligned4(prefix->prefix_len) || !aligned16(prefix->partial))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "group_start and prefix_len must be 4-byte aligned, partial 16-byte");
  if (rows == 0) return CONFKV_OK;
  const size_t np = partial_bytes(rows, p.Hq, p.d), nr = static_cast<size_t>(rows), wq = static_cast<size_t>(p.Hq) * p.d;
  if (prefix->partial_bytes < np) return fail(kv, CONFKV_ERR_CAPACITY, "partial is too small for the rows");
  if (overlap(prefix->partial, np, q, ((nr - 1) * q_stride + wq) * 2) || overlap(prefix->partial, np, out, nr * wq * 2) ||
      (lse && overlap(prefix->partial, np, lse, nr * p.Hq * 4)))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "partial overlaps q, out or lse");
  const size_t groups = static_cast<size_t>(prefix->groups);
  auto in_prefix = [&](const void* at, size_t n) {
    return overlap(at, n, prefix->group_start, (groups + 1) * 4) || overlap(at, n, prefix->prefix_len, groups * 4);
  };
  if (in_batch(batch, rows, prefix->partial, np) || in_prefix(prefix->partial, np) || in_prefix(out, nr * wq * 2) ||
      (lse && in_prefix(lse, nr * p.Hq * 4)))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "out, lse or partial overlaps the batch's or the prefix's tensors");
  DeviceGuard guard(kv->device);
  a.part = static_cast<float*>(prefix->partial);
  a.part_ml = a.part + nr * wq;
  a.bt.groups = prefix->groups;
  a.bt.group_start = prefix->group_start;
  a.bt.prefix_len = prefix->prefix_len;
  // the groups' rows over their prefixes, then each sequence's over the rest of its own
  AttendArgs shared = a;
  shared.bt.phase = 1;
  shared.bt.B = prefix->groups;
  shared.bt.mask = nullptr;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = attend(*kv, shared, prefix->groups, st);
  a.bt.phase = 2;
  if (e == cudaSuccess) e = attend(*kv, a, batch->batch, st);
  return launched(kv, e);
}

int confkv_paged_weigh(confkv_paged* kv, const confkv_paged_batch* batch, int layer, int rows, const void* q, int64_t q_stride,
                       const float* lse, const float* mass, float* mass_out, int32_t* pos, int cap, const int32_t* positions,
                       float decay, float gain, float scale, void* stream) {
  if (!kv) return CONFKV_ERR_INVALID_ARG;
  const Pool& p = kv->pool;
  if (const char* m = check_batch(batch, true)) return fail(kv, CONFKV_ERR_INVALID_ARG, m);
  if (layer < 0 || layer >= p.L) return fail(kv, CONFKV_ERR_INVALID_ARG, "no such layer");
  if (rows < 0) return fail(kv, CONFKV_ERR_INVALID_ARG, "rows < 0");
  if (static_cast<int64_t>(rows) * p.Hq >= (1ll << 31)) return fail(kv, CONFKV_ERR_INVALID_ARG, "rows x heads must be below 2^31");
  if (cap < 1) return fail(kv, CONFKV_ERR_INVALID_ARG, "cap must be positive");
  if (rows == 0) return CONFKV_OK;
  const int64_t wq = static_cast<int64_t>(p.Hq) * p.d;
  if (!q || !lse || !mass || !mass_out) return fail(kv, CONFKV_ERR_INVALID_ARG, "null q, lse, mass or mass_out");
  if (!aligned16(q) || !aligned4(lse) || !aligned4(mass) || !aligned4(mass_out) || !aligned4(pos) || !aligned4(positions))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "q must be 16-byte aligned, lse, mass, mass_out, pos and positions 4-byte");
  if (!good_stride(q_stride, wq)) return fail(kv, CONFKV_ERR_INVALID_ARG, "q_stride is below the row's width or no multiple of 8");
  if (!(scale >= 0.0f && std::isfinite(scale))) return fail(kv, CONFKV_ERR_INVALID_ARG, "scale must be finite and not negative");
  if (!std::isfinite(decay) || !std::isfinite(gain)) return fail(kv, CONFKV_ERR_INVALID_ARG, "decay and gain must be finite");
  const size_t nm = static_cast<size_t>(batch->batch) * p.Hkv * cap * 4, nr = static_cast<size_t>(rows);
  if (mass != mass_out && overlap(mass, nm, mass_out, nm))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "mass_out overlaps mass and is not mass itself");
  for (const void* out : {static_cast<const void*>(mass_out), static_cast<const void*>(pos)})
    if (out && (overlap(out, nm, q, ((nr - 1) * q_stride + wq) * 2) || overlap(out, nm, lse, nr * p.Hq * 4) ||
                (positions && overlap(out, nm, positions, nr * 4))))
      return fail(kv, CONFKV_ERR_INVALID_ARG, "mass_out or pos overlaps an input");
  if (in_batch(batch, rows, mass_out, nm) || (pos && in_batch(batch, rows, pos, nm)))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "mass_out or pos overlaps the batch's tensors");
  if (pos && (overlap(pos, nm, mass, nm) || overlap(pos, nm, mass_out, nm)))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "pos overlaps mass or mass_out");
  DeviceGuard guard(kv->device);
  const WeighArgs a{batch_of(batch), layer, rows, static_cast<const uint16_t*>(q), q_stride, lse, mass, mass_out, pos, cap,
                    positions, decay, gain, scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(p.d))};
  return launched(kv, launch_weigh(p, a, kv->maps, kv->limits.sms, static_cast<cudaStream_t>(stream)));
}

int confkv_paged_evict(confkv_paged* kv, int batch, int max_blocks, const int32_t* page_table, const int32_t* length,
                       int per_layer, const float* mass, const int32_t* pos, int cap, const int32_t* keep,
                       const int32_t* first, int protect, float* mass_out, int32_t* pos_out, int32_t* new_len, void* stream) {
  if (!kv) return CONFKV_ERR_INVALID_ARG;
  const Pool& p = kv->pool;
  if (batch < 0 || batch > 65536 || max_blocks < 1) return fail(kv, CONFKV_ERR_INVALID_ARG, "batch outside 0 .. 65536 or max_blocks < 1");
  if (cap < 1 || cap > kMaxEvictTokens) return fail(kv, CONFKV_ERR_INVALID_ARG, "cap must be in 1 .. 524288");
  if (protect < 0) return fail(kv, CONFKV_ERR_INVALID_ARG, "protect < 0");
  if (per_layer < 0 || per_layer > 1) return fail(kv, CONFKV_ERR_INVALID_ARG, "per_layer must be 0 or 1");
  if (static_cast<int64_t>(p.L) * batch * p.Hkv >= (1ll << 31)) return fail(kv, CONFKV_ERR_INVALID_ARG, "layers x batch x kv_heads must be below 2^31");
  if (batch == 0) return CONFKV_OK;
  if (!page_table || !length || !mass || !pos || !keep || !mass_out || !pos_out || !new_len)
    return fail(kv, CONFKV_ERR_INVALID_ARG, "null argument");
  if (!aligned4(page_table) || !aligned4(length) || !aligned4(mass) || !aligned4(pos) || !aligned4(keep) || !aligned4(first) ||
      !aligned4(mass_out) || !aligned4(pos_out) || !aligned4(new_len))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "arguments must be 4-byte aligned");
  const size_t nb = static_cast<size_t>(batch) * 4, ns = per_layer ? nb * p.L : nb;
  const size_t nm = static_cast<size_t>(p.L) * batch * p.Hkv * cap * 4;
  if ((mass == mass_out) != (pos == pos_out)) return fail(kv, CONFKV_ERR_INVALID_ARG, "mass and pos are kept in place both or neither");
  if (mass != mass_out && (overlap(mass, nm, mass_out, nm) || overlap(pos, nm, pos_out, nm)))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "an output overlaps its input and is not the input itself");
  struct Range {
    const void* at;
    size_t n;
  };
  const Range in[] = {{page_table, nb * max_blocks}, {length, ns}, {keep, ns}, {first, first ? nb : 0}},
              out[] = {{mass_out, nm}, {pos_out, nm}, {new_len, ns}};
  for (const Range& o : out)
    for (const Range& r : in)
      if (r.n && overlap(o.at, o.n, r.at, r.n)) return fail(kv, CONFKV_ERR_INVALID_ARG, "an output overlaps an input");
  if (overlap(mass_out, nm, pos_out, nm) || overlap(mass_out, nm, new_len, ns) || overlap(pos_out, nm, new_len, ns) ||
      overlap(mass_out, nm, pos, nm) || overlap(pos_out, nm, mass, nm) || overlap(new_len, ns, mass, nm) || overlap(new_len, ns, pos, nm))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "outputs overlap one another or an input");
  DeviceGuard guard(kv->device);
  const EvictArgs a{batch, max_blocks, cap, protect, per_layer, page_table, length, keep, first, mass, pos, mass_out, pos_out, new_len};
  return launched(kv, launch_evict(p, a, kv->limits.sms, static_cast<cudaStream_t>(stream)));
}

int confkv_paged_commit(confkv_paged* kv, int batch, int max_blocks, const int32_t* page_table,
                        const int32_t* ctx_len, const int32_t* path, int path_cap, const int32_t* path_len,
                        int32_t* new_len, void* stream) {
  if (!kv) return CONFKV_ERR_INVALID_ARG;
  if (batch < 0 || max_blocks < 1 || path_cap < 1 || path_cap > 1024)
    return fail(kv, CONFKV_ERR_INVALID_ARG, "batch < 0, max_blocks < 1 or path_cap outside 1 .. 1024");
  if (batch == 0) return CONFKV_OK;
  if (!page_table || !ctx_len || !path || !path_len || !new_len) return fail(kv, CONFKV_ERR_INVALID_ARG, "null argument");
  if (!aligned4(page_table) || !aligned4(ctx_len) || !aligned4(path) || !aligned4(path_len) || !aligned4(new_len))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "arguments must be 4-byte aligned");
  const size_t n = static_cast<size_t>(batch) * 4;
  if (overlap(new_len, n, ctx_len, n) || overlap(new_len, n, path_len, n) || overlap(new_len, n, path, n * path_cap) ||
      overlap(new_len, n, page_table, n * max_blocks))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "new_len overlaps an input");
  DeviceGuard guard(kv->device);
  const CommitArgs a{batch, max_blocks, path_cap, page_table, ctx_len, path, path_len, new_len};
  return launched(kv, launch_commit(kv->pool, a, static_cast<cudaStream_t>(stream)));
}

int confkv_paged_fork(confkv_paged* kv, int rows, int beams, int max_blocks, const int32_t* parent,
                      const int32_t* table_in, const int32_t* len_in, const int32_t* tail_pages,
                      int32_t* table_out, int32_t* len_out, void* stream) {
  if (!kv) return CONFKV_ERR_INVALID_ARG;
  if (rows < 0 || beams < 1 || rows % beams || max_blocks < 1)
    return fail(kv, CONFKV_ERR_INVALID_ARG, "rows must be a multiple of beams >= 1, max_blocks positive");
  if (rows == 0) return CONFKV_OK;
  if (!parent || !table_in || !len_in || !tail_pages || !table_out || !len_out)
    return fail(kv, CONFKV_ERR_INVALID_ARG, "null argument");
  if (!aligned4(parent) || !aligned4(table_in) || !aligned4(len_in) || !aligned4(tail_pages) || !aligned4(table_out) ||
      !aligned4(len_out))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "arguments must be 4-byte aligned");
  const size_t n = static_cast<size_t>(rows) * 4, nt = n * max_blocks;
  for (const int32_t* in : {parent, len_in, tail_pages})
    if (overlap(table_out, nt, in, n) || overlap(len_out, n, in, n))
      return fail(kv, CONFKV_ERR_INVALID_ARG, "an output overlaps an input");
  if (overlap(table_out, nt, table_in, nt) || overlap(len_out, n, table_in, nt) || overlap(table_out, nt, len_out, n))
    return fail(kv, CONFKV_ERR_INVALID_ARG, "an output overlaps an input or the other output");
  DeviceGuard guard(kv->device);
  const ForkArgs a{rows, beams, max_blocks, parent, table_in, len_in, tail_pages, table_out, len_out};
  return launched(kv, launch_fork(kv->pool, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {
bool beam_sizes(int batch, int beams, int vocab, int keep, int dtype) {
  return batch >= 1 && beams >= 1 && beams <= 32 && static_cast<long long>(batch) * beams <= 65535 && vocab >= 2 &&
         vocab <= (1 << 24) && keep >= 1 && keep <= 64 && dtype >= CONFKV_FP16 && dtype <= CONFKV_FP32;
}
}  // namespace

extern "C" {

size_t confkv_beam_workspace(int batch, int beams, int vocab, int keep, int dtype) {
  return beam_sizes(batch, beams, vocab, keep, dtype) ? beam_workspace(batch, beams, vocab, keep, dtype) : 0;
}

int confkv_beam_select(const void* logits, int dtype, int64_t row_stride, int batch, int beams, int vocab, int keep,
                       const float* scores, const uint8_t* finished, int pad_token, float* score_out,
                       int32_t* parent_out, int32_t* token_out, int32_t* flags_out, void* workspace,
                       size_t workspace_bytes, int device, void* stream) {
  if (!beam_sizes(batch, beams, vocab, keep, dtype) || !logits || !scores || !score_out || !parent_out || !token_out ||
      !workspace || row_stride < vocab || row_stride >= (1ll << 40) || pad_token < 0 || pad_token >= vocab)
    return CONFKV_ERR_INVALID_ARG;
  const uintptr_t elem = dtype == CONFKV_FP32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(logits) & elem) || !aligned4(scores) || !aligned4(score_out) ||
      !aligned4(parent_out) || !aligned4(token_out) || !aligned4(flags_out) || !aligned16(workspace))
    return CONFKV_ERR_INVALID_ARG;
  if (workspace_bytes < beam_workspace(batch, beams, vocab, keep, dtype)) return CONFKV_ERR_CAPACITY;
  // every input is read until the last row is done: no output may lie in one
  struct Range {
    const void* at;
    size_t n;
  };
  const size_t rows = static_cast<size_t>(batch) * beams, no = static_cast<size_t>(batch) * keep * 4;
  const Range in[] = {{scores, rows * 4}, {finished, finished ? rows : 0}, {workspace, workspace_bytes},
                      {logits, ((rows - 1) * row_stride + vocab) * (elem + 1)}},
              out[] = {{score_out, no}, {parent_out, no}, {token_out, no}, {flags_out, flags_out ? rows * 4 : 0}};
  for (int i = 0; i < 4; ++i) {
    for (const Range& r : in)
      if (out[i].n && r.n && overlap(out[i].at, out[i].n, r.at, r.n)) return CONFKV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (out[i].n && overlap(out[i].at, out[i].n, out[j].at, out[j].n)) return CONFKV_ERR_INVALID_ARG;
  }
  const BeamArgs a{logits, dtype, row_stride, batch, beams, vocab, keep, scores, finished, pad_token, score_out,
                   parent_out, token_out, flags_out, workspace};
  DeviceGuard guard(device);
  return launch_beam(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CONFKV_OK : CONFKV_ERR_CUDA;
}

}  // extern "C"
