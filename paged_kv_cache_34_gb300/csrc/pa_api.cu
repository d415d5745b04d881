// pa_api.cu -- the extern "C" entry points declared in include/pa.h.
//
// Host-side only: argument validation, the split-KV plan, TMA tensor-map
// encoding, and kernel launches on the caller's stream.  Nothing here
// allocates device memory, synchronises, or reads device data.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "pa.h"
#include "pa_internal.h"

namespace {

thread_local int32_t g_last_cuda_error = 0;

pa_status cuda_fail(cudaError_t e) {
  g_last_cuda_error = static_cast<int32_t>(e);
  return PA_ERR_CUDA;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ---- device properties, cached per device ---------------------------------
constexpr int kMaxDevices = 64;
int g_num_sms[kMaxDevices] = {0};

cudaError_t current_num_sms(int *out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDevices && g_num_sms[dev] > 0) {
    *out = g_num_sms[dev];
    return cudaSuccess;
  }
  int n = 0;
  e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDevices) g_num_sms[dev] = n;
  *out = n;
  return cudaSuccess;
}

// ---- cuTensorMapEncodeTiled through the runtime's driver entry point -----
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::once_flag g_encode_once;
EncodeTiledFn g_encode = nullptr;

EncodeTiledFn encode_fn() {
  std::call_once(g_encode_once, [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  });
  return g_encode;
}

// A 3-D map over rows of `heads` x `head_dim` 16-bit elements:
//   dim0 = head_dim (contiguous), dim1 = heads, dim2 = rows,
// with `row_stride` elements between rows; box (64, 1, box_rows) and
// 128-byte swizzle (the box's 64 elements are exactly one 128-byte line).
// A pool viewed as [rows, heads, head_dim] for TMA: boxes of 128 bytes of one
// head's row (64 16-bit elements, or 128 int8 codes) by box_rows rows, with
// the 128-byte swizzle the kernels' shared-memory reads expect.
// One-byte pools: boxes of one head's whole row (head_dim codes), with the
// 64-byte swizzle at head_dim 64.
bool encode_rows_map(CUtensorMap *map, const void *base, pa_dtype dtype, int head_dim,
                     int heads, int64_t rows, int64_t row_stride, int box_rows,
                     bool int8 = false, int box_heads = 1) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t eb = int8 ? 1 : 2;  // element bytes
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * eb,
                                 static_cast<cuuint64_t>(row_stride) * eb};
  const cuuint32_t box[3] = {int8 ? static_cast<cuuint32_t>(head_dim) : 64u,
                             static_cast<cuuint32_t>(box_heads),
                             static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = int8               ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle sw =
      int8 && head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  CUresult r = enc(map, dt, 3, const_cast<void *>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool valid_block_size(int bs) { return bs == 8 || bs == 16 || bs == 32 || bs == 64 || bs == 128; }

// The factor of the flash engine's scores: |scale| log2 e, and whether Q enters
// the product negated.  It has to be positive, so that a masked score (-inf)
// times it stays -inf: at scale 0 the query tiles are taken from behind the last
// row instead (q_off rows on), where TMA reads zeros, and every score is 0.
void flash_scale(float scale, int32_t rows, float *scale_log2, bool *negate, int32_t *q_off) {
  const double f = fabs(static_cast<double>(scale)) * 1.4426950408889634;
  *scale_log2 = scale == 0.0f ? 1.0f : static_cast<float>(f);  // > 0: f rounds up from 2^-149
  *negate = scale < 0.0f;
  *q_off = scale == 0.0f ? rows : 0;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The automatic plan is the balanced split, as long as its positions fit in
// int32 (else fixed partitions sized by plan_partition); `units` = decode
// units (KV-head slices) per sequence.
bool use_balanced(int num_seqs, int units, int max_ctx, int partition_size) {
  if (partition_size != 0 || max_ctx <= 0) return false;
  const int64_t t = static_cast<int64_t>(num_seqs) * units * ((max_ctx + 15) / 16) * 16;
  return t < (1LL << 30);
}

// Fixed split-KV plan.  Auto: every worker warp (kDecodeWarps per CTA,
// kDecodeCtasPerSm CTAs per SM) should get about eight items of the largest
// possible batch, so the static item schedule balances; a partition is at least
// 64 tokens (128 when eight query heads share a KV head) so the partial states
// stay a few percent of the K/V bytes.
int plan_partition(int num_seqs, int num_q_heads, int num_kv_heads, int max_ctx,
                   int partition_size, int num_sms) {
  if (partition_size > 0) return partition_size;
  const long units = static_cast<long>(num_seqs > 0 ? num_seqs : 1) * num_kv_heads *
                     pa::decode_slices(num_q_heads / num_kv_heads).nc;
  const long target_items =
      static_cast<long>(num_sms) * pa::kDecodeCtasPerSm * pa::kDecodeWarps * 8;
  long P = (units * max_ctx + target_items - 1) / target_items;
  P = ((P + pa::kDecodeSub - 1) / pa::kDecodeSub) * pa::kDecodeSub;
  const long pmin = (num_q_heads / num_kv_heads) > 4 ? 128 : 64;
  if (P < pmin) P = pmin;
  if (P > (1 << 20)) P = 1 << 20;
  return static_cast<int>(P);
}

}  // namespace

namespace pa {
void record_cuda_error(cudaError_t e) { g_last_cuda_error = static_cast<int32_t>(e); }

constexpr uint64_t kDefaultWaitNs = 2000000000ull;  // 2 s
std::atomic<uint64_t> g_wait_ns{kDefaultWaitNs};
uint64_t pipeline_wait_ns() { return g_wait_ns.load(std::memory_order_relaxed); }
}  // namespace pa

extern "C" {

int32_t pa_abi_version(void) { return PA_ABI_VERSION; }

int32_t pa_last_cuda_error(void) { return g_last_cuda_error; }

void pa_debug_set_wait_limit_ns(uint64_t ns) {
  pa::g_wait_ns.store(ns ? ns : pa::kDefaultWaitNs, std::memory_order_relaxed);
}

const char *pa_status_string(pa_status s) {
  switch (s) {
    case PA_OK: return "PA_OK";
    case PA_ERR_NULL: return "PA_ERR_NULL: a required pointer is NULL";
    case PA_ERR_SHAPE: return "PA_ERR_SHAPE: inconsistent sizes or strides";
    case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED: configuration not built";
    case PA_ERR_ALIGN: return "PA_ERR_ALIGN: pointer not 16-byte aligned or stride not x8";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE: workspace missing or too small";
    case PA_ERR_CUDA: return "PA_ERR_CUDA: a CUDA runtime call failed";
  }
  return "unknown pa_status";
}

}  // extern "C"

namespace {

// Validates a cache write and fills its launch arguments; enqueues nothing.
// *empty is set when there is nothing to write.
pa_status prepare_write(const void *key, const void *value, int64_t kv_row_stride,
                        void *key_cache, void *value_cache, const int64_t *slot_mapping,
                        int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                        int32_t block_size, int64_t num_blocks, pa_dtype dtype, int32_t *d_error,
                        pa::ReshapeArgs *out, bool *empty) {
  *empty = true;
  if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0)
    return PA_ERR_SHAPE;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (!key_cache || !value_cache) return PA_ERR_NULL;
  if (num_tokens == 0) return PA_OK;
  if (!key || !value || !slot_mapping) return PA_ERR_NULL;
  const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (kv_row_stride < row) return PA_ERR_SHAPE;
  if ((row * 2) % 16 != 0 || kv_row_stride % 8 != 0) return PA_ERR_ALIGN;
  if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache))
    return PA_ERR_ALIGN;
  pa::ReshapeArgs a;
  a.key = key;
  a.value = value;
  a.row_stride_bytes = kv_row_stride * 2;
  a.key_cache = key_cache;
  a.value_cache = value_cache;
  a.slot_mapping = slot_mapping;
  a.num_tokens = num_tokens;
  a.row_bytes = row * 2;
  a.num_slots = num_blocks * block_size;
  a.d_error = d_error;
  a.num_sms = 0;  // filled in at launch
  *out = a;
  *empty = false;
  return PA_OK;
}

// The write into 8-bit pools (INT8, or E4M3 with fp8).
pa_status write_8bit(const void *key, const void *value, int64_t kv_row_stride, void *key_cache,
                     void *value_cache, const int64_t *slot_mapping, int32_t num_tokens,
                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                     int64_t num_blocks, const float *k_scale, const float *v_scale,
                     pa_dtype dtype, int32_t *d_error, void *stream, bool fp8) {
  pa::ReshapeArgs w;
  bool empty = true;
  const pa_status st = prepare_write(key, value, kv_row_stride, key_cache, value_cache,
                                     slot_mapping, num_tokens, num_kv_heads, head_dim, block_size,
                                     num_blocks, dtype, d_error, &w, &empty);
  if (st != PA_OK) return st;
  if (!k_scale || !v_scale) return PA_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3u)
    return PA_ERR_ALIGN;
  // int8 pool rows in 16-byte chunks, a chunk within one head
  if (head_dim % 16 != 0) return PA_ERR_ALIGN;
  if (empty) return PA_OK;
  w.int8 = true;
  w.fp8 = fp8;
  w.dtype = dtype;
  w.head_dim = head_dim;
  w.k_scale = k_scale;
  w.v_scale = v_scale;
  cudaError_t e = current_num_sms(&w.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  e = pa::launch_reshape_and_cache(w, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

pa_status pa_reshape_and_cache(const void *key, const void *value, int64_t kv_row_stride,
                               void *key_cache, void *value_cache,
                               const int64_t *slot_mapping, int32_t num_tokens,
                               int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                               int64_t num_blocks, pa_dtype dtype, int32_t *d_error,
                               void *stream) {
  pa::ReshapeArgs w;
  bool empty = true;
  const pa_status st = prepare_write(key, value, kv_row_stride, key_cache, value_cache,
                                     slot_mapping, num_tokens, num_kv_heads, head_dim, block_size,
                                     num_blocks, dtype, d_error, &w, &empty);
  if (st != PA_OK || empty) return st;
  cudaError_t e = current_num_sms(&w.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  e = pa::launch_reshape_and_cache(w, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_rope_and_cache(void *query_out, int64_t q_out_row_stride, void *key_out,
                            int64_t k_out_row_stride, const void *query, int64_t q_row_stride,
                            const void *key, const void *value, int64_t kv_row_stride,
                            const int32_t *positions, const float *cos_sin, int64_t max_position,
                            int32_t rot_dim, int32_t interleaved, const void *q_weight,
                            const void *k_weight, float eps, void *key_cache, void *value_cache,
                            const int64_t *slot_mapping, int32_t num_tokens, int32_t num_q_heads,
                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                            int64_t num_blocks, pa_dtype dtype, int32_t *d_error, void *stream) {
  const bool cache = key_cache || value_cache || slot_mapping;
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || rot_dim < 0 ||
      rot_dim > head_dim || max_position < 0 || !(eps >= 0.0f) || !isfinite(eps))
    return PA_ERR_SHAPE;
  if (cache && (block_size <= 0 || num_blocks < 0 || num_blocks > INT64_MAX / block_size))
    return PA_ERR_SHAPE;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (rot_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
  if (num_q_heads > 65536 || num_kv_heads > 65536) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!query_out || !query || !key || (!cache && !key_out)) return PA_ERR_NULL;
  if (cache && (!key_cache || !value_cache || !slot_mapping || !value)) return PA_ERR_NULL;
  if (rot_dim > 0 && (!positions || !cos_sin)) return PA_ERR_NULL;
  const int64_t qrow = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t krow = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_row_stride < qrow || q_out_row_stride < qrow || kv_row_stride < krow ||
      (key_out && k_out_row_stride < krow))
    return PA_ERR_SHAPE;
  // byte offsets of every row fit in 64 bits
  const int64_t most = INT64_MAX / 4 / num_tokens;
  if (q_row_stride > most || q_out_row_stride > most || kv_row_stride > most ||
      (key_out && k_out_row_stride > most))
    return PA_ERR_SHAPE;
  if (q_row_stride % 8 || q_out_row_stride % 8 || kv_row_stride % 8 ||
      (key_out && k_out_row_stride % 8))
    return PA_ERR_ALIGN;
  if (!aligned16(query_out) || !aligned16(key_out) || !aligned16(query) || !aligned16(key) ||
      (cache && (!aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache))) ||
      !aligned16(q_weight) || !aligned16(k_weight) || (rot_dim && !aligned16(cos_sin)))
    return PA_ERR_ALIGN;
  if ((rot_dim && (reinterpret_cast<uintptr_t>(positions) & 3u)) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PA_ERR_ALIGN;
  // A row may be rewritten in place (same rows, same stride); other overlaps of
  // rows that are read and rows that are written are refused.
  struct Rows {
    const void *p;
    int64_t stride, row;
  };
  const int64_t last = num_tokens - 1;
  auto apart = [&](const Rows &x, const Rows &y, bool in_place) {
    if (!x.p || !y.p) return true;
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    const uintptr_t ae = a + 2 * (last * x.stride + x.row), be = b + 2 * (last * y.stride + y.row);
    if (a >= be || b >= ae) return true;
    if (x.stride != y.stride && num_tokens > 1) return false;
    if (in_place && a == b) return true;
    // views side by side in the rows of one buffer
    const uintptr_t s = 2 * static_cast<uintptr_t>(x.stride);
    if (num_tokens == 1) return false;
    const uintptr_t d = a < b ? (b - a) % s : s - (a - b) % s;  // y's columns behind x's
    return d >= 2 * static_cast<uintptr_t>(x.row) && d + 2 * static_cast<uintptr_t>(y.row) <= s;
  };
  const Rows q_in = {query, q_row_stride, qrow}, k_in = {key, kv_row_stride, krow};
  const Rows v_in = {cache ? value : nullptr, kv_row_stride, krow};
  const Rows q_o = {query_out, q_out_row_stride, qrow}, k_o = {key_out, k_out_row_stride, krow};
  if (!apart(q_in, q_o, true) || !apart(k_in, k_o, true) || !apart(q_in, k_o, false) ||
      !apart(k_in, q_o, false) || !apart(v_in, q_o, false) || !apart(v_in, k_o, false) ||
      !apart(q_o, k_o, false))
    return PA_ERR_SHAPE;
  // the other inputs, wherever they lie between the first and the last byte of the rows written
  struct Range {
    const void *p;
    uint64_t bytes;
  };
  const uint64_t n = num_tokens, weight = 2ull * head_dim;
  const uint64_t most_table = UINT64_MAX / 4 / (rot_dim ? rot_dim : 1);
  const Range other[] = {{positions, rot_dim ? 4 * n : 0},
                         {cos_sin, 4 * static_cast<uint64_t>(rot_dim) *
                                       (static_cast<uint64_t>(max_position) < most_table
                                            ? static_cast<uint64_t>(max_position)
                                            : most_table)},
                         {q_weight, q_weight ? weight : 0},
                         {k_weight, k_weight ? weight : 0},
                         {slot_mapping, cache ? 8 * n : 0}};
  for (const Rows &x : {q_o, k_o}) {
    if (!x.p) continue;
    const uintptr_t b = reinterpret_cast<uintptr_t>(x.p);
    const uintptr_t e = b + 2 * (last * x.stride + x.row);
    for (const Range &y : other) {
      const uintptr_t c = reinterpret_cast<uintptr_t>(y.p);
      if (y.bytes > 0 && c < e && (b < c || b - c < y.bytes)) return PA_ERR_SHAPE;
    }
  }
  pa::RopeArgs a;
  a.query_out = query_out;
  a.key_out = key_out;
  a.q_out_row_stride = q_out_row_stride;
  a.k_out_row_stride = k_out_row_stride;
  a.query = query;
  a.key = key;
  a.value = value;
  a.q_row_stride = q_row_stride;
  a.kv_row_stride = kv_row_stride;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.max_position = max_position;
  a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.key_cache = key_cache;
  a.value_cache = value_cache;
  a.slot_mapping = slot_mapping;
  a.num_slots = cache ? num_blocks * block_size : 0;
  a.num_tokens = num_tokens;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.dtype = dtype;
  a.d_error = d_error;
  cudaError_t e = current_num_sms(&a.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  e = pa::launch_rope_and_cache(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_copy_blocks(void *key_cache, void *value_cache, int64_t block_bytes,
                         int64_t num_blocks, const int64_t *block_mapping, int32_t num_pairs,
                         int32_t *d_error, void *stream) {
  if (num_pairs < 0 || num_blocks < 0 || block_bytes <= 0) return PA_ERR_SHAPE;
  if (!key_cache || !value_cache) return PA_ERR_NULL;
  if (block_bytes % 16 != 0 || !aligned16(key_cache) || !aligned16(value_cache))
    return PA_ERR_ALIGN;
  if (num_pairs == 0) return PA_OK;
  if (!block_mapping) return PA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(block_mapping) & 7u) return PA_ERR_ALIGN;
  pa::CopyBlocksArgs a;
  a.key_cache = key_cache;
  a.value_cache = value_cache;
  a.block_bytes = block_bytes;
  a.num_blocks = num_blocks;
  a.block_mapping = block_mapping;
  a.num_pairs = num_pairs;
  a.d_error = d_error;
  cudaError_t e = current_num_sms(&a.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  e = pa::launch_copy_blocks(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_build_tables(int32_t *block_table, int64_t block_table_stride,
                          int32_t max_blocks_per_seq, const int32_t *context_lens,
                          const int32_t *query_lens, const int32_t *free_blocks,
                          const int32_t *num_free, int32_t free_capacity,
                          int32_t *context_lens_out, int32_t *cu_seqlens_q,
                          int64_t *slot_mapping, int32_t *positions, int32_t *num_free_out,
                          int32_t num_seqs, int32_t max_tokens, int32_t block_size,
                          int64_t num_blocks, int32_t *d_error, void *stream) {
  if (num_seqs < 0 || max_tokens < 0 || max_blocks_per_seq < 0 || free_capacity < 0 ||
      num_blocks < 0 || block_size <= 0)
    return PA_ERR_SHAPE;
  if (block_table_stride < max_blocks_per_seq) return PA_ERR_SHAPE;
  if (!valid_block_size(block_size)) return PA_ERR_UNSUPPORTED;
  if (!cu_seqlens_q || !num_free || !num_free_out) return PA_ERR_NULL;
  if (num_seqs > 0 && (!context_lens || !query_lens || !context_lens_out)) return PA_ERR_NULL;
  if (num_seqs > 0 && max_blocks_per_seq > 0 && !block_table) return PA_ERR_NULL;
  if (free_capacity > 0 && !free_blocks) return PA_ERR_NULL;
  if (max_tokens > 0 && !slot_mapping) return PA_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(context_lens) |
       reinterpret_cast<uintptr_t>(query_lens) | reinterpret_cast<uintptr_t>(free_blocks) |
       reinterpret_cast<uintptr_t>(num_free) | reinterpret_cast<uintptr_t>(context_lens_out) |
       reinterpret_cast<uintptr_t>(cu_seqlens_q) | reinterpret_cast<uintptr_t>(positions) |
       reinterpret_cast<uintptr_t>(num_free_out)) & 3u)
    return PA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) return PA_ERR_ALIGN;
  // Every CTA reads the inputs while others write.  (The block table is both:
  // entries that are read are not written.)
  struct Range {
    const void *p;
    int64_t bytes;
  };
  const int64_t seqs = num_seqs;
  const Range table = {block_table, seqs > 0 && max_blocks_per_seq > 0
                                        ? ((seqs - 1) * block_table_stride + max_blocks_per_seq) * 4
                                        : 0};
  const Range in[] = {{context_lens, seqs * 4}, {query_lens, seqs * 4},
                      {free_blocks, free_capacity * 4LL}, {num_free, 4}, table};
  const Range written[] = {{context_lens_out, seqs * 4}, {cu_seqlens_q, (seqs + 1) * 4},
                           {slot_mapping, max_tokens * 8LL},
                           {positions, positions ? max_tokens * 4LL : 0}, {num_free_out, 4}};
  auto overlaps = [](const Range &x, const Range &y) {
    const char *a = static_cast<const char *>(x.p), *b = static_cast<const char *>(y.p);
    return x.bytes > 0 && y.bytes > 0 && a < b + y.bytes && b < a + x.bytes;
  };
  for (const Range &x : in) {
    for (const Range &y : written)
      if (overlaps(x, y)) return PA_ERR_SHAPE;
    if (&x != in + 4 && overlaps(x, table)) return PA_ERR_SHAPE;
  }
  pa::BuildTablesArgs a;
  a.block_table = block_table;
  a.block_table_stride = block_table_stride;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.context_lens = context_lens;
  a.query_lens = query_lens;
  a.free_blocks = free_blocks;
  a.num_free = num_free;
  a.free_capacity = free_capacity;
  a.context_lens_out = context_lens_out;
  a.cu_seqlens_q = cu_seqlens_q;
  a.slot_mapping = slot_mapping;
  a.positions = positions;
  a.num_free_out = num_free_out;
  a.num_seqs = num_seqs;
  a.max_tokens = max_tokens;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.d_error = d_error;
  cudaError_t e = current_num_sms(&a.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  e = pa::launch_build_tables(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_reshape_and_cache_int8(const void *key, const void *value, int64_t kv_row_stride,
                                    void *key_cache, void *value_cache,
                                    const int64_t *slot_mapping, int32_t num_tokens,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                    int64_t num_blocks, const float *k_scale,
                                    const float *v_scale, pa_dtype dtype, int32_t *d_error,
                                    void *stream) {
  return write_8bit(key, value, kv_row_stride, key_cache, value_cache, slot_mapping, num_tokens,
                    num_kv_heads, head_dim, block_size, num_blocks, k_scale, v_scale, dtype,
                    d_error, stream, false);
}

pa_status pa_reshape_and_cache_fp8(const void *key, const void *value, int64_t kv_row_stride,
                                   void *key_cache, void *value_cache,
                                   const int64_t *slot_mapping, int32_t num_tokens,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                   int64_t num_blocks, const float *k_scale,
                                   const float *v_scale, pa_dtype dtype, int32_t *d_error,
                                   void *stream) {
  return write_8bit(key, value, kv_row_stride, key_cache, value_cache, slot_mapping, num_tokens,
                    num_kv_heads, head_dim, block_size, num_blocks, k_scale, v_scale, dtype,
                    d_error, stream, true);
}

pa_status pa_decode_plan(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_dim, int32_t max_context_len, int32_t partition_size,
                         int32_t *partition_size_out, size_t *workspace_bytes_out) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_context_len < 0 || partition_size < 0)
    return PA_ERR_SHAPE;
  if (partition_size % pa::kDecodeSub != 0) return PA_ERR_SHAPE;
  int sms = 0;
  cudaError_t e = current_num_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  size_t ws = 0;
  int P = 0;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_SHAPE;
  const pa::DecodeSlices sl = pa::decode_slices(num_q_heads / num_kv_heads);
  if (use_balanced(num_seqs, num_kv_heads * sl.nc, max_context_len, partition_size)) {
    // Balanced split (P reported as 0): pieces x (heads per slice) rows of
    // partial state, plus the per-sequence prefix sums for the merge kernel.
    const pa::DecodeBalance d =
        pa::decode_balance(num_seqs, num_kv_heads * sl.nc, max_context_len, sms);
    const size_t rows = static_cast<size_t>(d.pieces) * sl.hs;
    ws = align256(rows * head_dim * sizeof(float)) + align256(rows * 2 * sizeof(float)) +
         align256((static_cast<size_t>(num_seqs) + 1) * sizeof(int32_t));
  } else {
    P = plan_partition(num_seqs, num_q_heads, num_kv_heads, max_context_len, partition_size,
                       sms);
    const int64_t nparts = max_context_len > 0 ? (max_context_len + P - 1) / P : 1;
    if (nparts > 1) {
      const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * nparts;
      ws = align256(rows * head_dim * sizeof(float)) + align256(rows * 2 * sizeof(float));
    }
  }
  if (partition_size_out) *partition_size_out = P;
  if (workspace_bytes_out) *workspace_bytes_out = ws;
  return PA_OK;
}

}  // extern "C"

namespace {

// The checks of a decode's arguments and the launch arguments that follow
// from them alone; `empty`: no sequence to attend for.
struct DecodeSetup {
  bool empty = true;
  pa::DecodeArgs args;
};
pa_status check_decode(void *out, int64_t out_row_stride, const void *query, int64_t q_row_stride,
                       const void *key_cache, const void *value_cache, const int32_t *block_table,
                       int64_t block_table_stride, int32_t max_blocks_per_seq,
                       const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
                       int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                       int64_t num_blocks, float scale, int32_t max_context_len,
                       int32_t partition_size, pa_dtype dtype, DecodeSetup *setup) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq < 0 || max_context_len < 0 ||
      partition_size < 0)
    return PA_ERR_SHAPE;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_SHAPE;
  if (block_table_stride < max_blocks_per_seq) return PA_ERR_SHAPE;
  if (!isfinite(scale)) return PA_ERR_SHAPE;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (!valid_block_size(block_size)) return PA_ERR_UNSUPPORTED;
  if (num_blocks * block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
  // elements within a query's row are 32-bit
  if (static_cast<int64_t>(num_q_heads) * head_dim > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (partition_size % pa::kDecodeSub != 0) return PA_ERR_SHAPE;
  setup->empty = num_seqs == 0;
  if (num_seqs == 0) return PA_OK;
  if (!out || !query || !key_cache || !value_cache || !block_table || !context_lens)
    return PA_ERR_NULL;
  const int64_t qrow = static_cast<int64_t>(num_q_heads) * head_dim;
  if (q_row_stride < qrow || out_row_stride < qrow) return PA_ERR_SHAPE;
  if (q_row_stride % 8 || out_row_stride % 8) return PA_ERR_ALIGN;
  if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache))
    return PA_ERR_ALIGN;
  pa::DecodeArgs &a = setup->args;
  a.out = out;
  a.out_row_stride = out_row_stride;
  a.query = query;
  a.q_row_stride = q_row_stride;
  a.block_table = block_table;
  a.block_table_stride = block_table_stride;
  const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
  a.capacity = static_cast<int32_t>(cap > INT32_MAX ? INT32_MAX : cap);
  a.context_lens = context_lens;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.max_context_len = max_context_len;
  a.ws_o = nullptr;
  a.ws_ml = nullptr;
  a.ws_pref = nullptr;
  a.slices = pa::decode_slices(num_q_heads / num_kv_heads);
  a.dtype = dtype;
  a.box_rows = block_size < pa::kDecodeSub ? block_size : pa::kDecodeSub;
  return PA_OK;
}

// The balanced split's launch shape (num_sms known) and its workspace.
void set_balanced(pa::DecodeArgs *a, void *workspace) {
  const pa::DecodeBalance d = pa::decode_balance(
      a->num_seqs, a->num_kv_heads * a->slices.nc, a->max_context_len, a->num_sms);
  a->partition_size = 0;
  a->num_partitions = 0;
  a->grid = d.grid;
  a->merge = true;
  const size_t rows = static_cast<size_t>(d.pieces) * a->slices.hs;
  char *w = static_cast<char *>(workspace);
  a->ws_o = reinterpret_cast<float *>(w);
  w += align256(rows * a->head_dim * sizeof(float));
  a->ws_ml = reinterpret_cast<float *>(w);
  w += align256(rows * 2 * sizeof(float));
  a->ws_pref = reinterpret_cast<int32_t *>(w);
}

// pa_decode, optionally preceded by the step's cache write `write` (launched
// first, after every check has passed, so an error enqueues nothing).
pa_status decode_call(void *out, int64_t out_row_stride, const void *query, int64_t q_row_stride,
                      const void *key_cache, const void *value_cache, const int32_t *block_table,
                      int64_t block_table_stride, int32_t max_blocks_per_seq,
                      const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
                      int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                      int64_t num_blocks, float scale, int32_t max_context_len,
                      int32_t partition_size, void *workspace, size_t workspace_bytes,
                      pa_dtype dtype, int32_t *d_error, void *stream,
                      const pa::ReshapeArgs *write, const float *k_scale = nullptr,
                      const float *v_scale = nullptr, bool fp8 = false) {
  const bool int8 = k_scale != nullptr || v_scale != nullptr;
  DecodeSetup setup;
  pa_status st = check_decode(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                              block_table, block_table_stride, max_blocks_per_seq, context_lens,
                              num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                              num_blocks, scale, max_context_len, partition_size, dtype, &setup);
  if (st != PA_OK) return st;
  if (setup.empty) {  // nothing to attend: only the step's write, if any
    if (!write) return PA_OK;
    pa::ReshapeArgs w = *write;
    cudaError_t e = current_num_sms(&w.num_sms);
    if (e == cudaSuccess) e = pa::launch_reshape_and_cache(w, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
  }
  if (int8) {
    if (!k_scale || !v_scale) return PA_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3u)
      return PA_ERR_ALIGN;
  }

  int32_t P = 0;
  size_t need = 0;
  st = pa_decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                      partition_size, &P, &need);
  if (st != PA_OK) return st;
  const bool balanced = P == 0;
  const int32_t nparts = balanced ? 0 : (max_context_len > 0 ? (max_context_len + P - 1) / P : 1);
  if (need > 0 && (!workspace || workspace_bytes < need ||
                   (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
    return PA_ERR_WORKSPACE;

  pa::DecodeArgs &a = setup.args;
  a.partition_size = P;
  a.num_partitions = nparts;
  const int units = num_kv_heads * a.slices.nc;  // decode units per sequence
  cudaError_t e = current_num_sms(&a.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  if (balanced) {
    set_balanced(&a, workspace);
  } else {
    // Items are at most S * units * partitions; kDecodeCtasPerSm CTAs per SM,
    // kDecodeWarps workers each.
    const int64_t items = static_cast<int64_t>(num_seqs) * units * nparts;
    int64_t grid = (items + pa::kDecodeWarps - 1) / pa::kDecodeWarps;
    if (grid > static_cast<int64_t>(pa::kDecodeCtasPerSm) * a.num_sms)
      grid = static_cast<int64_t>(pa::kDecodeCtasPerSm) * a.num_sms;
    if (grid < 1) grid = 1;
    a.grid = static_cast<int>(grid);
    a.merge = nparts > 1;
    if (need > 0) {
      const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * nparts;
      a.ws_o = static_cast<float *>(workspace);
      a.ws_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                          align256(rows * head_dim * sizeof(float)));
    }
  }
  a.d_error = d_error;
  a.wait_ns = pa::pipeline_wait_ns();
  // The item schedule keeps per-sequence prefix sums in shared memory.
  if (pa::decode_smem_bytes(head_dim, num_seqs, P, block_size, int8) > 227 * 1024)
    return PA_ERR_UNSUPPORTED;
  const int64_t rows = num_blocks * block_size;
  const int64_t row_stride = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (!encode_rows_map(&a.tm_k, key_cache, dtype, head_dim, num_kv_heads, rows, row_stride,
                       a.box_rows, int8) ||
      !encode_rows_map(&a.tm_v, value_cache, dtype, head_dim, num_kv_heads, rows, row_stride,
                       a.box_rows, int8))
    return cuda_fail(cudaErrorInvalidValue);
  a.kv_int8 = int8;
  a.kv_fp8 = int8 && fp8;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  if (write && (!balanced || int8)) {
    // Fixed partitions or one-byte pools: the write is its own launch; the
    // decode kernel reads context_lens, block_table and the query at once
    // and waits for the write (programmatic dependent launch) only before
    // its first K/V load.
    pa::ReshapeArgs w = *write;
    w.num_sms = a.num_sms;
    e = pa::launch_reshape_and_cache(w, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
    a.after_write = true;
  } else if (write) {
    // 16-bit pools, balanced schedule: the step's cache write runs inside
    // the decode launch.
    a.num_new = write->num_tokens;
    a.new_k = write->key;
    a.new_v = write->value;
    a.new_stride = write->row_stride_bytes / 2;
    a.slot_mapping = write->slot_mapping;
    a.k_pool = write->key_cache;
    a.v_pool = write->value_cache;
  }
  e = pa::launch_decode(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

pa_status pa_decode(void *out, int64_t out_row_stride, const void *query, int64_t q_row_stride,
                    const void *key_cache, const void *value_cache, const int32_t *block_table,
                    int64_t block_table_stride, int32_t max_blocks_per_seq,
                    const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                    int64_t num_blocks, float scale, int32_t max_context_len,
                    int32_t partition_size, void *workspace, size_t workspace_bytes,
                    pa_dtype dtype, int32_t *d_error, void *stream) {
  return decode_call(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                     block_table, block_table_stride, max_blocks_per_seq, context_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                     max_context_len, partition_size, workspace, workspace_bytes, dtype, d_error,
                     stream, nullptr);
}

pa_status pa_decode_int8(void *out, int64_t out_row_stride, const void *query,
                         int64_t q_row_stride, const void *key_cache, const void *value_cache,
                         const int32_t *block_table, int64_t block_table_stride,
                         int32_t max_blocks_per_seq, const int32_t *context_lens,
                         int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_dim, int32_t block_size, int64_t num_blocks,
                         const float *k_scale, const float *v_scale, float scale,
                         int32_t max_context_len, int32_t partition_size, void *workspace,
                         size_t workspace_bytes, pa_dtype dtype, int32_t *d_error,
                         void *stream) {
  if (!k_scale || !v_scale) return PA_ERR_NULL;
  return decode_call(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                     block_table, block_table_stride, max_blocks_per_seq, context_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                     max_context_len, partition_size, workspace, workspace_bytes, dtype, d_error,
                     stream, nullptr, k_scale, v_scale);
}

pa_status pa_decode_fp8(void *out, int64_t out_row_stride, const void *query,
                        int64_t q_row_stride, const void *key_cache, const void *value_cache,
                        const int32_t *block_table, int64_t block_table_stride,
                        int32_t max_blocks_per_seq, const int32_t *context_lens,
                        int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                        int32_t head_dim, int32_t block_size, int64_t num_blocks,
                        const float *k_scale, const float *v_scale, float scale,
                        int32_t max_context_len, int32_t partition_size, void *workspace,
                        size_t workspace_bytes, pa_dtype dtype, int32_t *d_error,
                        void *stream) {
  if (!k_scale || !v_scale) return PA_ERR_NULL;
  return decode_call(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                     block_table, block_table_stride, max_blocks_per_seq, context_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                     max_context_len, partition_size, workspace, workspace_bytes, dtype, d_error,
                     stream, nullptr, k_scale, v_scale, true);
}

pa_status pa_decode_write(void *out, int64_t out_row_stride, const void *query,
                          int64_t q_row_stride, const void *key, const void *value,
                          int64_t kv_row_stride, void *key_cache, void *value_cache,
                          const int64_t *slot_mapping, int32_t num_new_tokens,
                          const int32_t *block_table, int64_t block_table_stride,
                          int32_t max_blocks_per_seq, const int32_t *context_lens,
                          int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim, int32_t block_size, int64_t num_blocks, float scale,
                          int32_t max_context_len, int32_t partition_size, void *workspace,
                          size_t workspace_bytes, pa_dtype dtype, int32_t *d_error,
                          void *stream) {
  pa::ReshapeArgs w;
  bool empty = true;
  const pa_status st = prepare_write(key, value, kv_row_stride, key_cache, value_cache,
                                     slot_mapping, num_new_tokens, num_kv_heads, head_dim,
                                     block_size, num_blocks, dtype, d_error, &w, &empty);
  if (st != PA_OK) return st;
  return decode_call(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                     block_table, block_table_stride, max_blocks_per_seq, context_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                     max_context_len, partition_size, workspace, workspace_bytes, dtype, d_error,
                     stream, empty ? nullptr : &w);
}

pa_status pa_decode_write_int8(void *out, int64_t out_row_stride, const void *query,
                               int64_t q_row_stride, const void *key, const void *value,
                               int64_t kv_row_stride, void *key_cache, void *value_cache,
                               const int64_t *slot_mapping, int32_t num_new_tokens,
                               const int32_t *block_table, int64_t block_table_stride,
                               int32_t max_blocks_per_seq, const int32_t *context_lens,
                               int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                               int32_t head_dim, int32_t block_size, int64_t num_blocks,
                               const float *k_scale, const float *v_scale, float scale,
                               int32_t max_context_len, int32_t partition_size,
                               void *workspace, size_t workspace_bytes, pa_dtype dtype,
                               int32_t *d_error, void *stream) {
  if (!k_scale || !v_scale) return PA_ERR_NULL;
  pa::ReshapeArgs w;
  bool empty = true;
  const pa_status st = prepare_write(key, value, kv_row_stride, key_cache, value_cache,
                                     slot_mapping, num_new_tokens, num_kv_heads, head_dim,
                                     block_size, num_blocks, dtype, d_error, &w, &empty);
  if (st != PA_OK) return st;
  w.int8 = true;
  w.dtype = dtype;
  w.head_dim = head_dim;
  w.k_scale = k_scale;
  w.v_scale = v_scale;
  return decode_call(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                     block_table, block_table_stride, max_blocks_per_seq, context_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                     max_context_len, partition_size, workspace, workspace_bytes, dtype, d_error,
                     stream, empty ? nullptr : &w, k_scale, v_scale);
}

pa_status pa_decode_write_fp8(void *out, int64_t out_row_stride, const void *query,
                              int64_t q_row_stride, const void *key, const void *value,
                              int64_t kv_row_stride, void *key_cache, void *value_cache,
                              const int64_t *slot_mapping, int32_t num_new_tokens,
                              const int32_t *block_table, int64_t block_table_stride,
                              int32_t max_blocks_per_seq, const int32_t *context_lens,
                              int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, int64_t num_blocks,
                              const float *k_scale, const float *v_scale, float scale,
                              int32_t max_context_len, int32_t partition_size,
                              void *workspace, size_t workspace_bytes, pa_dtype dtype,
                              int32_t *d_error, void *stream) {
  if (!k_scale || !v_scale) return PA_ERR_NULL;
  pa::ReshapeArgs w;
  bool empty = true;
  const pa_status st = prepare_write(key, value, kv_row_stride, key_cache, value_cache,
                                     slot_mapping, num_new_tokens, num_kv_heads, head_dim,
                                     block_size, num_blocks, dtype, d_error, &w, &empty);
  if (st != PA_OK) return st;
  w.int8 = true;
  w.fp8 = true;
  w.dtype = dtype;
  w.head_dim = head_dim;
  w.k_scale = k_scale;
  w.v_scale = v_scale;
  return decode_call(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                     block_table, block_table_stride, max_blocks_per_seq, context_lens, num_seqs,
                     num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale,
                     max_context_len, partition_size, workspace, workspace_bytes, dtype, d_error,
                     stream, empty ? nullptr : &w, k_scale, v_scale, true);
}

pa_status pa_prefill_varlen(void *out, int64_t out_row_stride, const void *query,
                            int64_t q_row_stride, const void *key_cache,
                            const void *value_cache, const int32_t *block_table,
                            int64_t block_table_stride, int32_t max_blocks_per_seq,
                            const int32_t *cu_seqlens_q, const int32_t *context_lens,
                            int32_t num_seqs, int32_t total_q, int32_t max_seqlen_q,
                            int32_t max_context_len, int32_t num_q_heads,
                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                            int64_t num_blocks, float scale, int32_t causal, pa_dtype dtype,
                            int32_t *d_error, void *stream) {
  if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || max_context_len < 0 ||
      num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      num_blocks <= 0 || max_blocks_per_seq < 0)
    return PA_ERR_SHAPE;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_SHAPE;
  if (block_table_stride < max_blocks_per_seq) return PA_ERR_SHAPE;
  if (!isfinite(scale)) return PA_ERR_SHAPE;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (!(block_size == 16 || block_size == 32 || block_size == 64 || block_size == 128))
    return PA_ERR_UNSUPPORTED;
  if (num_blocks * block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  if (!out || !query || !key_cache || !value_cache || !block_table || !cu_seqlens_q ||
      !context_lens)
    return PA_ERR_NULL;
  const int64_t qrow = static_cast<int64_t>(num_q_heads) * head_dim;
  if (q_row_stride < qrow || out_row_stride < qrow) return PA_ERR_SHAPE;
  if (q_row_stride % 8 || out_row_stride % 8) return PA_ERR_ALIGN;
  if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache))
    return PA_ERR_ALIGN;

  pa::PrefillArgs a;
  a.out = out;
  a.out_row_stride = out_row_stride;
  a.query = query;
  a.q_row_stride = q_row_stride;
  a.block_table = block_table;
  a.block_table_stride = block_table_stride;
  const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
  a.capacity = static_cast<int32_t>(cap > INT32_MAX ? INT32_MAX : cap);
  a.cu_seqlens_q = cu_seqlens_q;
  a.context_lens = context_lens;
  a.num_seqs = num_seqs;
  a.total_q = total_q;
  a.max_seqlen_q = max_seqlen_q;
  a.max_context_len = max_context_len;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.causal = causal ? 1 : 0;
  a.d_error = d_error;
  a.dtype = dtype;
  a.wait_ns = pa::pipeline_wait_ns();
  cudaError_t e = current_num_sms(&a.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  const int64_t kv_rows = num_blocks * block_size;
  const int64_t kv_stride = static_cast<int64_t>(num_kv_heads) * head_dim;
  const int box = block_size;  // one box per block
  // The query tile is 128 rows: 128 / pg tokens x the pg query heads of one
  // KV head, the heads of a token adjacent.
  a.packed_heads = pa::prefill_packed_heads(num_q_heads / num_kv_heads, max_seqlen_q);
  if (!encode_rows_map(&a.tm_q, query, dtype, head_dim, num_q_heads, total_q, q_row_stride,
                       128 / a.packed_heads, false, a.packed_heads) ||
      !encode_rows_map(&a.tm_k, key_cache, dtype, head_dim, num_kv_heads, kv_rows, kv_stride,
                       box) ||
      !encode_rows_map(&a.tm_v, value_cache, dtype, head_dim, num_kv_heads, kv_rows, kv_stride,
                       box))
    return cuda_fail(cudaErrorInvalidValue);
  e = pa::launch_prefill(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_attention_varlen(void *out, int64_t out_row_stride, const void *query,
                              int64_t q_row_stride, const void *key, const void *value,
                              int64_t kv_row_stride, const int32_t *cu_seqlens,
                              int32_t num_seqs, int32_t total_tokens, int32_t max_seqlen,
                              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                              float scale, int32_t causal, pa_dtype dtype, int32_t *d_error,
                              void *stream) {
  if (num_seqs < 0 || total_tokens < 0 || max_seqlen < 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0 || head_dim <= 0)
    return PA_ERR_SHAPE;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_SHAPE;
  if (!isfinite(scale)) return PA_ERR_SHAPE;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_tokens == 0 || max_seqlen == 0) return PA_OK;
  if (!out || !query || !key || !value || !cu_seqlens) return PA_ERR_NULL;
  const int64_t qrow = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t kvrow = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_row_stride < qrow || out_row_stride < qrow || kv_row_stride < kvrow) return PA_ERR_SHAPE;
  if (q_row_stride % 8 || out_row_stride % 8 || kv_row_stride % 8) return PA_ERR_ALIGN;
  if (!aligned16(out) || !aligned16(query) || !aligned16(key) || !aligned16(value))
    return PA_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return PA_ERR_ALIGN;

  pa::AttentionVarlenArgs a;
  a.out = out;
  a.out_row_stride = out_row_stride;
  a.cu_seqlens = cu_seqlens;
  a.num_seqs = num_seqs;
  a.total = total_tokens;
  a.max_seqlen = max_seqlen;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.packed_heads = pa::flash_packed_heads(num_q_heads / num_kv_heads);
  auto items = [&](int tiles) {
    return pa::varlen_items(num_seqs, total_tokens, max_seqlen, num_q_heads, a.packed_heads,
                            tiles);
  };
  a.tiles = 2;
  a.grid = items(2);
  if (a.grid > INT32_MAX) return PA_ERR_UNSUPPORTED;
  if (scale == 0.0f && total_tokens > (1 << 30)) return PA_ERR_UNSUPPORTED;  // q_off + a row
  flash_scale(scale, total_tokens, &a.scale_log2, &a.negate, &a.q_off);
  a.causal = causal ? 1 : 0;
  a.d_error = d_error;
  a.dtype = dtype;
  a.wait_ns = pa::pipeline_wait_ns();
  cudaError_t e = current_num_sms(&a.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  // Few query tiles: one per item, its keys on both streams by turns, while all
  // items run at once (500 tokens 32/32 heads: 11.2 us, in pairs 14.1; 2000 8/2:
  // 21.5 and 33.8; 37 tokens 8/2: 7.2 and 8.4), of longer prompts in up to four
  // rounds (2000 tokens 32/8, 3.4 rounds: 40.4 and 46.8; 1024 32/8, 1.7: 20.1 and
  // 23.0), which pairs take half of: more items of few keys cost more than they
  // even out (30 x 100 tokens 8/2, 1.6 rounds: 14.7 and 11.7), and so do more
  // rounds, that load K and V for every tile (8000 tokens 16/4, 6.6: 210 and 167;
  // 4 x 1000 32/32, 6.7: 52 and 48).  "Longer" goes by the bound, the host's only
  // sign of a batch's longest prompt: by twice the mean length, loose bounds cost
  // nothing (30 x 100 8/2 with a bound of 131072: 12.2 us, by the bound 14.7), but
  // batches of one long prompt and many short ones do (2000 + 20 x 30 tokens 8/2:
  // 37.4 against 25.7; 8000 + 20 x 200 32/8, with the compact softmax: 394 against
  // 352).
  const int64_t rounds = max_seqlen >= 640 ? 4 : 1;
  if (items(1) <= rounds * a.num_sms) {
    a.tiles = 1;
    a.grid = items(1);
  }
  if (!encode_rows_map(&a.tm_q, query, dtype, head_dim, num_q_heads, total_tokens, q_row_stride,
                       128 / a.packed_heads, false, a.packed_heads) ||
      !encode_rows_map(&a.tm_k, key, dtype, head_dim, num_kv_heads, total_tokens, kv_row_stride,
                       128) ||
      !encode_rows_map(&a.tm_v, value, dtype, head_dim, num_kv_heads, total_tokens,
                       kv_row_stride, 128))
    return cuda_fail(cudaErrorInvalidValue);
  e = pa::launch_attention_varlen(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // extern "C"

namespace {

// Sizes of a shared-prefix decode; `shared` false: it is a plain decode (no
// group, no prefix, nothing to attend to).
struct SharedPlan {
  bool shared = false;
  int sms = 0, runs = 0;
  size_t decode_bytes = 0, o_bytes = 0, ml_bytes = 0, bytes = 0;
};
pa_status shared_plan(int32_t num_seqs, int32_t num_groups, int32_t num_q_heads,
                      int32_t num_kv_heads, int32_t head_dim, int32_t max_context_len,
                      int32_t max_prefix_len, int32_t block_size, SharedPlan *out) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_context_len < 0 ||
      num_groups < 0 || max_prefix_len < 0 || num_q_heads % num_kv_heads != 0)
    return PA_ERR_SHAPE;
  int32_t P = 0;
  SharedPlan s;
  s.shared = num_seqs > 0 && num_groups > 0 && max_prefix_len > 0 && max_context_len > 0;
  // The schedules count in 32 bits.  (A plain decode would not do in their
  // place: it reads each row's own entries for the prefix, and a row need not
  // hold them.)
  const int64_t most = 1LL << 30;
  const int units = num_kv_heads * pa::decode_slices(num_q_heads / num_kv_heads).nc;
  if (s.shared &&
      (max_context_len >= most || max_prefix_len >= most ||
       !use_balanced(num_seqs, units, max_context_len, 0) ||
       pa::shared_cost(num_seqs, num_groups, num_q_heads, num_kv_heads, max_prefix_len) >= most))
    return PA_ERR_UNSUPPORTED;
  // The own parts' schedule keeps 12 bytes per sequence in shared memory.
  if (s.shared && pa::decode_smem_bytes(head_dim, num_seqs, 0, block_size) +
                          4 * static_cast<size_t>(num_seqs) >
                      227 * 1024)
    return PA_ERR_UNSUPPORTED;
  const pa_status st = pa_decode_plan(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                      max_context_len, 0, &P, &s.decode_bytes);
  if (st != PA_OK) return st;
  const cudaError_t e = current_num_sms(&s.sms);
  if (e != cudaSuccess) return cuda_fail(e);
  s.bytes = s.decode_bytes;
  if (s.shared) {
    const int pg = pa::flash_packed_heads(num_q_heads / num_kv_heads);
    s.runs = pa::shared_runs(num_seqs, num_groups, num_q_heads, num_kv_heads, max_prefix_len,
                             s.sms);
    const size_t rows = static_cast<size_t>(num_seqs) * (num_q_heads + pg) +
                        512 * static_cast<size_t>(s.runs);
    if (rows > INT32_MAX) return PA_ERR_UNSUPPORTED;
    s.o_bytes = align256(rows * head_dim * sizeof(float));
    s.ml_bytes = align256(rows * 2 * sizeof(float));
    s.bytes += s.o_bytes + s.ml_bytes + align256((static_cast<size_t>(num_seqs) + 1) * 32);
  }
  *out = s;
  return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_decode_shared_plan(int32_t num_seqs, int32_t num_groups, int32_t num_q_heads,
                                int32_t num_kv_heads, int32_t head_dim, int32_t max_context_len,
                                int32_t max_prefix_len, size_t *workspace_bytes_out) {
  SharedPlan s;
  // (8: what the plan serves, the call serves at any block size)
  const pa_status st = shared_plan(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim,
                                   max_context_len, max_prefix_len, 8, &s);
  if (st == PA_OK && workspace_bytes_out) *workspace_bytes_out = s.bytes;
  return st;
}

pa_status pa_decode_shared(void *out, int64_t out_row_stride, const void *query,
                           int64_t q_row_stride, const void *key_cache, const void *value_cache,
                           const int32_t *block_table, int64_t block_table_stride,
                           int32_t max_blocks_per_seq, const int32_t *context_lens,
                           const int32_t *group_starts, const int32_t *prefix_lens,
                           int32_t num_groups, int32_t num_seqs, int32_t num_q_heads,
                           int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                           int64_t num_blocks, float scale, int32_t max_context_len,
                           int32_t max_prefix_len, void *workspace, size_t workspace_bytes,
                           pa_dtype dtype, int32_t *d_error, void *stream) {
  if (num_groups < 0 || max_prefix_len < 0) return PA_ERR_SHAPE;
  DecodeSetup c;
  pa_status st = check_decode(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                              block_table, block_table_stride, max_blocks_per_seq, context_lens,
                              num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                              num_blocks, scale, max_context_len, 0, dtype, &c);
  if (st != PA_OK || c.empty) return st;
  if (num_groups > 0 && max_prefix_len > 0) {
    if (!group_starts || !prefix_lens) return PA_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(group_starts) | reinterpret_cast<uintptr_t>(prefix_lens)) & 3u)
      return PA_ERR_ALIGN;
  }
  SharedPlan s;
  st = shared_plan(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, max_context_len,
                   max_prefix_len, block_size, &s);
  if (st != PA_OK) return st;
  if (!s.shared)
    return decode_call(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                       block_table, block_table_stride, max_blocks_per_seq, context_lens,
                       num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                       scale, max_context_len, 0, workspace, workspace_bytes, dtype, d_error,
                       stream, nullptr);
  if (!workspace || workspace_bytes < s.bytes ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PA_ERR_WORKSPACE;
  pa::DecodeSharedArgs a;
  pa::DecodeArgs &d = a.decode;
  d = c.args;
  d.num_sms = s.sms;
  set_balanced(&d, workspace);
  d.wait_ns = pa::pipeline_wait_ns();
  d.d_error = d_error;
  a.group_starts = group_starts;
  a.prefix_lens = prefix_lens;
  a.num_groups = num_groups;
  a.max_prefix = max_prefix_len;
  a.runs = s.runs;
  a.prefix_cost =
      pa::shared_cost(num_seqs, num_groups, num_q_heads, num_kv_heads, max_prefix_len);
  a.packed_heads = pa::flash_packed_heads(num_q_heads / num_kv_heads);
  flash_scale(scale, num_seqs, &a.scale_log2, &a.negate, &a.q_off);
  char *w = static_cast<char *>(workspace) + s.decode_bytes;
  a.ws_o = reinterpret_cast<float *>(w);
  w += s.o_bytes;
  a.ws_ml = reinterpret_cast<float *>(w);
  w += s.ml_bytes;
  a.ws_info = reinterpret_cast<int32_t *>(w);
  const int64_t rows = num_blocks * block_size;
  const int64_t row_stride = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (!encode_rows_map(&d.tm_k, key_cache, dtype, head_dim, num_kv_heads, rows, row_stride,
                       d.box_rows) ||
      !encode_rows_map(&d.tm_v, value_cache, dtype, head_dim, num_kv_heads, rows, row_stride,
                       d.box_rows) ||
      !encode_rows_map(&a.tm_q, query, dtype, head_dim, num_q_heads, num_seqs, q_row_stride,
                       128 / a.packed_heads, false, a.packed_heads) ||
      !encode_rows_map(&a.tm_k, key_cache, dtype, head_dim, num_kv_heads, rows, row_stride,
                       block_size) ||
      !encode_rows_map(&a.tm_v, value_cache, dtype, head_dim, num_kv_heads, rows, row_stride,
                       block_size))
    return cuda_fail(cudaErrorInvalidValue);
  const cudaError_t e = pa::launch_decode_shared(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // extern "C"

namespace {

// The write into 4-bit pools; *empty as for prepare_write.
pa_status prepare_write_fp4(const void *key, const void *value, int64_t kv_row_stride,
                            void *key_cache, void *value_cache, const int64_t *slot_mapping,
                            int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                            int32_t block_size, int64_t num_blocks, const float *k_scale,
                            const float *v_scale, pa_dtype dtype, int32_t *d_error,
                            pa::ReshapeArgs *out, bool *empty) {
  if (block_size > 0 && (num_blocks < 0 || num_blocks > INT64_MAX / block_size))
    return PA_ERR_SHAPE;
  const pa_status st = prepare_write(key, value, kv_row_stride, key_cache, value_cache,
                                     slot_mapping, num_tokens, num_kv_heads, head_dim, block_size,
                                     num_blocks, dtype, d_error, out, empty);
  if (st != PA_OK) return st;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (!valid_block_size(block_size) || num_kv_heads > 65536) return PA_ERR_UNSUPPORTED;
  if (!k_scale || !v_scale) return PA_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3u)
    return PA_ERR_ALIGN;
  if (*empty) return PA_OK;
  if (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) return PA_ERR_ALIGN;
  out->dtype = dtype;
  out->head_dim = head_dim;
  out->k_scale = k_scale;
  out->v_scale = v_scale;
  out->num_kv_heads = num_kv_heads;
  out->block_size = block_size;
  return PA_OK;
}

// The workspace of a decode over 4-bit pools: pieces x (heads per slice) partial states,
// then the prefix sums for the join.
size_t fp4_workspace(const pa::DecodeBalance &d, int hs, int head_dim, int num_seqs) {
  const size_t rows = static_cast<size_t>(d.pieces) * hs;
  return align256(rows * head_dim * sizeof(float)) + align256(rows * 2 * sizeof(float)) +
         align256((static_cast<size_t>(num_seqs) + 1) * sizeof(int32_t));
}

pa_status fp4_plan(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                   int32_t max_context_len, int *sms, pa::DecodeBalance *d, size_t *bytes) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_context_len < 0 || num_q_heads % num_kv_heads != 0)
    return PA_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  const pa::DecodeSlices sl = pa::decode_slices(num_q_heads / num_kv_heads);
  // the schedule's positions are 32-bit, its prefix sums in shared memory
  const int64_t units = static_cast<int64_t>(num_kv_heads) * sl.nc;
  if (static_cast<int64_t>(max_context_len) > (1 << 30) ||
      (num_seqs > 0 &&
       units * ((max_context_len + 31) / 32) * 32 > ((1LL << 30) - 1) / num_seqs) ||
      num_seqs > pa::kFp4MostSeqs || num_kv_heads > 65536 ||
      static_cast<int64_t>(num_q_heads) * head_dim > INT32_MAX)
    return PA_ERR_UNSUPPORTED;
  const cudaError_t e = current_num_sms(sms);
  if (e != cudaSuccess) return cuda_fail(e);
  *d = pa::fp4_balance(num_seqs, static_cast<int>(units), sl.ng, head_dim, max_context_len, *sms);
  *bytes = fp4_workspace(*d, sl.hs, head_dim, num_seqs);
  return PA_OK;
}

// pa_decode_fp4, optionally after the step's cache write (launched once every check has
// passed, so an error enqueues nothing).
pa_status decode_fp4(void *out, int64_t out_row_stride, const void *query, int64_t q_row_stride,
                     const void *key_cache, const void *value_cache, const int32_t *block_table,
                     int64_t block_table_stride, int32_t max_blocks_per_seq,
                     const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                     int64_t num_blocks, const float *k_scale, const float *v_scale, float scale,
                     int32_t max_context_len, void *workspace, size_t workspace_bytes,
                     pa_dtype dtype, int32_t *d_error, void *stream, const pa::ReshapeArgs *write) {
  DecodeSetup setup;
  pa_status st = check_decode(out, out_row_stride, query, q_row_stride, key_cache, value_cache,
                              block_table, block_table_stride, max_blocks_per_seq, context_lens,
                              num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                              num_blocks, scale, max_context_len, 0, dtype, &setup);
  if (st != PA_OK) return st;
  pa::DecodeArgs &a = setup.args;
  if (!setup.empty) {
    if (!k_scale || !v_scale) return PA_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
         reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(context_lens)) & 3u)
      return PA_ERR_ALIGN;
    pa::DecodeBalance d;
    size_t need = 0;
    st = fp4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len, &a.num_sms, &d,
                  &need);
    if (st != PA_OK) return st;
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
      return PA_ERR_WORKSPACE;
    a.grid = d.grid;
    const size_t rows = static_cast<size_t>(d.pieces) * a.slices.hs;
    char *w = static_cast<char *>(workspace);
    a.ws_o = reinterpret_cast<float *>(w);
    w += align256(rows * head_dim * sizeof(float));
    a.ws_ml = reinterpret_cast<float *>(w);
    w += align256(rows * 2 * sizeof(float));
    a.ws_pref = reinterpret_cast<int32_t *>(w);
    a.partition_size = 0;
    a.num_partitions = 0;
    a.k_pool = const_cast<void *>(key_cache);
    a.v_pool = const_cast<void *>(value_cache);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.d_error = d_error;
    a.wait_ns = pa::pipeline_wait_ns();
  }
  if (write) {
    pa::ReshapeArgs w = *write;
    cudaError_t e = current_num_sms(&w.num_sms);
    if (e == cudaSuccess) e = pa::launch_reshape_and_cache_fp4(w, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
    // The decode starts beside the write: lengths, block ids and the ring's set-up do not wait
    // for it (one call / without this / two calls, device us: 4 sequences up to 128 tokens, 8/2
    // heads of 64, 6.6 / 7.5 / 7.4; 32 up to 2000, 32/8, 17.6 / 18.5 / 18.5, the decode alone
    // 18.0; 4 up to 131072, 64/8, 87.5 / 88.1 / 88.2).
    a.after_write = true;
  }
  if (setup.empty) return PA_OK;
  const cudaError_t e = pa::launch_decode_fp4(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

pa_status pa_reshape_and_cache_fp4(const void *key, const void *value, int64_t kv_row_stride,
                                   void *key_cache, void *value_cache,
                                   const int64_t *slot_mapping, int32_t num_tokens,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                   int64_t num_blocks, const float *k_scale, const float *v_scale,
                                   pa_dtype dtype, int32_t *d_error, void *stream) {
  pa::ReshapeArgs w;
  bool empty = true;
  const pa_status st = prepare_write_fp4(key, value, kv_row_stride, key_cache, value_cache,
                                         slot_mapping, num_tokens, num_kv_heads, head_dim,
                                         block_size, num_blocks, k_scale, v_scale, dtype, d_error,
                                         &w, &empty);
  if (st != PA_OK || empty) return st;
  cudaError_t e = current_num_sms(&w.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  e = pa::launch_reshape_and_cache_fp4(w, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_gather_cache_fp4(void *key_out, int64_t k_out_row_stride, void *value_out,
                              int64_t v_out_row_stride, int32_t num_rows, const void *key_cache,
                              const void *value_cache, const int32_t *block_table,
                              int64_t block_table_stride, int32_t max_blocks_per_seq,
                              const int32_t *context_lens, const int32_t *row_starts,
                              int32_t num_seqs, int32_t max_context_len, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, int64_t num_blocks,
                              const float *k_scale, const float *v_scale, pa_dtype dtype,
                              int32_t *d_error, void *stream) {
  if (num_rows < 0 || max_blocks_per_seq < 0 || num_seqs < 0 || max_context_len < 0 ||
      num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0 ||
      block_table_stride < max_blocks_per_seq)
    return PA_ERR_SHAPE;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  if (!valid_block_size(block_size) || num_seqs > 65535 || num_kv_heads > 65536)
    return PA_ERR_UNSUPPORTED;
  const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (k_out_row_stride < row || v_out_row_stride < row) return PA_ERR_SHAPE;
  if (num_rows > 0 && (k_out_row_stride > INT64_MAX / 4 / num_rows ||
                       v_out_row_stride > INT64_MAX / 4 / num_rows))
    return PA_ERR_SHAPE;
  if (k_out_row_stride % 8 || v_out_row_stride % 8) return PA_ERR_ALIGN;
  if (num_seqs == 0 || max_context_len == 0) return PA_OK;
  if (!key_cache || !value_cache || !block_table || !context_lens || !row_starts || !k_scale ||
      !v_scale || (num_rows > 0 && (!key_out || !value_out)))
    return PA_ERR_NULL;
  if (!aligned16(key_out) || !aligned16(value_out) || !aligned16(key_cache) ||
      !aligned16(value_cache))
    return PA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(context_lens) |
       reinterpret_cast<uintptr_t>(row_starts) | reinterpret_cast<uintptr_t>(k_scale) |
       reinterpret_cast<uintptr_t>(v_scale)) & 3u)
    return PA_ERR_ALIGN;
  pa::GatherArgs a;
  a.key_out = key_out;
  a.value_out = value_out;
  a.k_stride_bytes = k_out_row_stride * 2;
  a.v_stride_bytes = v_out_row_stride * 2;
  a.num_rows = num_rows;
  a.key_cache = key_cache;
  a.value_cache = value_cache;
  a.block_table = block_table;
  a.block_table_stride = block_table_stride;
  const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
  a.capacity = static_cast<int32_t>(cap > INT32_MAX ? INT32_MAX : cap);
  a.context_lens = context_lens;
  a.row_starts = row_starts;
  a.num_seqs = num_seqs;
  a.max_context_len = max_context_len;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.dtype = dtype;
  a.d_error = d_error;
  cudaError_t e = current_num_sms(&a.num_sms);
  if (e != cudaSuccess) return cuda_fail(e);
  e = pa::launch_gather_cache_fp4(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

pa_status pa_decode_fp4_plan(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                             int32_t head_dim, int32_t max_context_len,
                             size_t *workspace_bytes_out) {
  int sms = 0;
  pa::DecodeBalance d;
  size_t bytes = 0;
  const pa_status st = fp4_plan(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                &sms, &d, &bytes);
  if (st == PA_OK && workspace_bytes_out) *workspace_bytes_out = bytes;
  return st;
}

pa_status pa_decode_fp4(void *out, int64_t out_row_stride, const void *query, int64_t q_row_stride,
                        const void *key_cache, const void *value_cache, const int32_t *block_table,
                        int64_t block_table_stride, int32_t max_blocks_per_seq,
                        const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                        int64_t num_blocks, const float *k_scale, const float *v_scale, float scale,
                        int32_t max_context_len, void *workspace, size_t workspace_bytes,
                        pa_dtype dtype, int32_t *d_error, void *stream) {
  return decode_fp4(out, out_row_stride, query, q_row_stride, key_cache, value_cache, block_table,
                    block_table_stride, max_blocks_per_seq, context_lens, num_seqs, num_q_heads,
                    num_kv_heads, head_dim, block_size, num_blocks, k_scale, v_scale, scale,
                    max_context_len, workspace, workspace_bytes, dtype, d_error, stream, nullptr);
}

pa_status pa_decode_write_fp4(void *out, int64_t out_row_stride, const void *query,
                              int64_t q_row_stride, const void *key, const void *value,
                              int64_t kv_row_stride, void *key_cache, void *value_cache,
                              const int64_t *slot_mapping, int32_t num_new_tokens,
                              const int32_t *block_table, int64_t block_table_stride,
                              int32_t max_blocks_per_seq, const int32_t *context_lens,
                              int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, int64_t num_blocks,
                              const float *k_scale, const float *v_scale, float scale,
                              int32_t max_context_len, void *workspace, size_t workspace_bytes,
                              pa_dtype dtype, int32_t *d_error, void *stream) {
  pa::ReshapeArgs w;
  bool empty = true;
  const pa_status st = prepare_write_fp4(key, value, kv_row_stride, key_cache, value_cache,
                                         slot_mapping, num_new_tokens, num_kv_heads, head_dim,
                                         block_size, num_blocks, k_scale, v_scale, dtype, d_error,
                                         &w, &empty);
  if (st != PA_OK) return st;
  return decode_fp4(out, out_row_stride, query, q_row_stride, key_cache, value_cache, block_table,
                    block_table_stride, max_blocks_per_seq, context_lens, num_seqs, num_q_heads,
                    num_kv_heads, head_dim, block_size, num_blocks, k_scale, v_scale, scale,
                    max_context_len, workspace, workspace_bytes, dtype, d_error, stream,
                    empty ? nullptr : &w);
}

}  // extern "C"
