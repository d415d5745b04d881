// pa_internal.h -- launcher interface between the C ABI shim (pa_api.cu) and
// the kernels.  Arguments arrive here already validated.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa.h"

namespace pa {

struct ReshapeArgs {
  const void *key;
  const void *value;
  int64_t row_stride_bytes;  // between consecutive tokens of key / value
  void *key_cache;
  void *value_cache;
  const int64_t *slot_mapping;
  int32_t num_tokens;
  int64_t row_bytes;  // Hkv * D * 2
  int64_t num_slots;  // num_blocks * block_size
  int32_t *d_error;
  int num_sms;
  // 8-bit pools: the inputs are `dtype` (fp16/bf16), the pools INT8 codes
  // (or, with fp8, E4M3 codes) under the per-KV-head scales; row_bytes
  // counts the 16-bit input row.
  bool int8 = false;
  bool fp8 = false;
  pa_dtype dtype = PA_F16;
  int32_t head_dim = 0;
  const float *k_scale = nullptr, *v_scale = nullptr;
  int32_t num_kv_heads = 0, block_size = 0;  // 4-bit pools
};
cudaError_t launch_reshape_and_cache(const ReshapeArgs &a, cudaStream_t stream);
cudaError_t launch_reshape_and_cache_fp4(const ReshapeArgs &a, cudaStream_t stream);

// pa_gather_cache_fp4
struct GatherArgs {
  void *key_out, *value_out;
  int64_t k_stride_bytes, v_stride_bytes;  // between rows
  int32_t num_rows;
  const void *key_cache, *value_cache;
  const int32_t *block_table;
  int64_t block_table_stride;
  int32_t capacity;
  const int32_t *context_lens, *row_starts;
  int32_t num_seqs, max_context_len, num_kv_heads, head_dim, block_size;
  int64_t num_blocks;
  const float *k_scale, *v_scale;
  pa_dtype dtype;
  int32_t *d_error;
  int num_sms;
};
cudaError_t launch_gather_cache_fp4(const GatherArgs &a, cudaStream_t stream);

// pa_rope_and_cache; strides in elements.
struct RopeArgs {
  void *query_out, *key_out;  // key_out nullable with a cache
  int64_t q_out_row_stride, k_out_row_stride;
  const void *query, *key, *value;
  int64_t q_row_stride, kv_row_stride;
  const int32_t *positions;
  const float *cos_sin;  // [max_position, rot]
  int64_t max_position;
  int32_t rot;  // rotated elements of a head, 0 for none
  bool interleaved;
  const void *q_weight, *k_weight;  // [head_dim], nullable: no norm
  float eps;
  void *key_cache, *value_cache;  // null: no write
  const int64_t *slot_mapping;
  int64_t num_slots;
  int32_t num_tokens, num_q_heads, num_kv_heads, head_dim;
  pa_dtype dtype;
  int32_t *d_error;
  int num_sms;
  int groups;  // lane groups per token where tokens share a CTA (the launcher's)
};
cudaError_t launch_rope_and_cache(const RopeArgs &a, cudaStream_t stream);

struct CopyBlocksArgs {
  void *key_cache;
  void *value_cache;
  int64_t block_bytes;  // one block of one pool, a multiple of 16
  int64_t num_blocks;
  const int64_t *block_mapping;  // [num_pairs][2] (src, dst)
  int32_t num_pairs;
  int32_t *d_error;
  int num_sms;
};
cudaError_t launch_copy_blocks(const CopyBlocksArgs &a, cudaStream_t stream);

struct BuildTablesArgs {
  int32_t *block_table;
  int64_t block_table_stride;
  int32_t max_blocks_per_seq;
  const int32_t *context_lens, *query_lens, *free_blocks, *num_free;
  int32_t free_capacity;
  int32_t *context_lens_out, *cu_seqlens_q;
  int64_t *slot_mapping;
  int32_t *positions;  // nullable
  int32_t *num_free_out;
  int32_t num_seqs, max_tokens, block_size;
  int64_t num_blocks;
  int32_t *d_error;
  int num_sms;
};
cudaError_t launch_build_tables(const BuildTablesArgs &a, cudaStream_t stream);

// Decode tiling shared by the planner and the kernels.
constexpr int kDecodeWarps = 4;     // consumer warps (independent workers) per CTA
constexpr int kDecodeCtasPerSm = 2;  // resident decode CTAs per SM
constexpr int kDecodeSub = 16;      // tokens per worker per pipeline stage
constexpr int kDecodeChunkCap = 2048;  // balanced schedule: most tokens per chunk
constexpr int kDecodeSliceHeads = 16;  // most query heads one K/V read serves

// The query heads of one KV head (the GQA group, G of them) are served in
// slices of at most kDecodeSliceHeads heads: one K/V read serves a whole
// slice (one or two 8-head column groups of the score tile), and a KV head
// with more query heads is read once per slice.  A decode unit is one
// (sequence, slice); a sequence has num_kv_heads * nc units.
struct DecodeSlices {
  int ng;  // 8-head column groups per slice (1 or 2)
  int hs;  // query heads per slice (the last slice may hold fewer)
  int nc;  // slices per KV head
};
inline DecodeSlices decode_slices(int group) {
  DecodeSlices s;
  s.hs = group < kDecodeSliceHeads ? group : kDecodeSliceHeads;
  s.ng = s.hs > 8 ? 2 : 1;
  s.nc = (group + s.hs - 1) / s.hs;
  return s;
}

// Balanced decode schedule sizes, shared by the planner and the launcher:
// the grid (CTAs) and the most pieces (workspace rows per slice head) the
// split can produce for max_context_len; `units` = decode units per sequence.
struct DecodeBalance {
  int grid, workers;
  int stages;      // of a worker's ring (4-bit pools)
  int64_t pieces;  // units + chunks
};
inline DecodeBalance decode_balance(int num_seqs, int units, int max_ctx, int num_sms) {
  DecodeBalance d;
  const int64_t t_max = static_cast<int64_t>(num_seqs) * units * ((max_ctx + 15) / 16) * 16;
  int64_t grid = (t_max / kDecodeSub + kDecodeWarps - 1) / kDecodeWarps;
  if (grid > static_cast<int64_t>(kDecodeCtasPerSm) * num_sms)
    grid = static_cast<int64_t>(kDecodeCtasPerSm) * num_sms;
  if (grid < 1) grid = 1;
  d.grid = static_cast<int>(grid);
  d.workers = d.grid * kDecodeWarps;
  const int64_t per = static_cast<int64_t>(d.workers) * kDecodeChunkCap;
  const int64_t k = t_max > 0 ? (t_max + per - 1) / per : 1;
  const int64_t chunks = k * d.workers;
  d.pieces = static_cast<int64_t>(num_seqs) * units + chunks;
  return d;
}

struct DecodeArgs {
  void *out;
  int64_t out_row_stride;  // elements between sequences
  const void *query;
  int64_t q_row_stride;
  const int32_t *block_table;
  int64_t block_table_stride;
  int32_t capacity;  // max_blocks_per_seq * block_size, clamped to int32
  const int32_t *context_lens;
  int32_t num_seqs, num_q_heads, num_kv_heads, head_dim, block_size;
  int64_t num_blocks;
  float scale_log2;  // scale * log2(e)
  int32_t max_context_len, partition_size, num_partitions;  // partition_size 0: balanced
  int grid;        // decode CTAs
  bool merge;      // launch the merge kernel
  float *ws_o;     // fixed: [S, Hq, num_partitions, D]; balanced: [pieces, G, D]
  float *ws_ml;    // same rows, 2 floats: max (log2 units), sum
  int32_t *ws_pref;  // balanced: [S + 1] prefix sums for the merge kernel
  // The previous kernel in the stream is this library's cache write, which
  // writes only K/V pool rows: the decode kernel may read everything else
  // before waiting for it.
  bool after_write = false;
  // The one-call step: the decode launch also writes num_new tokens' K/V
  // rows (new_k / new_v, new_stride elements apart) into the pools at
  // slot_mapping, and takes each sequence's newest row from the token
  // written to it.
  int32_t num_new = 0;
  const void *new_k = nullptr, *new_v = nullptr;
  int64_t new_stride = 0;
  const int64_t *slot_mapping = nullptr;
  void *k_pool = nullptr, *v_pool = nullptr;
  DecodeSlices slices;
  int32_t *d_error;
  pa_dtype dtype;
  // pool maps: box (64 elements | head_dim codes, 1, box_rows), swizzled
  CUtensorMap tm_k, tm_v;
  int box_rows;
  int num_sms;
  bool kv_int8 = false;  // one-byte pools with per-KV-head scales
  bool kv_fp8 = false;   // ... holding E4M3 codes rather than INT8
  const float *k_scale = nullptr, *v_scale = nullptr;
  uint64_t wait_ns = 0;  // bound of a pipeline wait (see pipeline_wait_ns)
};
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t stream);

// The decode over 4-bit pools: CTAs of four warps, each a worker with a ring of stages of
// its own; the balanced split over all of them.
constexpr int kFp4Warps = 4;
constexpr int kFp4StageTokens = 64;
constexpr int kFp4ChunkCap = 1 << 18;    // most tokens per chunk (workers x cap < 2^31)
constexpr int kFp4MostSeqs = 8192;       // prefix sums and lengths, 8 bytes each in shared memory
// CTAs an SM: registers.  128 values and two column groups would spill at three (32 of 2700
// to 4000 tokens, 128/8 heads, two and three: fp16 43.8 and 48.3 us, bf16 44.6 and 52.5).
constexpr int fp4_ctas_per_sm(int head_dim, int ng) {
  return head_dim == 128 ? 4 - ng : ng == 1 ? 4 : 3;
}
// Shared memory: the stages (keys and values, 4.5 bits an element), a barrier each, then
// prefix sums and lengths.
inline int fp4_decode_smem(int head_dim, int stages, int num_seqs) {
  return kFp4Warps * stages * (kFp4StageTokens * head_dim * 9 / 8 + 8) + 4 * (2 * num_seqs + 1);
}
// CTAs of an SM by its 228 KB of shared memory, 1 KB of which is taken for each.
inline int fp4_ctas_that_fit(int head_dim, int stages, int num_seqs) {
  return 228 * 1024 / (fp4_decode_smem(head_dim, stages, num_seqs) + 1024);
}
// Stages of a worker's ring.  At 128 values two of them leave an SM's shared memory room
// for three CTAs, three for two: fewer workers, most of their tokens on their way at once,
// fewer states to join.  That is the better where the bound leaves those few workers 256
// tokens or less (two / three, device us, 32/8 heads: 8 sequences of 100 to 2000 tokens
// 11.4 / 10.0, 16 13.6 / 12.4, 16 of 2000 18.5 / 17.3; but 24 of 2000 20.6 / 22.2, 32 of 100
// to 2000 18.5 / 19.3, 64 28.3 / 30.1; one of 30000, 64/8, 21.0 / 19.8, of 65000 27.1 / 27.9).
// From 628 sequences on their sums and lengths leave three stages one CTA only, two stages
// two of them (two / three: 640 of 400 tokens, one KV head, 26.9 / 29.6, 700 28.8 / 33.2;
// eight KV heads, 700 of 32 30.0 / 43.0, 1024 42.8 / 61.9).
inline int fp4_stages(int head_dim, int num_seqs, int64_t t_max, int num_sms) {
  if (head_dim == 64) return 3;
  return t_max <= 256LL * 2 * kFp4Warps * num_sms && fp4_ctas_that_fit(head_dim, 3, num_seqs) >= 2
             ? 3
             : 2;
}
// Short contexts are not cut: no states, no second launch (cut / whole, device us: 4
// sequences of 64 / 128 / 192 tokens, 8/2 heads of 64, 5.5 / 4.3, 5.7 / 5.3, 5.7 / 6.4; 32 of
// 128 / 256 / 384, 32/8 9.1 / 6.8, 10.5 / 9.8, 10.6 / 12.8; 256 of 128 / 256 25.7 / 21.8,
// 32.7 / 30.9).
inline bool fp4_whole_units(int max_ctx, int64_t units) {
  return max_ctx > 0 && max_ctx <= (units < 128 ? 128 : 256);
}
inline DecodeBalance fp4_balance(int num_seqs, int units, int ng, int head_dim, int max_ctx,
                                 int num_sms) {
  DecodeBalance d;
  const int64_t t_max = static_cast<int64_t>(num_seqs) * units * ((max_ctx + 31) / 32) * 32;
  d.stages = fp4_stages(head_dim, num_seqs, t_max, num_sms);
  int64_t most = fp4_ctas_that_fit(head_dim, d.stages, num_seqs);  // resident at once
  if (most > fp4_ctas_per_sm(head_dim, ng)) most = fp4_ctas_per_sm(head_dim, ng);
  most *= num_sms;
  // A worker takes 32 tokens at least, and 64 where that leaves 768 workers or more: fewer
  // states to join (32 / 64 tokens throughout, device us; one sequence of 8000 tokens,
  // 32/8 heads 11.5 / 10.4; 16 of 600 12.3 / 10.4; but 8 of 192 7.3 / 7.7, 1 of 1000 6.9 /
  // 7.4).
  const int64_t shares = t_max / 32;
  int64_t grid = shares <= 768 ? shares : (shares / 2 > 768 ? shares / 2 : 768);
  const int64_t all = static_cast<int64_t>(num_seqs) * units;
  if (fp4_whole_units(max_ctx, all)) grid = all;
  grid = (grid + kFp4Warps - 1) / kFp4Warps;
  grid = grid < 1 ? 1 : (grid > most ? most : grid);
  d.grid = static_cast<int>(grid);
  d.workers = d.grid * kFp4Warps;
  const int64_t per = static_cast<int64_t>(d.workers) * kFp4ChunkCap;
  d.pieces = static_cast<int64_t>(num_seqs) * units + (t_max + per) / per * d.workers;
  return d;
}
cudaError_t launch_decode_fp4(const DecodeArgs &a, cudaStream_t stream);
// Records a failed CUDA call for pa_last_cuda_error() (this thread).
void record_cuda_error(cudaError_t e);
// Bound of the kernels' pipeline waits for the next launches: 2 s, unless a
// test shortened it through pa_debug_set_wait_limit_ns.
uint64_t pipeline_wait_ns();
size_t decode_smem_bytes(int head_dim, int num_seqs, int partition_size, int block_size,
                         bool kv_int8 = false);

struct PrefillArgs {
  void *out;
  int64_t out_row_stride;
  const void *query;
  int64_t q_row_stride;
  const int32_t *block_table;
  int64_t block_table_stride;
  int32_t capacity;
  const int32_t *cu_seqlens_q;
  const int32_t *context_lens;
  int32_t num_seqs, total_q, max_seqlen_q, max_context_len;
  int32_t num_q_heads, num_kv_heads, head_dim, block_size;
  int64_t num_blocks;
  float scale_log2;
  int32_t causal;
  int32_t *d_error;
  pa_dtype dtype;
  // Query heads packed into a tile's rows (a power of two dividing 128 and
  // the GQA group, or 1); tm_q's box is 64 x packed_heads x 128 / packed_heads.
  int packed_heads = 1;
  CUtensorMap tm_q, tm_k, tm_v;
  int num_sms;
  uint64_t wait_ns = 0;  // bound of a pipeline wait (see pipeline_wait_ns)
};
// The query heads a prefill tile packs: the whole GQA group when it is a
// power of two up to 128 (and the packed rows of the longest sequence fit in
// int32), else 1.
inline int prefill_packed_heads(int group, int max_seqlen_q) {
  if (group < 1 || group > 128 || (group & (group - 1)) != 0) return 1;
  if (static_cast<int64_t>(max_seqlen_q) * group > 0x3fffffff) return 1;
  return group;
}
cudaError_t launch_prefill(const PrefillArgs &a, cudaStream_t stream);

// The query heads a tile of the flash engine packs into its rows: the largest
// divisor of the GQA group whose multiples fill at least 7/8 of 128 rows.
inline int flash_packed_heads(int group) {
  for (int d = group < 128 ? group : 128; d > 1; --d)
    if (group % d == 0 && (128 / d) * d >= 112) return d;
  return 1;
}

// The most items a batch of packed prompts has (one CTA per item) of `tiles`
// query tiles each, times head units; at most one item of a sequence is partly
// filled.
inline int64_t varlen_items(int num_seqs, int total, int max_seqlen, int num_q_heads,
                            int packed_heads, int tiles) {
  const int64_t rows = tiles * (128 / packed_heads);
  const int64_t longest = max_seqlen < total ? max_seqlen : total;
  const int64_t items = total / rows + num_seqs, most = num_seqs * ((longest + rows - 1) / rows);
  return (items < most ? items : most) * (num_q_heads / packed_heads);
}

struct AttentionVarlenArgs {
  void *out;
  int64_t out_row_stride;
  const int32_t *cu_seqlens;
  int32_t num_seqs, total, max_seqlen;
  int32_t num_q_heads, num_kv_heads, head_dim;
  int packed_heads;
  int64_t grid;      // varlen_items
  int tiles;         // query tiles per item, 1 or 2
  float scale_log2;  // |scale| * log2(e), not 0
  bool negate;       // the scale is negative
  int32_t q_off;     // scale 0: rows to move the query tiles by, out of the tensor
  int32_t causal;
  int32_t *d_error;
  pa_dtype dtype;
  // boxes: q 64 x packed_heads x 128 / packed_heads, k and v 64 x 1 x 128
  CUtensorMap tm_q, tm_k, tm_v;
  int num_sms;
  uint64_t wait_ns = 0;
};
cudaError_t launch_attention_varlen(const AttentionVarlenArgs &a, cudaStream_t stream);

// The most the prefix pass can cost (see flash_kernel.cuh), and its runs: one per
// CTA, at most one per SM; a run costs at least 2.
inline int64_t shared_cost(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads,
                           int max_prefix) {
  const int pg = flash_packed_heads(num_q_heads / num_kv_heads), tpt = 128 / pg;
  const int64_t tiles =
      (static_cast<int64_t>(num_seqs) / tpt + num_groups) * (num_q_heads / pg);
  return tiles * ((static_cast<int64_t>(max_prefix) + 127) / 128);
}

// The own parts start on the SMs that the prefix pass leaves free, so a pass of
// a few tiles per SM, which is mostly start-up, takes half of the SMs (32/8 heads,
// with half and with all: 32 sequences over 2000 tokens 35.4 and 35.9 us, over 4000
// 37.4 and 42.3, over 6000 39.0 and 43.4; 16 over 9000 30.7 and 36.6; 64 over 1000,
// 64/8: 55.7 and 59.9; but 40 over 4000, 16/16, with many own parts for few tiles:
// 64.5 and 60.7).  Of longer passes, one of single query tiles waits for memory,
// which fewer SMs keep as busy while the own parts start on the rest: it takes the
// largest power of two, 128 of 152 (with 128 and with 152: 8 sequences, 32/8 heads,
// over 9000 / 20000 / 32768 / 50000 tokens 20.9, 24.3 / 26.4, 30.3 / 38.7, 44.4 /
// 52.3, 54.8; 16, 40/8, over 9000 / 20000 / 50000 27.0, 28.3 / 34.9, 36.7 / 58.3,
// 59.6; 8, 40/40, over 9000 / 20000 / 50000 50.0, 53.6 / 83.7, 84.5 / 172.2, 171.4;
// 32/32 over 9000 / 20000 / 50000 46.9, 46.8 / 71.1, 71.8 / 143.5, 140.6; 112 and 140
// SMs lie in between).  Where tiles and heads are powers of two its runs also end
// where heads do (8 over 16384, 32/32: 57.5 and 63.0; over 16400: 61.8 and 63.9).
// One of tile pairs waits for the tensor cores and takes them all (256 sequences
// over 32768 tokens: 296 us, with 16 fewer 306, with half 386).
inline int shared_runs(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads,
                       int max_prefix, int num_sms) {
  const int64_t cost =
      shared_cost(num_seqs, num_groups, num_q_heads, num_kv_heads, max_prefix);
  int64_t most = num_sms;
  if (cost <= 6LL * num_sms)
    most = num_sms / 2;
  else if (num_seqs <= 128 / flash_packed_heads(num_q_heads / num_kv_heads))
    for (most = 1; 2 * most <= num_sms;) most *= 2;
  const int64_t runs = (cost + 1) / 2;
  return static_cast<int>(runs < 1 ? 1 : (runs < most ? runs : most));
}

struct DecodeSharedArgs {
  DecodeArgs decode;  // the whole decode, balanced split, its workspace
  const int32_t *group_starts, *prefix_lens;
  int32_t num_groups, max_prefix;
  int runs;            // CTAs of the prefix pass
  int64_t prefix_cost; // the most it can cost (shared_cost)
  int packed_heads;
  float scale_log2;    // |scale| * log2(e), not 0
  bool negate;         // the scale is negative
  int32_t q_off;       // scale 0: rows to move the query tiles by, out of the tensor
  CUtensorMap tm_q;    // box 64 x packed_heads x 128 / packed_heads
  CUtensorMap tm_k, tm_v;  // box 64 x 1 x block_size
  // [rows, D] and [rows, 2] states.  A group of n sequences takes n x packed_heads
  // rows per (head unit + block of its line): num_seqs x num_q_heads for the
  // head units, num_seqs x packed_heads + 256 x runs for the blocks (a block is
  // half a run long or more, or a group's last); 256 x runs keep runs apart.
  float *ws_o, *ws_ml;
  int32_t *ws_info;        // 8 words, then 8 per sequence
};
cudaError_t launch_decode_shared(const DecodeSharedArgs &a, cudaStream_t stream);

}  // namespace pa
