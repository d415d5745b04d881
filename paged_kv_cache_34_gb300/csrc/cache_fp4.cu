// cache_fp4.cu -- the write into 4-bit pools, and their reading back as 16-bit rows.
//
// Write (cannbot-skills "model-infer-kvcache" skill page §3.1, §3.3; App. A quantised-KV
// scales): token t's key and value rows go to position slot % block_size of block
// slot / block_size, each group of 16 values under a scale of its own (pa_fp4.cuh).
// Read: position j of sequence b, through its block table, to row row_starts[b] + j.
//
// Design: HBM bound, each byte moved once.  A thread holds one group of 16: 32 bytes of
// 16-bit values on one side, 8 bytes of codes and a scale byte on the other.  D / 16
// neighbouring threads hold a head's row, so the 16-bit side is read or written as whole
// lines and a row's codes are 64 (32) consecutive bytes.
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace fp4 {

template <class E, int D>
__global__ void __launch_bounds__(256) reshape_and_cache_fp4_kernel(const ReshapeArgs p) {
  using TL = Tile<D>;
  constexpr int L = D / 16;  // threads per head row
  griddep_wait();  // inputs may come from the kernel just before this one
  griddep_launch_dependents();
  const int per = 2 * p.num_kv_heads * L;  // groups of a token, keys then values
  for (int64_t t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    const int64_t slot = __ldg(p.slot_mapping + t);
    if (slot < 0) continue;
    if (slot >= p.num_slots) {
      if (threadIdx.x == 0) raise_error(p.d_error, PA_DEVERR_SLOT);
      continue;
    }
    const int64_t block = slot / p.block_size;
    const int off = static_cast<int>(slot - block * p.block_size);
    for (int i = threadIdx.x; i < per; i += blockDim.x) {
      const bool value = i >= p.num_kv_heads * L;
      const int j = value ? i - p.num_kv_heads * L : i, h = j / L, g = j % L;
      const char *row = static_cast<const char *>(value ? p.value : p.key) + t * p.row_stride_bytes;
      const uint4 *src = reinterpret_cast<const uint4 *>(row) + 2 * j;
      const uint4 a = __ldg(src), b = __ldg(src + 1);
      const float S = __ldg((value ? p.v_scale : p.k_scale) + h);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      float x[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[2 * e] = E::lo(w[e]);
        x[2 * e + 1] = E::hi(w[e]);
      }
      uint32_t scale = 0;
      uint2 codes = make_uint2(0, 0);
      if (head_scale_ok(S)) codes = quantise16(x, S, scale);
      else raise_error(p.d_error, PA_DEVERR_SCALE);
      uint8_t *tile = static_cast<uint8_t *>(value ? p.value_cache : p.key_cache) +
                      ((block * p.num_kv_heads + h) * (p.block_size / 8) + off / 8) * TL::kBytes;
      *reinterpret_cast<uint2 *>(tile + (off % 8) * TL::kRowBytes + 8 * g) = codes;
      tile[TL::kScales + (off % 8) * TL::kScaleBytes + g] = static_cast<uint8_t>(scale);
    }
  }
}

template <class E, int D>
__global__ void __launch_bounds__(256) gather_cache_fp4_kernel(const GatherArgs p) {
  using TL = Tile<D>;
  constexpr int L = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  const int len = checked_context_len(__ldg(p.context_lens + b), p.capacity, p.max_context_len,
                                      p.d_error, blockIdx.x == 0 && threadIdx.x == 0);
  if (len == 0) return;
  const int start = __ldg(p.row_starts + b);
  if (start < 0 || start > p.num_rows - len) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(p.d_error, PA_DEVERR_CU_SEQLENS);
    return;
  }
  const int per = 2 * p.num_kv_heads * L;
  for (int j = blockIdx.x; j < len; j += gridDim.x) {
    const int lb = j / p.block_size, off = j - lb * p.block_size;
    const int id = __ldg(p.block_table + b * p.block_table_stride + lb);
    if (id < 0 || id >= p.num_blocks) {
      if (threadIdx.x == 0) raise_error(p.d_error, PA_DEVERR_BLOCK_ID);
      continue;
    }
    for (int i = threadIdx.x; i < per; i += blockDim.x) {
      const bool value = i >= p.num_kv_heads * L;
      const int k = value ? i - p.num_kv_heads * L : i, h = k / L, g = k % L;
      const uint8_t *tile =
          static_cast<const uint8_t *>(value ? p.value_cache : p.key_cache) +
          ((static_cast<int64_t>(id) * p.num_kv_heads + h) * (p.block_size / 8) + off / 8) *
              TL::kBytes;
      const uint2 codes =
          *reinterpret_cast<const uint2 *>(tile + (off % 8) * TL::kRowBytes + 8 * g);
      const float s =
          F16::lo(e4m3_to_f16x2(tile[TL::kScales + (off % 8) * TL::kScaleBytes + g]));
      float S = __ldg((value ? p.v_scale : p.k_scale) + h);
      if (!head_scale_ok(S)) {
        raise_error(p.d_error, PA_DEVERR_SCALE);
        S = 0.f;
      }
      uint32_t c[8], w[8];
      widen8(codes.x, c[0], c[1], c[2], c[3]);
      widen8(codes.y, c[4], c[5], c[6], c[7]);
      // code * scale is exact (at most six bits); times S it is rounded to fp32, then to 16
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = E::pack2(F16::lo(c[e]) * s * S, F16::hi(c[e]) * s * S);
      const int64_t row = start + j;
      uint4 *dst = reinterpret_cast<uint4 *>(
                       static_cast<char *>(value ? p.value_out : p.key_out) +
                       row * (value ? p.v_stride_bytes : p.k_stride_bytes)) + 2 * k;
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

}  // namespace fp4

cudaError_t launch_reshape_and_cache_fp4(const ReshapeArgs &a, cudaStream_t stream) {
  const int per = 2 * a.num_kv_heads * a.head_dim / 16;
  const int threads = per < 256 ? (per + 31) / 32 * 32 : 256;
  const int64_t most = static_cast<int64_t>(a.num_sms) * (2048 / threads);
  const int grid = static_cast<int>(a.num_tokens < most ? a.num_tokens : most);
  auto kernel = a.dtype == PA_BF16 ? (a.head_dim == 128 ? fp4::reshape_and_cache_fp4_kernel<BF16, 128>
                                                        : fp4::reshape_and_cache_fp4_kernel<BF16, 64>)
                                   : (a.head_dim == 128 ? fp4::reshape_and_cache_fp4_kernel<F16, 128>
                                                        : fp4::reshape_and_cache_fp4_kernel<F16, 64>);
  return launch_pdl(kernel, dim3(grid), dim3(threads), 0, stream, a);
}

cudaError_t launch_gather_cache_fp4(const GatherArgs &a, cudaStream_t stream) {
  const int per = 2 * a.num_kv_heads * a.head_dim / 16;
  const int threads = per < 256 ? (per + 31) / 32 * 32 : 256;
  const int64_t most = static_cast<int64_t>(a.num_sms) * (2048 / threads) * 2;
  int64_t x = (most + a.num_seqs - 1) / a.num_seqs;
  if (x > a.max_context_len) x = a.max_context_len;
  auto kernel = a.dtype == PA_BF16 ? (a.head_dim == 128 ? fp4::gather_cache_fp4_kernel<BF16, 128>
                                                        : fp4::gather_cache_fp4_kernel<BF16, 64>)
                                   : (a.head_dim == 128 ? fp4::gather_cache_fp4_kernel<F16, 128>
                                                        : fp4::gather_cache_fp4_kernel<F16, 64>);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(x), static_cast<unsigned>(a.num_seqs)),
                    dim3(threads), 0, stream, a);
}

}  // namespace pa
