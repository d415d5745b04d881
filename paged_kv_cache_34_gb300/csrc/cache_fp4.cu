// cache_fp4.cu -- the write into 4-bit pools, and their reading back as 16-bit rows.
//
// Write (cannbot-skills "model-infer-kvcache" skill page §3.1, §3.3; App. A quantised-KV
// scales): token t's key and value rows go to position slot % block_size of block
// slot / block_size, each group of 16 values under a scale of its own (pa_fp4.cuh).
// Read: position j of sequence b, through its block table, to row row_starts[b] + j.
//
// Design: HBM bound, each byte moved once; next to that by the quotients (write) and
// conversions (read) of every value.
//  * Write: a thread holds one group of 16 of a row (D / 16 neighbours a head), the same
//    head's in every token it takes, so that what a head's groups share is worked out
//    once; the next token's values are on their way meanwhile.
//  * Read: a thread holds eight elements of a head's row, so that rows are written in whole
//    lines, and takes a tile of eight tokens at a time: one block id, eight rows on their way.
//    CTAs have a sequence each, or, where lengths may be far apart, all sequences' tiles by turns.
// Measured (16 prompts up to 2000 tokens, 32 KV heads of 128, bf16, 333 MB each way): write
// 55 us, 6.0 TB/s; read 57 us, 5.8 TB/s, of the 6.75 of a copy; 162 us together with a
// thread per group and token in both and the checked quotient throughout.
#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace fp4 {

// A token has 2 Hkv D / 16 groups (keys, then values): blockIdx.y says which blockDim.x of
// them, or, where a CTA has room for several tokens, blockDim.x is that many times as much.
template <class E, int D>
__global__ void __launch_bounds__(256, 4) reshape_and_cache_fp4_kernel(const ReshapeArgs p) {
  using TL = Tile<D>;
  constexpr int L = D / 16;  // threads per head row
  const int half = p.num_kv_heads * L;
  const int tokens = gridDim.y > 1 ? 1 : blockDim.x / (2 * half);  // of a CTA at a time
  const int mine = gridDim.y > 1 ? 0 : threadIdx.x / (2 * half);
  const int i = blockIdx.y * blockDim.x + threadIdx.x - mine * 2 * half;
  const bool value = i >= half, live = i < 2 * half;
  const int j = value ? i - half : i, h = j / L, g = j % L;
  griddep_wait();  // inputs may come from the kernel just before this one
  griddep_launch_dependents();
  if (!live) return;
  const HeadScale hs(__ldg((value ? p.v_scale : p.k_scale) + h));
  const char *rows = static_cast<const char *>(value ? p.value : p.key) + 32 * j;
  uint8_t *pool = static_cast<uint8_t *>(value ? p.value_cache : p.key_cache);
  const int shift = 31 - __clz(p.block_size);
  int64_t slot = -1;
  uint4 a, b;
  const uint32_t t0 = blockIdx.x * tokens + mine, step = gridDim.x * tokens;
  const char *src = rows + t0 * p.row_stride_bytes;  // the next token's
  const int64_t *slots = p.slot_mapping + t0;
  const int64_t src_step = step * p.row_stride_bytes;
  auto fetch = [&](uint32_t t) {
    if (t >= static_cast<uint32_t>(p.num_tokens)) return;
    slot = __ldg(slots);
    a = __ldg(reinterpret_cast<const uint4 *>(src));
    b = __ldg(reinterpret_cast<const uint4 *>(src) + 1);
    slots += step;
    src += src_step;
  };
  fetch(t0);
  for (uint32_t t = t0; t < static_cast<uint32_t>(p.num_tokens); t += step) {
    const int64_t at = slot;
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    fetch(t + step);
    if (at < 0) continue;
    if (at >= p.num_slots) {
      if (i == 0) raise_error(p.d_error, PA_DEVERR_SLOT);
      continue;
    }
    if (hs.s == 0.f) raise_error(p.d_error, PA_DEVERR_SCALE);
    uint32_t scale;
    const uint2 codes = quantise16<E>(v, hs, scale);
    const int64_t block = at >> shift;
    const uint32_t off = static_cast<uint32_t>(at) & (p.block_size - 1), row = off & 7;
    uint8_t *tile = pool + (((block * p.num_kv_heads + h) << (shift - 3)) + (off >> 3)) * TL::kBytes;
    *reinterpret_cast<uint2 *>(tile + row * TL::kRowBytes + 8 * g) = codes;
    tile[TL::kScales + row * TL::kScaleBytes + g] = static_cast<uint8_t>(scale);
  }
}

// One tile's `n` rows of one 16-byte chunk: chunk c of head scale S, rows `stride` bytes apart.
template <class E, int D>
__device__ __forceinline__ void gather_tile(const uint8_t *tile, char *dst, int64_t stride, int n,
                                            float S, int c) {
  using TL = Tile<D>;
  if (S == 0.f) {  // zeros, even where the pool's scales are NaN
    for (int r = 0; r < n; ++r)
      *reinterpret_cast<uint4 *>(dst + r * stride) = make_uint4(0, 0, 0, 0);
    return;
  }
  // (all eight rows of a tile are the pool's, whatever the context ends at)
  uint32_t codes[8], scale[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    codes[r] = *reinterpret_cast<const uint32_t *>(tile + r * TL::kRowBytes + 4 * c);
    scale[r] = tile[TL::kScales + r * TL::kScaleBytes + c / 2];
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if (r >= n) break;
    uint32_t e[4], w[4];
    widen8(codes[r], e[0], e[1], e[2], e[3]);
    // code * scale is exact in fp16 (six bits); times S it is rounded to fp32, then to 16
    const uint32_t f = e4m3_to_f16x2(scale[r] * 0x101u);
    const __half2 s2 = *reinterpret_cast<const __half2 *>(&f);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&e[x]), s2);
      const uint32_t z = *reinterpret_cast<const uint32_t *>(&y);
      w[x] = E::pack2(F16::lo(z) * S, F16::hi(z) * S);
    }
    *reinterpret_cast<uint4 *>(dst + r * stride) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// blockIdx.y: the sequence; blockIdx.z: which blockDim.x of the 2 Hkv D / 8 chunks of a row.
template <class E, int D>
__global__ void __launch_bounds__(256) gather_cache_fp4_kernel(const GatherArgs p) {
  using TL = Tile<D>;
  constexpr int L = D / 8;
  const int i = blockIdx.z * blockDim.x + threadIdx.x, half = p.num_kv_heads * L;
  const bool value = i >= half, first = blockIdx.x == 0 && i == 0;
  const int k = value ? i - half : i, h = k / L, c = k % L;
  griddep_wait();
  griddep_launch_dependents();
  if (i >= 2 * half) return;
  const int b = blockIdx.y;
  const int len = checked_context_len(__ldg(p.context_lens + b), p.capacity, p.max_context_len,
                                      p.d_error, first);
  if (len == 0) return;
  const int start = __ldg(p.row_starts + b);
  if (start < 0 || start > p.num_rows - len) {
    if (first) raise_error(p.d_error, PA_DEVERR_CU_SEQLENS);
    return;
  }
  float S = __ldg((value ? p.v_scale : p.k_scale) + h);
  if (!head_scale_ok(S)) {
    raise_error(p.d_error, PA_DEVERR_SCALE);
    S = 0.f;
  }
  const uint8_t *pool = static_cast<const uint8_t *>(value ? p.value_cache : p.key_cache);
  const int64_t stride = value ? p.v_stride_bytes : p.k_stride_bytes;
  char *out = static_cast<char *>(value ? p.value_out : p.key_out) + start * stride + 16 * k;
  const int32_t *table = p.block_table + b * p.block_table_stride;
  const int shift = 31 - __clz(p.block_size) - 3, tiles = (len + 7) / 8;  // (tiles a block: 2^shift)
  int id = static_cast<int>(blockIdx.x) < tiles ? __ldg(table + (blockIdx.x >> shift)) : 0;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int now = id;
    if (t + static_cast<int>(gridDim.x) < tiles) id = __ldg(table + ((t + gridDim.x) >> shift));
    if (now < 0 || now >= p.num_blocks) {
      if (i == 0) raise_error(p.d_error, PA_DEVERR_BLOCK_ID);
      continue;
    }
    const uint8_t *tile = pool + (((static_cast<int64_t>(now) * p.num_kv_heads + h) << shift) +
                                  (t & ((1 << shift) - 1))) * TL::kBytes;
    gather_tile<E, D>(tile, out + 8 * static_cast<int64_t>(t) * stride, stride, min(8, len - 8 * t),
                      S, c);
  }
}

// The tiles of all sequences as one list, dealt out to the CTAs in turn.  A CTA goes through
// the sequences kListSeqs at a time: their tiles are summed up, and those of its places that
// fall among them are looked up by bisection.  blockIdx.y: which blockDim.x of a row's chunks;
// where a CTA has room for several rows, that many tiles share a turn.
constexpr int kListSeqs = 256;

template <class E, int D>
__global__ void __launch_bounds__(kListSeqs) gather_list_fp4_kernel(const GatherArgs p) {
  using TL = Tile<D>;
  constexpr int L = D / 8;
  __shared__ int64_t s_sum[kListSeqs + 1];  // tiles ahead of each sequence
  __shared__ int64_t s_warp[kListSeqs / 32];
  __shared__ int s_len[kListSeqs], s_start[kListSeqs];
  const int half = p.num_kv_heads * L, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int at_once = 2 * half < kListSeqs ? kListSeqs / (2 * half) : 1;
  const int mine = at_once > 1 ? tid / (2 * half) : 0;
  const int i = blockIdx.y * kListSeqs + tid - mine * 2 * half;
  const bool value = i >= half, live = i < 2 * half && mine < at_once;
  const int k = value ? i - half : i, h = k / L, c = k % L;
  const bool report = blockIdx.x == 0 && blockIdx.y == 0;
  griddep_wait();
  griddep_launch_dependents();
  float S = live ? __ldg((value ? p.v_scale : p.k_scale) + h) : 1.f;
  bool tell = !head_scale_ok(S);  // once
  if (tell) S = 0.f;
  const uint8_t *pool = static_cast<const uint8_t *>(value ? p.value_cache : p.key_cache);
  const int64_t stride = value ? p.v_stride_bytes : p.k_stride_bytes;
  char *out = static_cast<char *>(value ? p.value_out : p.key_out) + 16 * k;
  const int shift = 31 - __clz(p.block_size) - 3;  // (tiles a block: 2^shift)
  if (tid == 0) s_sum[0] = 0;
  int64_t at = static_cast<int64_t>(blockIdx.x) * at_once + mine;  // place in the list from here on
  const int64_t step = static_cast<int64_t>(gridDim.x) * at_once;
  int len = 0, start = 0;
  auto fetch = [&](int b) {  // a thread's sequence of the next round
    len = b < p.num_seqs ? __ldg(p.context_lens + b) : 0;
    start = b < p.num_seqs ? __ldg(p.row_starts + b) : 0;
  };
  fetch(tid);
  for (int base = 0; base < p.num_seqs; base += kListSeqs) {
    int n = checked_context_len(len, p.capacity, p.max_context_len, p.d_error, report);
    if (n > 0 && (start < 0 || start > p.num_rows - n)) {
      if (report) raise_error(p.d_error, PA_DEVERR_CU_SEQLENS);
      n = 0;
    }
    s_len[tid] = n;
    s_start[tid] = start;
    fetch(base + kListSeqs + tid);
    int64_t sum = (n + 7) / 8;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += s_warp[w];
    s_sum[tid + 1] = sum;
    __syncthreads();
    const int64_t total = s_sum[kListSeqs];
    int q = 0, t = 0, id = 0;  // the place's sequence, its tile and its block
    auto look = [&]() {
      if (at >= total) return;
      int lo = 0;
#pragma unroll
      for (int w = kListSeqs / 2; w > 0; w >>= 1)
        if (s_sum[lo + w] <= at) lo += w;
      q = lo;
      t = static_cast<int>(at - s_sum[lo]);
      id = __ldg(p.block_table + (base + lo) * p.block_table_stride + (t >> shift));
    };
    if (live) {
      look();
      while (at < total) {
        const int now = id, tile = t, rows = s_len[q];
        const int64_t row = s_start[q] + 8 * static_cast<int64_t>(t);
        at += step;
        look();
        if (tell) raise_error(p.d_error, PA_DEVERR_SCALE);
        tell = false;
        if (now < 0 || now >= p.num_blocks) {
          if (i == 0) raise_error(p.d_error, PA_DEVERR_BLOCK_ID);
          continue;
        }
        const int64_t place = (static_cast<int64_t>(now) * p.num_kv_heads + h) << shift;
        gather_tile<E, D>(pool + (place + (tile & ((1 << shift) - 1))) * TL::kBytes,
                          out + row * stride, stride, min(8, rows - 8 * tile), S, c);
      }
    }
    at -= total;
    __syncthreads();  // everyone is done with the sums
  }
}

}  // namespace fp4

cudaError_t launch_reshape_and_cache_fp4(const ReshapeArgs &a, cudaStream_t stream) {
  const int per = 2 * a.num_kv_heads * a.head_dim / 16;
  const int tokens = per <= 128 ? 256 / per : 1, parts = (per + 255) / 256;
  const int threads = parts > 1 ? 256 : per * tokens;
  const int64_t ctas = (static_cast<int64_t>(a.num_tokens) + tokens - 1) / tokens;
  // As many CTAs as run at once, four an SM: a thread's next token is on its way while it
  // works on one (4, 8, 10 and 24 an SM: 16 prompts up to 2000 tokens, 32 heads, 55.3, 55.6,
  // 59.0, 57.9 us; 64 of 300 to 500, 8 heads, 23.8, 24.4, 26.0, 27.1; three resident 61,
  // five, of 51 registers, 61).
  const int64_t most = (static_cast<int64_t>(a.num_sms) * 4 + parts - 1) / parts;
  const int grid = static_cast<int>(ctas < most ? ctas : most);
  auto kernel = a.dtype == PA_BF16 ? (a.head_dim == 128 ? fp4::reshape_and_cache_fp4_kernel<BF16, 128>
                                                        : fp4::reshape_and_cache_fp4_kernel<BF16, 64>)
                                   : (a.head_dim == 128 ? fp4::reshape_and_cache_fp4_kernel<F16, 128>
                                                        : fp4::reshape_and_cache_fp4_kernel<F16, 64>);
  return launch_pdl(kernel, dim3(grid, parts), dim3(threads), 0, stream, a);
}

cudaError_t launch_gather_cache_fp4(const GatherArgs &a, cudaStream_t stream) {
  const int per = 2 * a.num_kv_heads * a.head_dim / 8;
  const int threads = per < 256 ? (per + 31) / 32 * 32 : 256;
  const int parts = (per + threads - 1) / threads;
  const int64_t tiles = (static_cast<int64_t>(a.max_context_len) + 7) / 8;
  // 4096 threads an SM over all sequences (8192, 2048: 6 sequences of 1500 to 8000 tokens,
  // 8 KV heads, 24.0 us, 25.7, 26.3; 16 up to 2000, 32 KV heads, 57.2, 54.7, 61.8).
  int64_t x = (static_cast<int64_t>(a.num_sms) * (4096 / threads) + parts - 1) / parts;
  x = (x + a.num_seqs - 1) / a.num_seqs;
  if (x > tiles) x = tiles;
  // Where a CTA may have more than eight tiles of its sequence to go through, lengths far
  // apart would leave most of them idle behind one long context: all sequences' tiles as one
  // list instead (each for itself / list, us, 8 heads of 128: one of 100000 among 127 of 100
  // 760 / 98, among 1999 6050 / 256; one of 10000 among 31 of 100 21 / 13; but even lengths,
  // 16 of 20000 267 / 269, 16 of 2000 with 32 heads, at most 6.6 tiles a CTA, 110 / 113, 64 of
  // 10000 with 2 heads of 64, 4.1 tiles, 70.7 / 74).
  if (a.num_seqs > 1 && tiles > 8 * x) {
    // 16 CTAs an SM, four of them resident, where the lengths are one round of sums, else
    // the resident ones alone (4 / 16: 16 of 20000 274 / 269, one of 100000 among 127 of 100
    // 100 / 98; among 5000 of 64, 2 heads of 64, 58 / 98, one of 30000 among 40000 172 / 528).
    const int per_sm = a.num_seqs <= fp4::kListSeqs ? 16 : 4;
    const int lists = (per + fp4::kListSeqs - 1) / fp4::kListSeqs;
    int64_t ctas = (static_cast<int64_t>(a.num_sms) * per_sm + lists - 1) / lists;
    const int64_t places = a.num_rows / 8 + static_cast<int64_t>(a.num_seqs);  // tiles at most
    if (ctas > places) ctas = places;
    auto kernel = a.dtype == PA_BF16 ? (a.head_dim == 128 ? fp4::gather_list_fp4_kernel<BF16, 128>
                                                          : fp4::gather_list_fp4_kernel<BF16, 64>)
                                     : (a.head_dim == 128 ? fp4::gather_list_fp4_kernel<F16, 128>
                                                          : fp4::gather_list_fp4_kernel<F16, 64>);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(lists)),
                      dim3(fp4::kListSeqs), 0, stream, a);
  }
  auto kernel = a.dtype == PA_BF16 ? (a.head_dim == 128 ? fp4::gather_cache_fp4_kernel<BF16, 128>
                                                        : fp4::gather_cache_fp4_kernel<BF16, 64>)
                                   : (a.head_dim == 128 ? fp4::gather_cache_fp4_kernel<F16, 128>
                                                        : fp4::gather_cache_fp4_kernel<F16, 64>);
  return launch_pdl(kernel,
                    dim3(static_cast<unsigned>(x), static_cast<unsigned>(a.num_seqs),
                         static_cast<unsigned>(parts)),
                    dim3(threads), 0, stream, a);
}

}  // namespace pa
