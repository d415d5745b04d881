// rope.cu -- norm and position rotation of a step's query and key heads, and
// the write of its keys and values into the paged pools, in one pass.
//
// Operation: token t at position p = positions[t]; a query or key head's row x
// of D values becomes, in fp32,
//     y   = x * rsqrt(mean(x^2) + eps) * w        (with a weight; else y = x)
//     y_a, y_b -> y_a c_i - y_b s_i, y_b c_i + y_a s_i      for i < R / 2,
// where (a, b) is (i, i + R / 2), or (2i, 2i + 1) when interleaved, and c, s are
// the table's row p (R / 2 cosines, then R / 2 sines); elements from R on keep y.
// One rounding to 16 bits follows.  Keys and values then go to pool row
// slot_mapping[t] (cannbot-skills "model-infer-kvcache" skill page §3.1, §3.3).
//
// Design: HBM bound; every byte is moved once.  D / 16 lanes hold a head's row, 16
// values each: chunk j and its partner R / 16 chunks on, so that both halves of a
// rotated pair sit in one lane and a norm takes log2(D / 16) shuffles.  A CTA takes
// a token at a time, a lane group per head in as many rounds as it needs, so that a
// token's cosines and sines are read once per lane whatever the number of heads.  A
// lane's next row, the next token's among them, is on its way while the current one
// is worked on, and the next token's position and slot before that (16 prompts up to
// 2000 tokens, 32/8 heads, with norms: 76 us, 5.7 TB/s of the 6.75 of a copy; without
// the next row on its way 82).  64 registers, 1024 threads an SM (with 94 and one CTA
// of 384 threads 149).
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace rope {

// 16 bytes of a row that may be rewritten in place by the thread that reads it.
__device__ __forceinline__ uint4 load_row(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <class E>
__device__ __forceinline__ void unpack8(const uint4 &v, float *f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = E::lo(w[i]);
    f[2 * i + 1] = E::hi(w[i]);
  }
}
template <class E>
__device__ __forceinline__ uint4 pack8(const float *f) {
  return make_uint4(E::pack2(f[0], f[1]), E::pack2(f[2], f[3]), E::pack2(f[4], f[5]),
                    E::pack2(f[6], f[7]));
}

// NORM: some weight is given.  PAIRS: neighbouring elements are rotated.
template <class E, int D, bool NORM, bool PAIRS>
__global__ void __launch_bounds__(512, 2) rope_and_cache_kernel(const RopeArgs p) {
  constexpr int L = D / 16;  // lanes per head
  using T = typename E::T;
  const int grp = threadIdx.x / L, ln = threadIdx.x % L, groups = blockDim.x / L;
  const int half = p.rot / 16;  // 8-element chunks of half of the rotated part
  // this lane's chunks: a rotated pair, or two that pass
  const bool turn = ln < half;
  const int ca = turn ? ln : 2 * half + 2 * (ln - half), cb = turn ? ln + half : ca + 1;
  const bool cache = p.key_cache != nullptr;
  const int rows = p.num_q_heads + p.num_kv_heads * (cache ? 2 : 1);
  griddep_wait();  // inputs may come from the kernel just before this one
  griddep_launch_dependents();
  int64_t slot = -1;
  int pos = 0;
  auto ahead = [&](int64_t t) {
    if (t >= p.num_tokens) return;
    if (p.rot) pos = __ldg(p.positions + t);
    if (cache) slot = __ldg(p.slot_mapping + t);
  };
  // A lane's chunks of row r of token t: query heads, then key heads, then value heads.
  auto fetch = [&](int64_t t, int r, uint4 &va, uint4 &vb) {
    if (t >= p.num_tokens || r >= rows) return;
    int h = r - p.num_q_heads;
    const T *src = static_cast<const T *>(p.query) + t * p.q_row_stride + r * D;
    if (h >= 0) {
      const bool value = h >= p.num_kv_heads;
      if (value) h -= p.num_kv_heads;
      src = static_cast<const T *>(value ? p.value : p.key) + t * p.kv_row_stride + h * D;
    }
    va = load_row(src + 8 * ca);
    vb = load_row(src + 8 * cb);
  };
  uint4 na, nb;  // the chunks of the row after the current one
  ahead(blockIdx.x);
  fetch(blockIdx.x, grp, na, nb);
  for (int64_t t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    const int64_t at = slot;
    const int row = pos;
    ahead(t + gridDim.x);  // the next token's, while this one's rows are on their way
    const bool known = !p.rot || (row >= 0 && row < p.max_position);
    if (threadIdx.x == 0) {
      if (!known) raise_error(p.d_error, PA_DEVERR_POSITION);
      else if (at >= p.num_slots) raise_error(p.d_error, PA_DEVERR_SLOT);
    }
    const bool store = known && at >= 0 && at < p.num_slots;
    float c[8], s[8];
    if (turn && known) {  // half-split: the pair's eight angles; neighbours: four for each chunk
      const float *cs = p.cos_sin + static_cast<int64_t>(row) * p.rot;
      const float4 *x0 = reinterpret_cast<const float4 *>(cs + (PAIRS ? 4 * ca : 8 * ca));
      const float4 *x1 = PAIRS ? reinterpret_cast<const float4 *>(cs + 4 * cb) : x0 + 1;
      const int h4 = p.rot / 8;  // float4s of half a row
      const float4 v0 = __ldg(x0), v1 = __ldg(x1), v2 = __ldg(x0 + h4), v3 = __ldg(x1 + h4);
      c[0] = v0.x, c[1] = v0.y, c[2] = v0.z, c[3] = v0.w;
      c[4] = v1.x, c[5] = v1.y, c[6] = v1.z, c[7] = v1.w;
      s[0] = v2.x, s[1] = v2.y, s[2] = v2.z, s[3] = v2.w;
      s[4] = v3.x, s[5] = v3.y, s[6] = v3.z, s[7] = v3.w;
    }
    // every lane takes every round: the norm's shuffles need whole warps
    for (int r0 = 0; r0 < rows; r0 += groups) {
      const int r = r0 + grp;
      uint4 va = na, vb = nb;
      if (r0 + groups < rows) fetch(t, r + groups, na, nb);
      else fetch(t + gridDim.x, grp, na, nb);
      const bool live = known && r < rows, q = r < p.num_q_heads;
      const int kh = r - p.num_q_heads;  // the key head, or num_kv_heads + the value head
      const bool value = kh >= p.num_kv_heads;
      float a[8], b[8];
      unpack8<E>(va, a);
      unpack8<E>(vb, b);
      if constexpr (NORM) {
        const void *w = q ? p.q_weight : p.k_weight;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
#pragma unroll
        for (int m = 1; m < L; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (w && live && !value) {
          const float f = rsqrtf(ss * (1.f / D) + p.eps);
          float wa[8];
          unpack8<E>(__ldg(reinterpret_cast<const uint4 *>(w) + ca), wa);
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] *= f * wa[i];
          unpack8<E>(__ldg(reinterpret_cast<const uint4 *>(w) + cb), wa);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] *= f * wa[i];
        }
      }
      if (!live) continue;
      if (!value) {
        if (turn) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if constexpr (PAIRS) {
              if (i & 1) continue;
              const float a0 = a[i], b0 = b[i];
              a[i] = a0 * c[i / 2] - a[i + 1] * s[i / 2];
              a[i + 1] = a[i + 1] * c[i / 2] + a0 * s[i / 2];
              b[i] = b0 * c[4 + i / 2] - b[i + 1] * s[4 + i / 2];
              b[i + 1] = b[i + 1] * c[4 + i / 2] + b0 * s[4 + i / 2];
            } else {
              const float a0 = a[i];
              a[i] = a0 * c[i] - b[i] * s[i];
              b[i] = b[i] * c[i] + a0 * s[i];
            }
          }
        }
        va = pack8<E>(a);
        vb = pack8<E>(b);
        if (q || p.key_out) {
          T *dst = q ? static_cast<T *>(p.query_out) + t * p.q_out_row_stride + r * D
                     : static_cast<T *>(p.key_out) + t * p.k_out_row_stride + kh * D;
          *reinterpret_cast<uint4 *>(dst + 8 * ca) = va;
          *reinterpret_cast<uint4 *>(dst + 8 * cb) = vb;
        }
      }
      if (!q && store) {
        T *dst = static_cast<T *>(value ? p.value_cache : p.key_cache) +
                 (at * p.num_kv_heads + kh - (value ? p.num_kv_heads : 0)) * D;
        *reinterpret_cast<uint4 *>(dst + 8 * ca) = va;
        *reinterpret_cast<uint4 *>(dst + 8 * cb) = vb;
      }
    }
  }
}

template <class E, int D>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
  constexpr int L = D / 16;
  // Where every token has a CTA at once, wide CTAs take its rows in one round; beyond
  // that, narrow ones keep more rounds' loads in flight (32/8 heads, norms, up to 512
  // and up to 128 threads: 32 tokens 2.4 and 3.6 us, 304 3.1 and 4.0, 456 5.1 and 4.2,
  // 2432 21.2 and 13.9, 16700 122 and 76.5; up to 64 threads 76.1 and 13.3, but 456
  // 6.4).
  const int rows = a.num_q_heads + a.num_kv_heads * (a.key_cache ? 2 : 1);
  const int widest = a.num_tokens <= 2 * a.num_sms ? 512 : 128;
  const int rounds = (rows * L + widest - 1) / widest;
  const int threads = ((rows + rounds - 1) / rounds * L + 31) / 32 * 32;
  const int64_t most = static_cast<int64_t>(a.num_sms) * (1024 / threads);
  const int grid = static_cast<int>(a.num_tokens < most ? a.num_tokens : most);
  const bool norm = a.q_weight || a.k_weight;
  auto kernel = norm ? (a.interleaved ? rope_and_cache_kernel<E, D, true, true>
                                      : rope_and_cache_kernel<E, D, true, false>)
                     : (a.interleaved ? rope_and_cache_kernel<E, D, false, true>
                                      : rope_and_cache_kernel<E, D, false, false>);
  return launch_pdl(kernel, dim3(grid), dim3(threads), 0, stream, a);
}

}  // namespace rope

cudaError_t launch_rope_and_cache(const RopeArgs &a, cudaStream_t stream) {
  if (a.dtype == PA_BF16)
    return a.head_dim == 128 ? rope::launch<BF16, 128>(a, stream)
                             : rope::launch<BF16, 64>(a, stream);
  return a.head_dim == 128 ? rope::launch<F16, 128>(a, stream) : rope::launch<F16, 64>(a, stream);
}

}  // namespace pa
