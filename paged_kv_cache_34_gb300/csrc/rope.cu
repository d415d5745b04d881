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
// a token at a time (few heads: several), a lane group per head in as many rounds as
// it needs, so that a token's cosines and sines are read once per lane whatever the
// number of heads.  A lane's next row, the next token's among them, is on its way
// while the current one is worked on, and the next token's position and slot before
// that; values stay fp32 pairs for two-wide arithmetic, as instructions are the next
// limit.  16 prompts up to 2000 tokens, 32/8 heads, with norms: 71 us, 6.1 TB/s of the
// 6.75 of a copy (76 with scalar arithmetic; 82 without the next row on its way too).
// 64 registers, 1024 threads an SM (with 94 and one CTA of 384 threads 149).
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

// Eight values as four fp32 pairs, for packed arithmetic.
template <class E>
__device__ __forceinline__ void unpack8(const uint4 &v, uint64_t (&f)[4]) {
  f[0] = f2_pack(E::lo(v.x), E::hi(v.x));
  f[1] = f2_pack(E::lo(v.y), E::hi(v.y));
  f[2] = f2_pack(E::lo(v.z), E::hi(v.z));
  f[3] = f2_pack(E::lo(v.w), E::hi(v.w));
}
template <class E>
__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f2_unpack(f[i], a, b);
    w[i] = E::pack2(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Neighbours (x, y) by the angle in the lower or upper half of c and s.
__device__ __forceinline__ uint64_t turn_pair(uint64_t v, uint64_t c, uint64_t s, bool upper) {
  float x, y, c0, c1, s0, s1;
  f2_unpack(v, x, y);
  f2_unpack(c, c0, c1);
  f2_unpack(s, s0, s1);
  if (upper) c0 = c1, s0 = s1;
  return f2_pack(x * c0 - y * s0, y * c0 + x * s0);
}

// NORM: some weight is given.  PAIRS: neighbouring elements are rotated.  SHARED: the
// CTA takes several tokens at once, with `groups` lane groups for each; otherwise one,
// with all its lanes.
template <class E, int D, bool NORM, bool PAIRS, bool SHARED>
__global__ void __launch_bounds__(512, 2) rope_and_cache_kernel(const RopeArgs p) {
  constexpr int L = D / 16;  // lanes per head
  using T = typename E::T;
  const int groups = SHARED ? p.groups : blockDim.x / L;
  const int at_once = SHARED ? blockDim.x / L / groups : 1;
  const int grp = SHARED ? threadIdx.x / L % groups : threadIdx.x / L;
  const int mine = SHARED ? threadIdx.x / L / groups : 0, ln = threadIdx.x % L;
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
  const uint32_t tokens = mine < at_once ? p.num_tokens : 0;  // (none for lanes left over)
  auto ahead = [&](uint32_t t) {
    if (t >= tokens) return;
    if (p.rot) pos = __ldg(p.positions + t);
    if (cache) slot = __ldg(p.slot_mapping + t);
  };
  // A lane's chunks of row r of token t: query heads, then key heads, then value heads.
  auto fetch = [&](uint32_t t, int r, uint4 &va, uint4 &vb) {
    if (t >= tokens || r >= rows) return;
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
  const uint32_t step = gridDim.x * at_once;
  ahead(blockIdx.x * at_once + mine);
  fetch(blockIdx.x * at_once + mine, grp, na, nb);
  // (every thread takes every turn: the norm's shuffles need whole warps)
  for (uint32_t t0 = blockIdx.x * at_once; t0 < p.num_tokens; t0 += step) {
    const uint32_t t = t0 + mine;
    const int64_t at = slot;
    const int row = pos;
    ahead(t + step);  // the next token's, while this one's rows are on their way
    const bool has = t < tokens;
    const bool known = has && (!p.rot || (row >= 0 && row < p.max_position));
    if (has && grp == 0 && ln == 0) {
      if (!known) raise_error(p.d_error, PA_DEVERR_POSITION);
      else if (at >= p.num_slots) raise_error(p.d_error, PA_DEVERR_SLOT);
    }
    const bool store = known && at >= 0 && at < p.num_slots;
    // Half-split: the pair's eight cosines, its sines and their negatives, two by two;
    // neighbours: the four cosines and sines of each chunk.
    uint64_t c[4], s[4], ns[PAIRS ? 1 : 4];
    if (turn && known) {
      const float *cs = p.cos_sin + static_cast<int64_t>(row) * p.rot;
      const float4 *x0 = reinterpret_cast<const float4 *>(cs + (PAIRS ? 4 * ca : 8 * ca));
      const float4 *x1 = PAIRS ? reinterpret_cast<const float4 *>(cs + 4 * cb) : x0 + 1;
      const int h4 = p.rot / 8;  // float4s of half a row
      const float4 v0 = __ldg(x0), v1 = __ldg(x1), v2 = __ldg(x0 + h4), v3 = __ldg(x1 + h4);
      c[0] = f2_pack(v0.x, v0.y), c[1] = f2_pack(v0.z, v0.w);
      c[2] = f2_pack(v1.x, v1.y), c[3] = f2_pack(v1.z, v1.w);
      s[0] = f2_pack(v2.x, v2.y), s[1] = f2_pack(v2.z, v2.w);
      s[2] = f2_pack(v3.x, v3.y), s[3] = f2_pack(v3.z, v3.w);
      if constexpr (!PAIRS) {
        ns[0] = f2_pack(-v2.x, -v2.y), ns[1] = f2_pack(-v2.z, -v2.w);
        ns[2] = f2_pack(-v3.x, -v3.y), ns[3] = f2_pack(-v3.z, -v3.w);
      }
    }
    for (int r0 = 0; r0 < rows; r0 += groups) {
      const int r = r0 + grp;
      uint4 va = na, vb = nb;
      if (r0 + groups < rows) fetch(t, r + groups, na, nb);
      else fetch(t + step, grp, na, nb);
      const bool live = known && r < rows, q = r < p.num_q_heads;
      const int kh = r - p.num_q_heads;  // the key head, or num_kv_heads + the value head
      const bool value = kh >= p.num_kv_heads;
      uint64_t a[4], b[4];
      unpack8<E>(va, a);
      unpack8<E>(vb, b);
      if constexpr (NORM) {
        const void *w = q ? p.q_weight : p.k_weight;
        uint64_t s2 = f2_mul(a[0], a[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s2 = f2_fma(a[i], a[i], s2);
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = f2_fma(b[i], b[i], s2);
        float ss, s1;
        f2_unpack(s2, ss, s1);
        ss += s1;
#pragma unroll
        for (int m = 1; m < L; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (w && live && !value) {
          const float f = rsqrtf(ss * (1.f / D) + p.eps);
          const uint64_t f2 = f2_pack(f, f);
          uint64_t wa[4];
          unpack8<E>(__ldg(reinterpret_cast<const uint4 *>(w) + ca), wa);
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = f2_mul(a[i], f2_mul(f2, wa[i]));
          unpack8<E>(__ldg(reinterpret_cast<const uint4 *>(w) + cb), wa);
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = f2_mul(b[i], f2_mul(f2, wa[i]));
        }
      }
      if (!live) continue;
      if (!value) {
        if (turn) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (PAIRS) {
              a[i] = turn_pair(a[i], c[i / 2], s[i / 2], i & 1);
              b[i] = turn_pair(b[i], c[2 + i / 2], s[2 + i / 2], i & 1);
            } else {
              const uint64_t a0 = a[i];
              a[i] = f2_fma(a0, c[i], f2_mul(b[i], ns[i]));
              b[i] = f2_fma(b[i], c[i], f2_mul(a0, s[i]));
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

template <class E, int D, bool SHARED>
cudaError_t launch(const RopeArgs &a, int threads, int64_t ctas, cudaStream_t stream) {
  const int64_t most = static_cast<int64_t>(a.num_sms) * (1024 / threads);
  const bool norm = a.q_weight || a.k_weight;
  auto kernel = norm ? (a.interleaved ? rope_and_cache_kernel<E, D, true, true, SHARED>
                                      : rope_and_cache_kernel<E, D, true, false, SHARED>)
                     : (a.interleaved ? rope_and_cache_kernel<E, D, false, true, SHARED>
                                      : rope_and_cache_kernel<E, D, false, false, SHARED>);
  const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
  return launch_pdl(kernel, grid, dim3(threads), 0, stream, a);
}

template <class E, int D>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
  constexpr int L = D / 16;
  // Where every token has a CTA at once, wide CTAs take its rows in one round; beyond
  // that, narrow ones keep more rounds' loads in flight (device us, 32/8 heads of 128, norms,
  // up to 512 and up to 128 threads: 32 tokens 2.4 and 2.7, 304 3.1 and 3.5, 380 4.5 and
  // 3.8, 456 4.5 and 3.8, 2432 13.6 and 10.8, 16700 103 and 70; without norms 304 2.6 and
  // 2.9, 380 3.7 and 3.1; up to 64 threads 68.8 and 10.0, but 456 4.8).
  const int rows = a.num_q_heads + a.num_kv_heads * (a.key_cache ? 2 : 1);
  const bool wide = a.num_tokens <= 2 * a.num_sms;
  const int widest = wide ? 512 : 128;
  int rounds = (rows * L + widest - 1) / widest;
  if (!wide && rounds == 1) {
    // Few heads: several tokens share a CTA, so that the rounds, and the loads on their
    // way, are several here too (8/2 heads of 64, norms, 1, 2, 3, 4 and 6 rounds: 1000
    // tokens 2.1, 2.6, 2.8, 3.3 and 3.9 us, 65000 53, 48, 44, 49 and 44; of 128: 3000
    // tokens 4.6, 4.5, 5.5, 5.3 and 6.5, 65000 95, 87, 79, 84 and 77).
    rounds = a.num_tokens < 32 * a.num_sms ? 2 : 6;
    if (rounds > rows) rounds = rows;
    RopeArgs p = a;
    p.groups = (rows + rounds - 1) / rounds;
    const int at_once = 128 / (p.groups * L);
    return launch<E, D, true>(p, (p.groups * at_once * L + 31) / 32 * 32,
                              (static_cast<int64_t>(a.num_tokens) + at_once - 1) / at_once, stream);
  }
  const int threads = ((rows + rounds - 1) / rounds * L + 31) / 32 * 32;
  return launch<E, D, false>(a, threads, a.num_tokens, stream);
}

}  // namespace rope

cudaError_t launch_rope_and_cache(const RopeArgs &a, cudaStream_t stream) {
  if (a.dtype == PA_BF16)
    return a.head_dim == 128 ? rope::launch<BF16, 128>(a, stream)
                             : rope::launch<BF16, 64>(a, stream);
  return a.head_dim == 128 ? rope::launch<F16, 128>(a, stream) : rope::launch<F16, 64>(a, stream);
}

}  // namespace pa
