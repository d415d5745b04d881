// decode_shared.cu -- paged decode of a batch whose groups of sequences share
// a prefix: the prefix is read once for its whole group.
//
// Operation: pa_decode's (cannbot-skills page §3.1, §3.6; mhpq.cn article
// §3.3), with sequence b's first P keys and values taken from the block-table
// row of its group's first sequence (the coreui.cn page's shared, ref-counted
// pages: requests forked from one prompt hold the same pages).  Softmax states
// over disjoint keys join exactly: with (m_i, l_i, o_i) the maximum, the sum
// and the unnormalised output over part i,
//     M = max_i m_i,  out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
//
// Three launches:
//  1. the prefix pass (flash_kernel.cuh): all of a group's (sequence, head)
//     rows of one KV head are query rows of tensor-core tiles over the
//     prefix's pages, split over the keys into equal runs;
//  2. the own parts: the decode kernel over each sequence's tokens from P on,
//     every piece leaving its state.  It depends on nothing of launch 1 and
//     starts on SMs as that frees them;
//  3. the join below.
#include <math.h>

#include "decode_kernel.cuh"
#include "flash_kernel.cuh"

namespace pa {

namespace {

constexpr int kJoinWarps = 4;
constexpr int kJoinBatch = 4;  // states in flight per warp

// One CTA per (sequence, query head).  Its states are those of the own
// part's pieces (runs of the balanced split) and of the prefix's runs; warp w
// folds states w, w + 4, ..., the warps' results are folded in shared memory.
template <class E, int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
    shared_join_kernel(const dec::DecodeParams p, const float *px_o, const float *px_ml,
                       const int32_t *info, int pg, int tpt) {
  constexpr int V = D / 32;  // output elements per lane
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  __shared__ float s_o[kJoinWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.hq, h = blockIdx.x - b * p.hq;
  const int L = checked_context_len(__ldg(p.context_lens + b), p.capacity, p.max_ctx, p.err, false);
  griddep_wait();  // both launches' states
  griddep_launch_dependents();
  const int32_t *seq = info + static_cast<int64_t>(b + 1) * flash::kInfoWords;
  const int prefix = seq[0];

  // own part: rows own_row + i * hs of ws_o, i < n_own
  int n_own = 0;
  int64_t own_row = 0;
  const int start = dec::own_start(prefix, p.box_rows);
  if (L > prefix) {
    const int own = L - start;
    const int kvh = h / p.group, hg = h - kvh * p.group;
    const int sl = hg / p.hs, g = kvh * p.nc + sl;
    const int C = dec::balanced_chunk(p.ws_pref[p.num_seqs], p.num_workers, p.chunk_cap);
    const int U = p.ws_pref[b] + g * dec::ceil16(own);
    const int c0 = U / C;
    n_own = (U + own - 1) / C - c0 + 1;
    own_row = (static_cast<int64_t>(b) * p.vh + g + c0) * p.hs + hg - sl * p.hs;
  }
  // prefix: rows pre_row + i * 256 of px_o, i < n_pre
  int n_pre = 0;
  int64_t pre_row = 0;
  if (prefix > 0 && L > 0) {
    const int64_t C = *reinterpret_cast<const int64_t *>(info);
    const int first = seq[1], n = seq[2];
    const int64_t cost0 = *reinterpret_cast<const int64_t *>(seq + 4);
    const int nkt = (prefix + flash::kKeys - 1) / flash::kKeys;
    const int tiles = (n - 1) / tpt + 1, head = h / pg, pair = (b - first) / (2 * tpt);
    const int w = 2 * pair + 1 < tiles ? 2 : 1;
    const int64_t U = cost0 + static_cast<int64_t>(head) * tiles * nkt +
                      2 * static_cast<int64_t>(pair) * nkt;
    const int64_t c0 = U / C;
    n_pre = static_cast<int>((U + static_cast<int64_t>(w) * (nkt - 1)) / C - c0) + 1;
    pre_row = static_cast<int64_t>(first) * p.hq + static_cast<int64_t>(head) * n * pg +
              (b - first) * pg + h - head * pg + c0 * 256;
  }
  const int n_all = n_own + n_pre;

  float M = -INFINITY, l = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int i0 = warp; i0 < n_all; i0 += kJoinWarps * kJoinBatch) {
    float2 st[kJoinBatch];
    float ov[kJoinBatch][V];
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const int i = i0 + k * kJoinWarps;
      const bool pre = i >= n_own;
      const int64_t row = pre ? pre_row + static_cast<int64_t>(i - n_own) * 256
                              : own_row + static_cast<int64_t>(i) * p.hs;
      const float *o = (pre ? px_o : p.ws_o) + row * D + lane * V;
      st[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) ov[k][v] = 0.f;
      if (i < n_all) {
        st[k] = reinterpret_cast<const float2 *>(pre ? px_ml : p.ws_ml)[row];
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(o);
          ov[k][0] = x.x;
          ov[k][1] = x.y;
          ov[k][2] = x.z;
          ov[k][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2 *>(o);
          ov[k][0] = x.x;
          ov[k][1] = x.y;
        }
      }
    }
    float Mn = M;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) Mn = fmaxf(Mn, st[k].x);
    if (Mn == -INFINITY) continue;  // nothing visible yet
    const float cr = exp2f(M - Mn);  // 0 while M is -inf
    l *= cr;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= cr;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const float f = exp2f(st[k].x - Mn);  // 0 for padding and empty states
      l += f * st[k].y;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += f * ov[k][v];
    }
    M = Mn;
  }
  if (lane == 0) {
    s_m[warp] = M;
    s_l[warp] = l;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) s_o[warp][lane * V + v] = acc[v];
  __syncthreads();
  if (warp != 0) return;
  float Mt = -INFINITY;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) Mt = fmaxf(Mt, s_m[w]);
  float lt = 0.f, out_v[V];
#pragma unroll
  for (int v = 0; v < V; ++v) out_v[v] = 0.f;
  if (Mt != -INFINITY) {
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = exp2f(s_m[w] - Mt);  // 0 for a warp that saw nothing
      lt += f * s_l[w];
#pragma unroll
      for (int v = 0; v < V; ++v) out_v[v] += f * s_o[w][lane * V + v];
    }
  }
  // a sum that is not positive (no visible key, or only bad blocks) gives zeros
  const bool good = lt > 0.f;
  const float inv = good ? 1.f / lt : 0.f;
  typename E::T *out =
      static_cast<typename E::T *>(p.out) + b * p.out_row_stride + h * D + lane * V;
  uint32_t w[V / 2];
#pragma unroll
  for (int v = 0; v < V / 2; ++v)
    w[v] = good ? E::pack2(out_v[2 * v] * inv, out_v[2 * v + 1] * inv) : 0u;
  if constexpr (V == 4) *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t *>(out) = w[0];
}

template <class E, int D>
cudaError_t launch_all(const DecodeSharedArgs &a, const flash::Params &f,
                       const dec::DecodeParams &p, cudaStream_t stream) {
  // No group has more rows than the batch: within one query tile, the single-
  // tile build, which has more K and V in flight.
  cudaError_t e =
      p.num_seqs <= f.tpt
          ? flash::launch<E, D, flash::kPagedSingle>(f, a.tm_q, a.tm_k, a.tm_v, a.runs, stream)
          : flash::launch<E, D, flash::kPaged>(f, a.tm_q, a.tm_k, a.tm_v, a.runs, stream);
  if (e != cudaSuccess) return e;
  e = p.hs > 8 ? dec::launch_kernel<E, D, true, 0, 2, false, true>(a.decode, p, stream)
               : dec::launch_kernel<E, D, true, 0, 1, false, true>(a.decode, p, stream);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.hq;
  return launch_pdl(shared_join_kernel<E, D>, dim3(static_cast<unsigned>(rows)),
                    dim3(kJoinWarps * 32), 0, stream, p, static_cast<const float *>(a.ws_o),
                    static_cast<const float *>(a.ws_ml),
                    static_cast<const int32_t *>(a.ws_info), a.packed_heads,
                    128 / a.packed_heads);
}

}  // namespace

cudaError_t launch_decode_shared(const DecodeSharedArgs &a, cudaStream_t stream) {
  const DecodeArgs &d = a.decode;
  dec::DecodeParams p = decode_params(d);
  p.group_starts = a.group_starts;
  p.prefix_lens = a.prefix_lens;
  p.num_groups = a.num_groups;
  p.max_prefix = a.max_prefix;
  flash::Params f = {};
  f.hq = d.num_q_heads;
  f.group = d.num_q_heads / d.num_kv_heads;
  f.pg = a.packed_heads;
  f.tpt = 128 / a.packed_heads;
  f.hu = f.hq / f.pg;
  f.scale_log2 = a.scale_log2;
  f.negate = a.negate ? 1u : 0u;
  f.num_seqs = d.num_seqs;
  f.block_table = d.block_table;
  f.bt_stride = d.block_table_stride;
  f.ctx = d.context_lens;
  f.capacity = d.capacity;
  f.max_ctx = d.max_context_len;
  f.group_starts = a.group_starts;
  f.prefix_lens = a.prefix_lens;
  f.num_groups = a.num_groups;
  f.max_prefix = a.max_prefix;
  f.block_size = d.block_size;
  f.num_blocks = d.num_blocks;
  f.ws_o = a.ws_o;
  f.ws_ml = a.ws_ml;
  f.ws_info = a.ws_info;
  f.err = d.d_error;
  f.wait_ns = flash::wait_limit(d.wait_ns);
  const bool bf = d.dtype == PA_BF16;
  if (d.head_dim == 64)
    return bf ? launch_all<BF16, 64>(a, f, p, stream) : launch_all<F16, 64>(a, f, p, stream);
  return bf ? launch_all<BF16, 128>(a, f, p, stream) : launch_all<F16, 128>(a, f, p, stream);
}

}  // namespace pa
