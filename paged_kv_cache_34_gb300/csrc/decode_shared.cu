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

// W warps fold one row, a (sequence, query head): the states of the own part's
// pieces, then those of the prefix's runs; warp w takes states w, w + W, ...,
// kJoinBatch at a time with every load in flight, and the warps' results are
// folded in shared memory.  Little code, it starts from a cold instruction
// cache: one loop over both parts' states took 62 us where this takes 58 on
// 64 sequences in 6 groups, and with the block search, where no group needs it,
// 4 sequences over 500 tokens take 18.7 against 15.8 (32 over 4000: 37.5 and 37.3).
constexpr int kJoinWarps = 4;
constexpr int kJoinBatch = 4;
// Four warps to a row where the own parts' workers are this many to a unit (a
// sequence and KV head), so that a row can have a batch of states for each warp
// (4 sequences of 8000 own tokens, 8/2 heads, 152 workers a unit: 19.8 us for the
// call, with one warp 36.1; 32 of up to 3000, 8/1, 38: 21.0 and 32.6; 8 of 500,
// 32/8, 19: 20.1 and 21.7); else one (32 of up to 1000, 32/8, 4.8: 37.3, with four
// 36.8; 64 of 500, 64/8, 2.4: 55.6 and 69.6; 256 of them, 0.6: 173 and 225).
constexpr int kJoinWideStates = 16;

// BLOCKS: a group may have more than two query tiles.
template <class E, int D, int W, bool BLOCKS>
__global__ void __launch_bounds__(kJoinWarps * 32)
    shared_join_kernel(const dec::DecodeParams p, const float *px_o, const float *px_ml,
                       const int32_t *info, int pg, int tpt) {
  constexpr int V = D / 32;  // output elements per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kJoinWarps / W) + warp / W, w = warp % W;
  if (row >= p.num_seqs * p.hq) return;  // (a whole row's warps, never some of them)
  const int b = row / p.hq, h = row - b * p.hq;
  const int L = checked_context_len(__ldg(p.context_lens + b), p.capacity, p.max_ctx, p.err, false);
  griddep_wait();  // both launches' states
  griddep_launch_dependents();
  const int32_t *seq_info = info + static_cast<int64_t>(b + 1) * flash::kInfoWords;
  const int4 seq = *reinterpret_cast<const int4 *>(seq_info);
  const unsigned run_c = static_cast<unsigned>(info[0]);
  const int total = p.ws_pref[p.num_seqs], pref = p.ws_pref[b];
  const int prefix = seq.x, first = seq.y, n = seq.z;
  const int ws0 = BLOCKS ? seq_info[4] : first * p.hq;  // the group's first workspace row

  const int own = L > prefix ? L - dec::own_start(prefix, p.box_rows) : 0;

  float M = -INFINITY, l = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  // The prefix's states: those of a head unit's tiles in each block of its
  // group's line, for up to two query tiles one block (part 1), else lane i
  // looking at block blk0 + i (parts 2, 3, ...).
  const int head = h / pg, pair = (b - first) / (2 * tpt);
  const int nkt = (prefix + flash::kKeys - 1) / flash::kKeys;
  int T = 0, line = 0, ks = 1, blk0 = 0, blocks = 0;
  if (prefix > 0 && L > 0) {
    T = (n - 1) / tpt + 1;
    if (BLOCKS && T > 2) {
      line = p.hq / pg * nkt;
      ks = flash::block_tiles(T, run_c, line);
      blk0 = head * nkt / ks;
      blocks = (head * nkt + nkt - 1) / ks - blk0 + 1;
    }
  }
#pragma unroll 1
  for (int part = 0; part < 2 || (BLOCKS && (part - 2) * 32 < blocks); ++part) {
    const float *o = px_o, *ml = px_ml;  // the part's states, `step` rows apart
    int count = 0, step = 256, ends = 0, at = 0;
    int64_t at0 = 0;
    if (part == 0 && own > 0) {
      const int kvh = h / p.group, hg = h - kvh * p.group;
      const int sl = hg / p.hs, g = kvh * p.nc + sl;
      const unsigned C =
          static_cast<unsigned>(dec::balanced_chunk(total, p.num_workers, p.chunk_cap));
      const unsigned U = pref + g * dec::ceil16(own), c0 = U / C;
      count = static_cast<int>((U + own - 1) / C - c0) + 1;
      at0 = (static_cast<int64_t>(b) * p.vh + g + c0) * p.hs + hg - sl * p.hs;
      o = p.ws_o;
      ml = p.ws_ml;
      step = p.hs;
    } else if (part == 1 && T > 0 && (!BLOCKS || T <= 2)) {
      const unsigned U = seq.w + T * head * nkt, c0 = U / run_c;
      count = static_cast<int>((U + T * (nkt - 1)) / run_c - c0) + 1;
      at0 = ws0 + 256 * static_cast<int64_t>(c0) + head * n * pg + (b - first) * pg + h - head * pg;
    } else if (BLOCKS && part > 1) {
      const int i = (part - 2) * 32 + lane, blk = blk0 + i;
      if (i < blocks) {
        const int t0 = blk * ks, len = min(ks, line - t0);
        const int lo = max(head * nkt - t0, 0), hi = min(head * nkt + nkt - t0, len);
        const int w = 2 * pair + 1 < T ? 2 : 1, U = seq.w + t0 * T + pair * 2 * len;
        const int c0 = (U + w * lo) / static_cast<int>(run_c);
        count = (U + w * (hi - 1)) / static_cast<int>(run_c) - c0 + 1;
        at = ws0 + flash::item_row(n, pg, tpt, nkt, blk, t0, len, pair, head) + 256 * c0 +
             (b - first - pair * 2 * tpt) * pg + h - head * pg;
      }
      ends = flash::warp_scan(count, lane);
      at -= 256 * (ends - count);  // state k of the part is at row at + 256 k of its lane
      count = __shfl_sync(0xffffffffu, ends, 31);
    }
    o += lane * V;
#pragma unroll 1
    for (int i0 = w; i0 < count; i0 += W * kJoinBatch) {
      float2 st[kJoinBatch];
      float ov[kJoinBatch][V];
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        const int at_k = i0 + k * W < count ? i0 + k * W : i0;
        int64_t i = at0 + static_cast<int64_t>(step) * at_k;
        if (BLOCKS && part > 1)
          i += __shfl_sync(0xffffffffu, at,
                           __ffs(__ballot_sync(0xffffffffu, ends > at_k)) - 1);
        st[k] = *reinterpret_cast<const float2 *>(ml + i * 2);
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(o + i * D);
          ov[k][0] = x.x;
          ov[k][1] = x.y;
          ov[k][2] = x.z;
          ov[k][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2 *>(o + i * D);
          ov[k][0] = x.x;
          ov[k][1] = x.y;
        }
        if (i0 + k * W >= count) st[k] = make_float2(-INFINITY, 0.f);
      }
      float Mn = M;
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) Mn = fmaxf(Mn, st[k].x);
      if (Mn == -INFINITY) {  // nothing visible yet: the sums are 0, or NaN of NaN scores
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k) l += st[k].y;
        continue;
      }
      const float cr = fast_exp2(M - Mn);  // 0 while M is -inf
      l *= cr;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= cr;
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        const float f = fast_exp2(st[k].x - Mn);  // 0 for padding and empty states
        l += f * st[k].y;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += f * ov[k][v];
      }
      M = Mn;
    }
  }
  if constexpr (W > 1) {
    __shared__ float s_m[W], s_l[W];
    __shared__ float s_o[W][D];
    if (lane == 0) {
      s_m[w] = M;
      s_l[w] = l;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s_o[w][lane * V + v] = acc[v];
    __syncthreads();
    if (w != 0) return;
    float Mt = -INFINITY;
#pragma unroll
    for (int k = 0; k < W; ++k) Mt = fmaxf(Mt, s_m[k]);
    l = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      // 0 for a warp that saw nothing (its sum is 0, or NaN, which stays)
      const float f = Mt == -INFINITY ? 1.f : fast_exp2(s_m[k] - Mt);
      l += f * s_l[k];
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += f * s_o[k][lane * V + v];
    }
  }
  // no visible key, or only bad blocks, give zeros; a sum that is NaN gives NaN
  const bool good = l != 0.f;
  const float inv = good ? 1.f / l : 0.f;
  typename E::T *out =
      static_cast<typename E::T *>(p.out) + b * p.out_row_stride + h * D + lane * V;
  uint32_t x[V / 2];
#pragma unroll
  for (int v = 0; v < V / 2; ++v)
    x[v] = good ? E::pack2(acc[2 * v] * inv, acc[2 * v + 1] * inv) : 0u;
  if constexpr (V == 4) *reinterpret_cast<uint2 *>(out) = make_uint2(x[0], x[1]);
  else *reinterpret_cast<uint32_t *>(out) = x[0];
}

// Up to this cost per run (of what the batch may cost at most) the prefix pass
// takes the compact softmax: it starts and ends items more than it runs (64/8
// heads, compact and unrolled: 64 sequences in 6 groups over 5000 tokens, cost 21 a
// run: 58.2 and 59.6 us; 64 over 10000, 21: 61.9 and 63.1; 64 over 20000, 41: 71.7
// and 72.4; 256 over 10000, 71: 158.0 and 156.6; 64 over 40000, 82: 96.0 and 95.3;
// 256 over 40000, 280: 299 and 287; of many groups or heads the compact one stays
// ahead by 1 %: 200 in 10 over 20000, 32/8, 132: 190.7 and 192.1).
constexpr int64_t kCompactCost = 64;

template <class E, int D>
cudaError_t launch_all(const DecodeSharedArgs &a, const flash::Params &f,
                       const dec::DecodeParams &p, cudaStream_t stream) {
  // No group has more rows than the batch: within one query tile, the single-
  // tile build, which has more K and V in flight; it waits for memory, and takes
  // the compact softmax (16 sequences over 32768 tokens, 32/8 heads: 50.5 us
  // against 53.1).
  cudaError_t e;
  if (p.num_seqs <= f.tpt)
    e = flash::launch<E, D, flash::kPagedSingle, true>(f, a.tm_q, a.tm_k, a.tm_v, a.runs, stream);
  else if (a.prefix_cost <= kCompactCost * a.runs)
    e = flash::launch<E, D, flash::kPaged, true>(f, a.tm_q, a.tm_k, a.tm_v, a.runs, stream);
  else
    e = flash::launch<E, D, flash::kPaged, false>(f, a.tm_q, a.tm_k, a.tm_v, a.runs, stream);
  if (e != cudaSuccess) return e;
  e = p.hs > 8 ? dec::launch_kernel<E, D, true, 0, 2, false, true>(a.decode, p, stream)
               : dec::launch_kernel<E, D, true, 0, 1, false, true>(a.decode, p, stream);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.hq;
  const bool wide =
      p.num_workers >= kJoinWideStates * static_cast<int64_t>(p.num_seqs) * p.vh;
  const int64_t blocks = wide ? rows : (rows + kJoinWarps - 1) / kJoinWarps;
  auto join = f.blocks ? (wide ? shared_join_kernel<E, D, kJoinWarps, true>
                               : shared_join_kernel<E, D, 1, true>)
                       : (wide ? shared_join_kernel<E, D, kJoinWarps, false>
                               : shared_join_kernel<E, D, 1, false>);
  return launch_pdl(join, dim3(static_cast<unsigned>(blocks)), dim3(kJoinWarps * 32), 0,
                    stream, p, static_cast<const float *>(a.ws_o),
                    static_cast<const float *>(a.ws_ml), static_cast<const int32_t *>(a.ws_info),
                    a.packed_heads, 128 / a.packed_heads);
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
  f.q_off = a.q_off;
  f.num_seqs = d.num_seqs;
  f.block_table = d.block_table;
  f.bt_stride = d.block_table_stride;
  f.ctx = d.context_lens;
  f.capacity = d.capacity;
  f.max_ctx = d.max_context_len;
  f.group_starts = a.group_starts;
  f.prefix_lens = a.prefix_lens;
  f.num_groups = a.num_groups;
  f.blocks = d.num_seqs > 2 * f.tpt;
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
