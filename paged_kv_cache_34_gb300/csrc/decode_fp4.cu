// decode_fp4.cu -- paged attention for one query token per sequence over 4-bit pools.
//
// Operation (cannbot-skills "model-infer-kvcache" skill page §3.1 mapping, §3.6 decode
// data flow; App. A quantised-KV scales): for sequence b, query head h of KV head g,
//     out = sum_j softmax_j(scale q . K_j) V_j,   j < context_lens[b],
// K_j, V_j the values of position j's codes (pa_fp4.cuh).
//
// Design: HBM bound by its bytes (72 a row of 128 values), and next to that by the
// instructions that widen the codes.  The units, slices and the balanced split of the
// token stream are those of decode_kernel.cuh; every warp is a worker with a chunk of
// its own.  Scores are transposed on the tensor cores, S^T[16 tokens x 8 heads] =
// K[16 x D] Q^T[D x 8], then O^T[D x 8] += V^T[D x 16] P^T[16 x 8].
//  * Codes are widened in registers, two per instruction, and multiplied by their
//    group's scale in fp16, which is exact (2 + 4 significant bits, at least 2^-10).  The
//    head's scale goes into the scores' factor (K) and the output (V).
//  * K: lane (g, t) reads quarter t of row g: elements (D / 4) t .. are the k-steps'
//    elements 4 ks .. in any order that the query shares, and hold two groups (one at
//    D 64), so a lane needs two scales of a row.
//  * V: lane (g, t) owns elements (D / 8) g .. of O, all of one group, for the tokens
//    2t, 2t + 1 of a tile.  The fragment pairs tokens: their codes' halves are
//    interleaved before they are widened, four instructions for 16 values.
#include "decode_kernel.cuh"
#include "pa_fp4.cuh"

namespace pa {
namespace fp4 {

using dec::Cursor;
using dec::DecodeParams;
using dec::Item;
using dec::Sched;

constexpr int kWarps = kFp4Warps;

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

template <class E, int D, int NG>
__global__ void __launch_bounds__(kWarps * 32, fp4_ctas_per_sm(NG))
    decode_fp4_kernel(const DecodeParams p, const uint8_t *__restrict__ kpool,
                      const uint8_t *__restrict__ vpool) {
  using TL = Tile<D>;
  constexpr int KSTEPS = D / 16, KW = D / 32, VW = D / 64;
  constexpr bool QS = E::kBF16;
  extern __shared__ int s_pref[];  // [S + 1] prefix sums, then [S] lengths
  int *s_len = s_pref + p.num_seqs + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
  const int nseq = p.num_seqs;
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < nseq; base += 32) {
      const int b = base + lane;
      int items = 0;
      if (b < nseq) {
        const int L = checked_context_len(__ldg(p.context_lens + b), p.capacity, p.max_ctx, p.err,
                                          blockIdx.x == 0);
        s_len[b] = L;
        items = dec::ceil16(L) * p.vh;
      }
      int incl = items;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (b < nseq) s_pref[b + 1] = carry + incl;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_pref[0] = 0;
  }
  __syncthreads();
  Sched sc;
  sc.pref = s_pref;
  sc.len = s_len;
  sc.S = nseq;
  sc.vh = p.vh;
  sc.hq = p.hq;
  sc.G = p.group;
  sc.nc = p.nc;
  sc.hs = p.hs;
  sc.P = 0;
  sc.NP = 0;
  sc.NW = p.num_workers;
  sc.balanced = true;
  sc.total = s_pref[nseq];
  sc.C = dec::balanced_chunk(sc.total, sc.NW, p.chunk_cap);
  sc.chunks = (sc.total + sc.C - 1) / sc.C;
  const int gw = blockIdx.x * kWarps + warp;
  if (blockIdx.x == 0)
    for (int i = tid; i <= nseq; i += blockDim.x) p.ws_pref[i] = s_pref[i];
  // empty sequences have no pieces: their zeros
  for (int b = gw; b < nseq; b += sc.NW) {
    if (s_len[b] != 0) continue;
    uint4 *orow = reinterpret_cast<uint4 *>(static_cast<typename E::T *>(p.out) +
                                            b * p.out_row_stride);
    for (int e = lane; e < p.hq * D / 8; e += 32) orow[e] = make_uint4(0, 0, 0, 0);
  }
  const int bs_shift = 31 - __clz(p.block_size);
  const int tiles_shift = bs_shift - 3;  // tiles of a (block, head)

  Cursor cu = dec::first_cursor(sc, gw);
  Item m;
  while (dec::next_piece(sc, cu, m)) {
    int nh;
    const int h0 = dec::slice_head0(sc, m.g, nh);
    const int kvh = p.nc == 1 ? m.g : m.g / p.nc;
    uint32_t qf[NG][KSTEPS][2];
    dec::load_q<E, D, true, NG>(qf, p, m.b, h0, nh, lane);
    const float ks = __ldg(p.k_scale + kvh), vs = __ldg(p.v_scale + kvh);
    bool bad = !(head_scale_ok(ks) && head_scale_ok(vs));
    if (bad && lane == 0) raise_error(p.err, PA_DEVERR_SCALE);
    const float sl = p.scale_log2 * ks;
    float slh[QS ? NG : 1][2];
    if constexpr (QS) {
      float qsc[NG];
      dec::q_bf16_to_f16<D, NG>(qf, qsc);
#pragma unroll
      for (int n = 0; n < NG; ++n) {  // heads 8n + 2t, +1 sit in head columns 2t, 2t + 1
        slh[n][0] = sl * __shfl_sync(0xffffffffu, qsc[n], 8 * t4);
        slh[n][1] = sl * __shfl_sync(0xffffffffu, qsc[n], 8 * t4 + 4);
      }
    }
    float o[NG][KSTEPS][4], mst[NG][2], lst[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int mt = 0; mt < KSTEPS; ++mt) o[n][mt][0] = o[n][mt][1] = o[n][mt][2] = o[n][mt][3] = 0;
      mst[n][0] = mst[n][1] = -INFINITY;
      lst[n][0] = lst[n][1] = 0.f;
    }
    const int32_t *row = p.block_table + static_cast<int64_t>(m.b) * p.bt_stride;
    for (int j0 = m.start; j0 < m.end; j0 += 32) {
      int64_t at[4];  // byte offsets of the four tiles, -1 past the end or in a bad block
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = j0 + 8 * q;
        at[q] = -1;
        if (j < m.end) {
          const int id = __ldg(row + (j >> bs_shift));
          if (id >= 0 && id < p.num_blocks)
            at[q] = (((static_cast<int64_t>(id) * p.hkv + kvh) << tiles_shift) +
                     ((j & (p.block_size - 1)) >> 3)) * TL::kBytes;
          else {
            bad = true;
            if (lane == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
          }
        }
      }
      float s2[NG][2][4];
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) s2[n][u][0] = s2[n][u][1] = s2[n][u][2] = s2[n][u][3] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t kw[2][KW], sc2[2][2];  // [row g of tile 2u | 2u + 1]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int w = 0; w < KW; ++w) kw[r][w] = 0;
          uint32_t sb = 0;
          if (at[2 * u + r] >= 0) {
            const uint8_t *tile = kpool + at[2 * u + r];
            const uint8_t *src = tile + g8 * TL::kRowBytes + t4 * (D / 8);
            const uint8_t *ss = tile + TL::kScales + g8 * TL::kScaleBytes;
            if constexpr (D == 128) {
              const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src));
              kw[r][0] = v.x, kw[r][1] = v.y, kw[r][2] = v.z, kw[r][3] = v.w;
              sb = __ldg(reinterpret_cast<const uint16_t *>(ss) + t4);
            } else {
              const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src));
              kw[r][0] = v.x, kw[r][1] = v.y;
              sb = __ldg(ss + t4) * 0x101u;
            }
          }
          const uint32_t s = e4m3_to_f16x2(sb);
          sc2[r][0] = __byte_perm(s, s, 0x1010);
          sc2[r][1] = __byte_perm(s, s, 0x3232);
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {  // k-steps 2w, 2w + 1
          uint32_t a[4], b[4];
          widen8(kw[0][w], a[0], a[1], a[2], a[3]);
          widen8(kw[1][w], b[0], b[1], b[2], b[3]);
          const int hf = D == 128 ? w >> 1 : 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = hmul2(a[i], sc2[0][hf]);
            b[i] = hmul2(b[i], sc2[1][hf]);
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            mma_16816<false>(s2[n][u], a[0], b[0], a[1], b[1], qf[n][2 * w][0], qf[n][2 * w][1]);
            mma_16816<false>(s2[n][u], a[2], b[2], a[3], b[3], qf[n][2 * w + 1][0],
                             qf[n][2 * w + 1][1]);
          }
        }
      }
      // Scores of tokens j0 + 16u + g (s2[n][u][0..1], heads 8n + 2t, +1) and + 8 (2..3).
      uint32_t pb[NG][2][2];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const float slA = QS ? slh[QS ? n : 0][0] : sl, slB = QS ? slh[QS ? n : 0][1] : sl;
        float sv[2][4], mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int t0 = j0 + 16 * u + g8;
          const bool in0 = t0 < m.end, in1 = t0 + 8 < m.end;
          sv[u][0] = in0 ? s2[n][u][0] * slA : -INFINITY;
          sv[u][1] = in0 ? s2[n][u][1] * slB : -INFINITY;
          sv[u][2] = in1 ? s2[n][u][2] * slA : -INFINITY;
          sv[u][3] = in1 ? s2[n][u][3] * slB : -INFINITY;
          mx0 = fmaxf(mx0, fmaxf(sv[u][0], sv[u][2]));
          mx1 = fmaxf(mx1, fmaxf(sv[u][1], sv[u][3]));
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          mx0 = fmaxf(mx0, dec::shfl_xor(mx0, x));
          mx1 = fmaxf(mx1, dec::shfl_xor(mx1, x));
        }
        const float mn0 = fmaxf(mst[n][0], mx0), mn1 = fmaxf(mst[n][1], mx1);
        const float cr0 = mn0 == -INFINITY ? 0.f : exp2f(mst[n][0] - mn0);
        const float cr1 = mn1 == -INFINITY ? 0.f : exp2f(mst[n][1] - mn1);
        mst[n][0] = mn0;
        mst[n][1] = mn1;
        // P is rounded to fp16 for the tensor core; the sums take the same rounded
        // values, so the output is a weighted mean of V under the rounded weights.
        float ls0 = 0.f, ls1 = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t w0 = F16::pack2(exp2f(sv[u][0] - mn0), exp2f(sv[u][1] - mn1));
          const uint32_t w1 = F16::pack2(exp2f(sv[u][2] - mn0), exp2f(sv[u][3] - mn1));
          ls0 += F16::lo(w0) + F16::lo(w1);
          ls1 += F16::hi(w0) + F16::hi(w1);
          pb[n][u][0] = movmatrix_trans(w0);
          pb[n][u][1] = movmatrix_trans(w1);
        }
        lst[n][0] = lst[n][0] * cr0 + ls0;
        lst[n][1] = lst[n][1] * cr1 + ls1;
#pragma unroll
        for (int mt = 0; mt < KSTEPS; ++mt) {
          o[n][mt][0] *= cr0;
          o[n][mt][1] *= cr1;
          o[n][mt][2] *= cr0;
          o[n][mt][3] *= cr1;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t vx[2][VW], vy[2][VW], sv[2];  // tokens 2t and 2t + 1 of tile 2u | 2u + 1
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int w = 0; w < VW; ++w) vx[r][w] = vy[r][w] = 0;
          uint32_t sb = 0;
          if (at[2 * u + r] >= 0) {
            const uint8_t *tile = vpool + at[2 * u + r];
            const uint8_t *src = tile + 2 * t4 * TL::kRowBytes + g8 * (D / 16);
            const uint8_t *ss = tile + TL::kScales + 2 * t4 * TL::kScaleBytes +
                                (D == 128 ? g8 : g8 >> 1);
            if constexpr (D == 128) {
              const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
              const uint2 y = __ldg(reinterpret_cast<const uint2 *>(src + TL::kRowBytes));
              vx[r][0] = x.x, vx[r][1] = x.y, vy[r][0] = y.x, vy[r][1] = y.y;
            } else {
              vx[r][0] = __ldg(reinterpret_cast<const uint32_t *>(src));
              vy[r][0] = __ldg(reinterpret_cast<const uint32_t *>(src + TL::kRowBytes));
            }
            // rows past the context hold anything: their scale, and so their value, is 0
            const int t0 = j0 + 8 * (2 * u + r) + 2 * t4;
            if (t0 < m.end) sb = __ldg(ss);
            if (t0 + 1 < m.end) sb |= static_cast<uint32_t>(__ldg(ss + TL::kScaleBytes)) << 8;
          }
          sv[r] = e4m3_to_f16x2(sb);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          uint32_t ev[2][4], od[2][4];  // elements 2b and 2b + 1 of the lane's words, both tokens
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t x = vx[r][w], y = vy[r][w];
            const uint32_t e = (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
            const uint32_t d = ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
            widen8(e, ev[r][0], ev[r][1], ev[r][2], ev[r][3]);
            widen8(d, od[r][0], od[r][1], od[r][2], od[r][3]);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              ev[r][b] = hmul2(ev[r][b], sv[r]);
              od[r][b] = hmul2(od[r][b], sv[r]);
            }
          }
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int n = 0; n < NG; ++n)
              mma_16816<false>(o[n][4 * w + b], ev[0][b], od[0][b], ev[1][b], od[1][b],
                               pb[n][u][0], pb[n][u][1]);
        }
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    // The piece's result: lane (g, t) holds elements (D / 8) g + i of head 2t in
    // o[i / 2][i % 2 ? 2 : 0] and of head 2t + 1 in o[i / 2][i % 2 ? 3 : 1].
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        lst[n][0] += dec::shfl_xor(lst[n][0], x);
        lst[n][1] += dec::shfl_xor(lst[n][1], x);
      }
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int h = 8 * n + 2 * t4 + hh;
        if (h >= nh) continue;
        const float l = lst[n][hh];
        if (m.direct) {
          // (a NaN sum, from a NaN query, stays)
          const float f = bad || l == 0.f ? 0.f : vs / l;
          uint32_t w[KSTEPS];
#pragma unroll
          for (int mt = 0; mt < KSTEPS; ++mt)
            w[mt] = f == 0.f ? 0u : E::pack2(o[n][mt][hh] * f, o[n][mt][hh + 2] * f);
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<typename E::T *>(p.out) +
                                                 m.b * p.out_row_stride + (h0 + h) * D +
                                                 (D / 8) * g8);
#pragma unroll
          for (int i = 0; i < KSTEPS / 4; ++i)
            dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
          const int64_t r = m.prow + h;
          const float f = bad ? 0.f : vs;
          float4 *dst = reinterpret_cast<float4 *>(p.ws_o + r * D + (D / 8) * g8);
#pragma unroll
          for (int i = 0; i < KSTEPS / 2; ++i)
            dst[i] = bad ? make_float4(0.f, 0.f, 0.f, 0.f)
                         : make_float4(o[n][2 * i][hh] * f, o[n][2 * i][hh + 2] * f,
                                       o[n][2 * i + 1][hh] * f, o[n][2 * i + 1][hh + 2] * f);
          if (g8 == 0)
            reinterpret_cast<float2 *>(p.ws_ml)[r] =
                make_float2(bad ? -INFINITY : mst[n][hh], bad ? 0.f : l);
        }
      }
    }
  }
}

// Joins the pieces of each (sequence, query head) by log-sum-exp:
//   M = max m_i, w_i = 2^(m_i - M), out = sum w_i o_i / sum w_i l_i.
// One CTA of four warps per (sequence, query head); a lane holds D / 32 elements, warp w
// takes pieces w, w + 4, ..., eight at a time.
constexpr int kJoinWarps = 4, kJoinBatch = 8;

template <class E, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) decode_fp4_join_kernel(const DecodeParams p) {
  constexpr int V = D / 32;
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps], s_o[kJoinWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.hq, h = blockIdx.x - b * p.hq;
  // (context_lens is no output of the launch before: read while that runs)
  const int L = checked_context_len(__ldg(p.context_lens + b), p.capacity, p.max_ctx, p.err, false);
  griddep_wait();
  griddep_launch_dependents();
  if (L <= 0) return;
  const int total = p.ws_pref[p.num_seqs], pref = p.ws_pref[b];
  const int kvh = h / p.group, hg = h - kvh * p.group, slc = hg / p.hs;
  const int g = kvh * p.nc + slc;
  const int C = dec::balanced_chunk(total, p.num_workers, p.chunk_cap);
  const int U = pref + g * dec::ceil16(L);
  const int c0 = U / C, n = (U + L - 1) / C - c0 + 1;
  if (n <= 1) return;  // written by the decode kernel itself
  const int64_t row0 = (static_cast<int64_t>(b) * p.vh + g + c0) * p.hs + hg - slc * p.hs;
  const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
  float M = -INFINITY, l = 0.f, acc[V] = {};
  for (int i0 = warp; i0 < n; i0 += kJoinWarps * kJoinBatch) {
    float2 st[kJoinBatch];
    float ov[kJoinBatch][V];
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const int i = i0 + k * kJoinWarps;
      const int64_t r = row0 + static_cast<int64_t>(i < n ? i : i0) * p.hs;
      st[k] = i < n ? ml[r] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) ov[k][v] = i < n ? p.ws_o[r * D + V * lane + v] : 0.f;
    }
    float Mn = M;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) Mn = fmaxf(Mn, st[k].x);
    const float cr = Mn == -INFINITY ? 0.f : exp2f(M - Mn);
    l *= cr;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= cr;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      // a piece that saw no key has sum 0 (a NaN query's: NaN, which stays)
      const float w = st[k].x == -INFINITY ? 1.f : exp2f(st[k].x - Mn);
      l += w * st[k].y;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += w * ov[k][v];
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
  float Mt = -INFINITY, lt = 0.f, out[V] = {};
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) Mt = fmaxf(Mt, s_m[w]);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float f = s_m[w] == -INFINITY ? 1.f : exp2f(s_m[w] - Mt);
    lt += f * s_l[w];
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] += f * s_o[w][lane * V + v];
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  typename E::T *dst =
      static_cast<typename E::T *>(p.out) + b * p.out_row_stride + h * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2)
    *reinterpret_cast<uint32_t *>(dst + v) = E::pack2(out[v] * inv, out[v + 1] * inv);
}

template <class E, int D, int NG>
cudaError_t launch(const DecodeArgs &a, const DecodeParams &p, cudaStream_t stream) {
  const int smem = fp4_decode_smem(a.num_seqs);
  cudaError_t e = allow_dynamic_smem<decode_fp4_kernel<E, D, NG>>();
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_fp4_kernel<E, D, NG>, dim3(static_cast<unsigned>(a.grid)),
                 dim3(kWarps * 32), smem, stream, p, static_cast<const uint8_t *>(a.k_pool),
                 static_cast<const uint8_t *>(a.v_pool));
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_fp4_join_kernel<E, D>,
                    dim3(static_cast<unsigned>(static_cast<int64_t>(a.num_seqs) * a.num_q_heads)),
                    dim3(kJoinWarps * 32), 0, stream, p);
}

template <class E>
cudaError_t launch_type(const DecodeArgs &a, const DecodeParams &p, cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.slices.ng == 2 ? launch<E, 128, 2>(a, p, stream) : launch<E, 128, 1>(a, p, stream);
  return a.slices.ng == 2 ? launch<E, 64, 2>(a, p, stream) : launch<E, 64, 1>(a, p, stream);
}

}  // namespace fp4

cudaError_t launch_decode_fp4(const DecodeArgs &a, cudaStream_t stream) {
  dec::DecodeParams p = decode_params(a);
  const DecodeBalance d = fp4_balance(a.num_seqs, a.num_kv_heads * a.slices.nc, a.slices.ng,
                                      a.max_context_len, a.num_sms);
  p.num_workers = d.workers;
  p.chunk_cap = kFp4ChunkCap;
  return a.dtype == PA_BF16 ? fp4::launch_type<BF16>(a, p, stream)
                            : fp4::launch_type<F16>(a, p, stream);
}

}  // namespace pa
