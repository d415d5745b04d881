// decode_fp4.cu -- paged attention for one query token per sequence over 4-bit pools.
//
// Operation (cannbot-skills "model-infer-kvcache" skill page §3.1 mapping, §3.6 decode
// data flow; App. A quantised-KV scales): for sequence b, query head h of KV head g,
//     out = sum_j softmax_j(scale q . K_j) V_j,   j < context_lens[b],
// K_j, V_j the values of position j's codes (pa_fp4.cuh).
//
// Design: HBM bound by its bytes (72 a row of 128 values), and next to that by the
// instructions that widen the codes and the issue of the products.  The units, slices and
// the balanced split of the token stream are those of decode_kernel.cuh; every warp is a
// worker with a chunk of its own.  Scores are transposed on the tensor cores, S^T[16
// tokens x 8 heads] = K[16 x D] Q^T[D x 8], then O^T[D x 8] += V^T[D x 16] P^T[16 x 8].
//  * Each warp feeds a ring of its own: a stage is 64 tokens of a piece, a bulk copy per
//    block and pool (a tile's codes and scales are one run of bytes), which the lane that
//    holds the block's id issues, as soon as the warp has read what was there; no warp
//    waits for another.
//  * Codes are widened in registers, two per instruction, and multiplied by their
//    group's scale in fp16, which is exact (2 + 4 significant bits, at least 2^-10).  The
//    head's scale goes into the scores' factor (K) and the output (V).
//  * K: lane (g, t) reads quarter t of row g: elements (D / 4) t .. are the k-steps'
//    elements 4 ks .. in any order that the query shares, and hold two groups (one at
//    D 64), so a lane needs two scales of a row.
//  * V: lane (g, t) owns elements (D / 8) g .. of O, all of one group, for the tokens
//    2t, 2t + 1 of a tile.  The fragment pairs tokens: their codes' halves are
//    interleaved before they are widened, four instructions for 16 values.
// Measured (4 sequences up to 131072 tokens, 64/8 heads of 128, 443 MB): 83 us, 5.3 TB/s of
// the 6.75 of a copy.  On the way: direct loads 188, stages of 32 tokens 97, of 64 with the
// block ids passed round 88 (64 of 4000, 64/8 heads of 64, 53 and 47 with each lane's copies
// its own).  Dropped: five CTAs an SM with 96 registers 114, stages of 32 tokens and four
// CTAs 94, the next tile's scores beside this one's sums 94.  The copies alone take 68, the
// products with their widening alone 73, the join 4.  Operands widened into tensor memory
// for products of 128 tokens 111: a tile's waits cost more than the narrow products.
#include "decode_kernel.cuh"
#include "pa_fp4.cuh"

namespace pa {
namespace fp4 {

using dec::DecodeParams;

constexpr int kWarps = kFp4Warps;
constexpr int kTokens = kFp4StageTokens;
constexpr float kLift = 7.f;  // log2 of the weight of the score that a reference was taken from

__host__ __device__ __forceinline__ int ceil32(int x) { return (x + 31) & ~31; }

// The balanced split: the units' contexts, each rounded up to 32 tokens, end to end, cut
// into chunks of a multiple of 32, at most one or two per worker (32-bit arithmetic is
// exact while total < 2^30 and workers * cap < 2^31).  So a piece starts at a multiple of
// 32 of its sequence.  Where the bound is a few stages, units are chunks instead, all of
// the bound's length (partition_size), and nothing is joined.
__device__ __forceinline__ int chunk_tokens(int total, int workers, int cap) {
  const uint32_t t = total, per = static_cast<uint32_t>(workers) * cap;
  const uint32_t n = (t > per ? (t + per - 1) / per : 1u) * workers;
  const int c = ceil32(static_cast<int>((t + n - 1) / n));
  return c > 0 ? c : 32;
}

// A piece of work: tokens start .. end - 1 of unit g (a slice of a KV head's query heads)
// of sequence b; `whole`: the unit's whole context.  Its partial state goes to the
// workspace rows (b vh + g + chunk) hs + head.
struct Piece {
  int b, g, start, end, chunk;
  bool whole;
};
struct Cursor {
  int chunk, at;  // a worker's chunk and its place in it
};
// The next piece of a worker's chunks; false at the end.
__device__ inline bool next_piece(const DecodeParams &p, const int *pref, const int *len, int C,
                                  int chunks, Cursor &cu, Piece &m) {
  const int total = pref[p.num_seqs];
  while (cu.chunk < chunks) {
    const int end = min((cu.chunk + 1) * C, total);
    if (cu.at >= end) {
      cu.chunk += p.num_workers;
      cu.at = cu.chunk * C;
      continue;
    }
    int lo = 0, hi = p.num_seqs;  // pref[lo] <= at < pref[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pref[mid] <= cu.at) lo = mid;
      else hi = mid;
    }
    const int L = len[lo], W = p.partition_size ? p.partition_size : ceil32(L);
    const int rel = cu.at - pref[lo];
    m.b = lo;
    m.g = rel / W;
    m.start = rel - m.g * W;
    const int stop = min(W, m.start + (end - cu.at));
    cu.at += stop - m.start;
    m.end = min(stop, L);
    if (m.end <= m.start) continue;  // (an empty sequence, where units are one chunk each)
    m.chunk = cu.chunk;
    m.whole = m.start == 0 && stop == W;
    return true;
  }
  return false;
}
// The first query head of unit g and the number of heads in it.
__device__ __forceinline__ int first_head(const DecodeParams &p, int g, int &n) {
  const int kvh = p.nc == 1 ? g : g / p.nc, sl = g - kvh * p.nc;
  n = min(p.hs, p.group - sl * p.hs);
  return kvh * p.group + sl * p.hs;
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }
__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(as_half2(a), b);
  return *reinterpret_cast<const uint32_t *>(&r);
}

// (not volatile, unlike the shared forms: nothing but their operands orders them)
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t transpose(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint4 lds_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// A stage's wait, bounded.  The first test does not block (a blocking one can take longer than
// a short bound), and a bound below the timer's resolution (1 us) leaves it at that.
__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (ok) return true;
  return limit_ns >= 1000 && mbar_wait_bounded(bar, parity, limit_ns);
}
// Untiled copy of `bytes` (a multiple of 16) into shared memory, both ends 16-byte aligned.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

template <class E, int D, int NG>
__global__ void __launch_bounds__(kWarps * 32, fp4_ctas_per_sm(D, NG))
    decode_fp4_kernel(const DecodeParams p, const uint8_t *__restrict__ kpool,
                      const uint8_t *__restrict__ vpool, const int stages) {
  using TL = Tile<D>;
  constexpr int KSTEPS = D / 16, KW = D / 32, VW = D / 64;
  constexpr int kHalf = kTokens / 8 * TL::kBytes, kSub = 32;  // a stage's keys, or its values
  constexpr bool QS = E::kBF16;
  // each warp's stages; barriers; [S + 1] prefix sums, [S] lengths
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * stages * 2 * kHalf;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kWarps * stages * 2 * kHalf);
  const uint32_t full = smem_u32(bars + warp * stages);
  int *s_pref = reinterpret_cast<int *>(bars + kWarps * stages);
  int *s_len = s_pref + p.num_seqs + 1;
  const int nseq = p.num_seqs;
  // Inputs come from earlier kernels; right after the step's write, only the pools'
  // rows come from the kernel just before this one.
  if (!p.after_write) griddep_wait();
  griddep_launch_dependents();
  if (lane == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(full + 8 * s, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < nseq; base += 32) {
      const int b = base + lane;
      int items = 0;
      if (b < nseq) {
        const int L = checked_context_len(__ldg(p.context_lens + b), p.capacity, p.max_ctx, p.err,
                                          blockIdx.x == 0);
        s_len[b] = L;
        items = (p.partition_size ? p.partition_size : ceil32(L)) * p.vh;
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
  const int total = s_pref[nseq];
  const int C =
      p.partition_size ? p.partition_size : chunk_tokens(total, p.num_workers, p.chunk_cap);
  const int chunks = (total + C - 1) / C;
  const int gw = blockIdx.x * kWarps + warp;
  if (blockIdx.x == 0)
    for (int i = tid; i <= nseq; i += blockDim.x) p.ws_pref[i] = s_pref[i];
  // empty sequences have no pieces: their zeros
  for (int b = gw; b < nseq; b += p.num_workers) {
    if (s_len[b] != 0) continue;
    uint4 *orow = reinterpret_cast<uint4 *>(static_cast<typename E::T *>(p.out) +
                                            b * p.out_row_stride);
    for (int e = lane; e < p.hq * D / 8; e += 32) orow[e] = make_uint4(0, 0, 0, 0);
  }
  const int bs = p.block_size, bs_shift = 31 - __clz(bs);

  // Feeding the ring.  A stage is kTokens of a piece: a run of tiles per block, keys and
  // values.  Lane q loads the id of the stage's q-th block, for the stage after as one is
  // issued, and copies that block's part.
  Cursor pc = {gw, gw * C};
  int f_cur = 0, f_end = 0, f_kvh = 0, f_id = -1;  // the stage to issue next (f_end 0: none)
  const int32_t *f_row = nullptr;
  uint32_t bad_stages = 0;
  auto look = [&]() {  // the next stage's place and its block ids
    if (f_cur >= f_end) {
      Piece m;
      f_end = 0;
      if (!next_piece(p, s_pref, s_len, C, chunks, pc, m)) return;
      f_cur = m.start;
      f_end = m.end;
      f_kvh = p.nc == 1 ? m.g : m.g / p.nc;
      f_row = p.block_table + static_cast<int64_t>(m.b) * p.bt_stride;
    }
    const int blk = (f_cur >> bs_shift) + lane;
    if (blk << bs_shift < min(f_end, f_cur + kTokens)) f_id = __ldg(f_row + blk);
  };
  const uint32_t block_bytes = static_cast<uint32_t>(p.hkv << (bs_shift - 3)) * TL::kBytes;
  auto issue = [&](int s) {
    if (f_end == 0) return;
    const uint32_t bar = full + 8 * s;
    const int stop = min(f_end, f_cur + kTokens);
    // lane q's tokens of the stage: from .. to - 1, of its q-th block
    const int base = (f_cur & -bs) + (lane << bs_shift);
    const int from = max(f_cur, base), to = min(stop, base + bs);
    const bool wrong =
        from < to && static_cast<uint32_t>(f_id) >= static_cast<uint32_t>(p.num_blocks);
    uint32_t bytes = 0;
    if (from < to && !wrong) {
      bytes = (to - from + 7) / 8 * TL::kBytes;
      const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(f_id)) * block_bytes +
                          ((f_kvh << (bs_shift - 3)) + ((from & (bs - 1)) >> 3)) * TL::kBytes;
      const uint32_t dst = ring + s * 2 * kHalf + (from - f_cur) / 8 * TL::kBytes;
      bulk_load(dst, kpool + at, bytes, bar);
      bulk_load(dst + kHalf, vpool + at, bytes, bar);
    }
    const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
    if (lane == 0) mbar_arrive_expect_tx(bar, 2 * sum);
    bad_stages = __any_sync(0xffffffffu, wrong) ? bad_stages | (1u << s) : bad_stages & ~(1u << s);
    f_cur += kTokens;
    look();
  };
  look();
  if (p.after_write) griddep_wait();
  int issued = 0;
#pragma unroll 1
  for (int s = 0; s < stages; ++s) {
    if (f_end) ++issued;
    issue(s);
  }

  Cursor cu = {gw, gw * C};
  Piece m;
  int s = 0;  // the stage to read next and its phase
  uint32_t phase = 0;
  bool alive = true;
  while (alive && next_piece(p, s_pref, s_len, C, chunks, cu, m)) {
    int nh;
    const int h0 = first_head(p, m.g, nh);
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
    float o[NG][KSTEPS][4], ref[NG][2], lst[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int mt = 0; mt < KSTEPS; ++mt) o[n][mt][0] = o[n][mt][1] = o[n][mt][2] = o[n][mt][3] = 0;
      ref[n][0] = ref[n][1] = -INFINITY;
      lst[n][0] = lst[n][1] = 0.f;
    }
#pragma unroll 1
    for (int j0 = m.start; j0 < m.end; j0 += kTokens) {
      // (one lane's wait running out ends the warp's)
      if (!__all_sync(0xffffffffu, wait_stage(full + 8 * s, phase, p.wait_ns))) {
        if (lane == 0) raise_error(p.err, PA_DEVERR_TIMEOUT);
        alive = false;
        break;
      }
      if (bad_stages >> s & 1) {
        bad = true;
        if (lane == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
      }
#pragma unroll 1
      for (int sub = 0; sub < kTokens && j0 + sub < m.end; sub += kSub) {
        const uint32_t kst = ring + s * 2 * kHalf + sub / 8 * TL::kBytes, vst = kst + kHalf;
        const int left = m.end - j0 - sub;  // tokens from here on
        float s2[NG][2][4];
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u) s2[n][u][0] = s2[n][u][1] = s2[n][u][2] = s2[n][u][3] = 0.f;
        uint32_t kw[4][KW];  // row g of each tile
        __half2 kf[4][2];    // its groups' scales
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t tile = kst + i * TL::kBytes;
          const uint32_t src = tile + g8 * TL::kRowBytes + t4 * (D / 8);
          const uint32_t ss = tile + TL::kScales + g8 * TL::kScaleBytes;
          uint32_t sb;
          if constexpr (D == 128) {
            const uint4 v = lds_v4(src);
            kw[i][0] = v.x, kw[i][1] = v.y, kw[i][2] = v.z, kw[i][3] = v.w;
            sb = lds_u16(ss + 2 * t4);
          } else {
            const uint2 v = lds_v2(src);
            kw[i][0] = v.x, kw[i][1] = v.y;
            sb = lds_u8(ss + t4);
          }
          const __half2 f = as_half2(e4m3_to_f16x2(sb));
          kf[i][0] = __low2half2(f);
          kf[i][1] = __high2half2(f);
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {  // k-steps 2w, 2w + 1
          const int hf = D == 128 ? w >> 1 : 0;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t a[4], b[4];
            widen8(kw[2 * u][w], a[0], a[1], a[2], a[3]);
            widen8(kw[2 * u + 1][w], b[0], b[1], b[2], b[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] = hmul2(a[i], kf[2 * u][hf]);
              b[i] = hmul2(b[i], kf[2 * u + 1][hf]);
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              mma(s2[n][u], a[0], b[0], a[1], b[1], qf[n][2 * w]);
              mma(s2[n][u], a[2], b[2], a[3], b[3], qf[n][2 * w + 1]);
            }
          }
        }
        uint32_t vx[4][VW], vy[4][VW];  // tokens 2t and 2t + 1 of each tile
        __half2 vf[4];                  // their scales
        auto load_v = [&](int i) {
          const uint32_t tile = vst + i * TL::kBytes;
          const uint32_t src = tile + 2 * t4 * TL::kRowBytes + g8 * (D / 16);
          const uint32_t ss = tile + TL::kScales + 2 * t4 * TL::kScaleBytes +
                              (D == 128 ? g8 : g8 >> 1);
          if constexpr (D == 128) {
            const uint2 x = lds_v2(src), y = lds_v2(src + TL::kRowBytes);
            vx[i][0] = x.x, vx[i][1] = x.y, vy[i][0] = y.x, vy[i][1] = y.y;
          } else {
            vx[i][0] = lds_u32(src);
            vy[i][0] = lds_u32(src + TL::kRowBytes);
          }
          uint32_t sx = lds_u8(ss), sy = lds_u8(ss + TL::kScaleBytes);
          vf[i] = as_half2(e4m3_to_f16x2(sx | sy << 8));
        };
        // rows past the context hold anything: their scale, and so their value, is 0 (a
        // branch of its own, rarely taken: 85.7 -> 83.7 us in the long case)
        auto tails = [&](int from, int to) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i < from || i >= to) continue;
            const int t0 = 8 * i + 2 * t4;
            uint32_t x = *reinterpret_cast<const uint32_t *>(&vf[i]);
            if (t0 >= left) x = 0;
            else if (t0 + 1 >= left) x &= 0xffffu;
            vf[i] = as_half2(x);
          }
        };
        // (their loads run under the softmax, where the registers allow it)
        if constexpr (NG == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) load_v(i);
          if (left < kSub) tails(0, 4);
        }
        // Scores of tokens j0 + 16u + g (s2[n][u][0..1], heads 8n + 2t, +1) and + 8 (2..3).
        uint32_t pb[NG][2][2];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          const float slA = QS ? slh[QS ? n : 0][0] : sl, slB = QS ? slh[QS ? n : 0][1] : sl;
          // Exponents against a reference that only follows the largest score once that
          // is more than 8 above where the reference was taken: a stage whose scores stay
          // below needs one vote and no maximum over lanes.  The reference is kLift below
          // its score, so that weights reach up to 2^15, the top of fp16's range, and keep
          // its 11 bits down to 2^-21 of the largest and something down to 2^-32 (a
          // reference at the score itself lost keys 2^25 times less likely than one before
          // them: with 2^18 of them behind it in a worker's share, 1/128 of the sum).
          float a[2][4];
          auto exponents = [&]() {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              a[u][0] = s2[n][u][0] * slA - ref[n][0];
              a[u][1] = s2[n][u][1] * slB - ref[n][1];
              a[u][2] = s2[n][u][2] * slA - ref[n][0];
              a[u][3] = s2[n][u][3] * slB - ref[n][1];
            }
            if (left < kSub) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                if (16 * u + g8 >= left) a[u][0] = a[u][1] = -INFINITY;
                if (16 * u + g8 + 8 >= left) a[u][2] = a[u][3] = -INFINITY;
              }
            }
          };
          exponents();
          float mx0 = fmaxf(fmaxf(a[0][0], a[0][2]), fmaxf(a[1][0], a[1][2]));
          float mx1 = fmaxf(fmaxf(a[0][1], a[0][3]), fmaxf(a[1][1], a[1][3]));
          if (__any_sync(0xffffffffu, fmaxf(mx0, mx1) > 8.f + kLift)) {
            // (the first stage always: the reference is -inf)
            mx0 = mx1 = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (16 * u + g8 < left) {
                mx0 = fmaxf(mx0, s2[n][u][0] * slA);
                mx1 = fmaxf(mx1, s2[n][u][1] * slB);
              }
              if (16 * u + g8 + 8 < left) {
                mx0 = fmaxf(mx0, s2[n][u][2] * slA);
                mx1 = fmaxf(mx1, s2[n][u][3] * slB);
              }
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
              mx0 = fmaxf(mx0, dec::shfl_xor(mx0, x));
              mx1 = fmaxf(mx1, dec::shfl_xor(mx1, x));
            }
            mx0 = fmaxf(mx0 - kLift, ref[n][0]);
            mx1 = fmaxf(mx1 - kLift, ref[n][1]);
            const float cr0 = mx0 == -INFINITY ? 0.f : fast_exp2(ref[n][0] - mx0);
            const float cr1 = mx1 == -INFINITY ? 0.f : fast_exp2(ref[n][1] - mx1);
            ref[n][0] = mx0;
            ref[n][1] = mx1;
            lst[n][0] *= cr0;
            lst[n][1] *= cr1;
#pragma unroll
            for (int mt = 0; mt < KSTEPS; ++mt) {
              o[n][mt][0] *= cr0;
              o[n][mt][1] *= cr1;
              o[n][mt][2] *= cr0;
              o[n][mt][3] *= cr1;
            }
            exponents();
          }
          // P is rounded to fp16 for the tensor core; the sums take the same rounded
          // values, so the output is a weighted mean of V under the rounded weights.
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t w0 = F16::pack2(fast_exp2(a[u][0]), fast_exp2(a[u][1]));
            const uint32_t w1 = F16::pack2(fast_exp2(a[u][2]), fast_exp2(a[u][3]));
            F16::add_halves(w0, lst[n][0], lst[n][1]);
            F16::add_halves(w1, lst[n][0], lst[n][1]);
            pb[n][u][0] = transpose(w0);
            pb[n][u][1] = transpose(w1);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (NG != 1) {
            load_v(2 * u);
            load_v(2 * u + 1);
            if (left < kSub) tails(2 * u, 2 * u + 2);
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            uint32_t ev[2][4], od[2][4];  // elements 2b and 2b + 1 of the lane's words, both tokens
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t x = vx[2 * u + r][w], y = vy[2 * u + r][w];
              const uint32_t e = (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
              const uint32_t d = ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
              widen8(e, ev[r][0], ev[r][1], ev[r][2], ev[r][3]);
              widen8(d, od[r][0], od[r][1], od[r][2], od[r][3]);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                ev[r][b] = hmul2(ev[r][b], vf[2 * u + r]);
                od[r][b] = hmul2(od[r][b], vf[2 * u + r]);
              }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
              for (int n = 0; n < NG; ++n)
                mma(o[n][4 * w + b], ev[0][b], od[0][b], ev[1][b], od[1][b], pb[n][u]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (f_end) ++issued;
      issue(s);
      --issued;
      if (++s == stages) {
        s = 0;
        phase ^= 1;
      }
    }
    if (!alive) break;
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
        if (m.whole) {
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
          const int64_t r = (static_cast<int64_t>(m.b) * p.vh + m.g + m.chunk) * p.hs + h;
          const float f = bad ? 0.f : vs;
          float4 *dst = reinterpret_cast<float4 *>(p.ws_o + r * D + (D / 8) * g8);
#pragma unroll
          for (int i = 0; i < KSTEPS / 2; ++i)
            dst[i] = bad ? make_float4(0.f, 0.f, 0.f, 0.f)
                         : make_float4(o[n][2 * i][hh] * f, o[n][2 * i][hh + 2] * f,
                                       o[n][2 * i + 1][hh] * f, o[n][2 * i + 1][hh + 2] * f);
          if (g8 == 0)
            reinterpret_cast<float2 *>(p.ws_ml)[r] =
                make_float2(bad ? -INFINITY : ref[n][hh], bad ? 0.f : l);
        }
      }
    }
  }
  // A wait ran out: leave once the copies in flight are in.
  for (; issued > 0; --issued) {
    mbar_wait_bounded(full + 8 * s, phase);
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
}

// Joins the pieces of each (sequence, query head), their references m_i, sums l_i and
// unnormalised outputs o_i: M = max m_i, w_i = 2^(m_i - M), out = sum w_i o_i / sum w_i l_i.
// W warps per (sequence, query head), K a CTA; a lane holds D / 32 elements, warp w of them
// takes pieces w, w + W, ..., eight at a time.  One long context among many short ones has most
// of the pieces, in rows that follow one another: with SHARE a CTA's rows are gridDim.x apart,
// and what is more than kJoinOwn pieces a warp is left to all of its warps together.
constexpr int kJoinBatch = 8;
constexpr int kJoinOwn = 16;
// Up to so many sequences each warp sums the lengths up itself while the decode still runs,
// instead of reading the sums that it leaves (128 of 400 to 700 tokens 33.0 against 33.2 us, 8
// of 1500, 32/8 heads, 10.6 and 11.1; with 256 lengths a warp 39.7 against 39.4).
constexpr int kJoinSums = 128;

// A row's state: reference, sum and a lane's V = D / 32 elements.
template <int V>
struct JoinState {
  float m = -INFINITY, l = 0.f, o[V] = {};
};
// Pieces first, first + step, ... of the n whose states start at workspace row row0.
template <int D>
__device__ __forceinline__ void join_pieces(const DecodeParams &p, int64_t row0, int n, int first,
                                            int step, int lane, JoinState<D / 32> &t) {
  constexpr int V = D / 32;
  const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
  for (int i0 = first; i0 < n; i0 += step * kJoinBatch) {
    float2 st[kJoinBatch];
    float ov[kJoinBatch][V];
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      const int i = i0 + k * step;
      const int64_t r = row0 + static_cast<int64_t>(i < n ? i : i0) * p.hs;
      st[k] = i < n ? __ldcg(ml + r) : make_float2(-INFINITY, 0.f);
      const float *src = p.ws_o + r * D + V * lane;
      if constexpr (V == 4) {
        const float4 x =
            i < n ? __ldcg(reinterpret_cast<const float4 *>(src)) : make_float4(0, 0, 0, 0);
        ov[k][0] = x.x, ov[k][1] = x.y, ov[k][2] = x.z, ov[k][3] = x.w;
      } else {
        const float2 x = i < n ? __ldcg(reinterpret_cast<const float2 *>(src)) : make_float2(0, 0);
        ov[k][0] = x.x, ov[k][1] = x.y;
      }
    }
    float m = t.m;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) m = fmaxf(m, st[k].x);
    const float cr = m == -INFINITY ? 0.f : exp2f(t.m - m);
    t.l *= cr;
#pragma unroll
    for (int v = 0; v < V; ++v) t.o[v] *= cr;
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k) {
      // a piece that saw no key has sum 0 (a NaN query's: NaN, which stays)
      const float w = st[k].x == -INFINITY ? 1.f : exp2f(st[k].x - m);
      t.l += w * st[k].y;
#pragma unroll
      for (int v = 0; v < V; ++v) t.o[v] += w * ov[k][v];
    }
    t.m = m;
  }
}

template <class E, int D, int W, int K, bool SHARE>
__global__ void __launch_bounds__(K * 32) decode_fp4_join_kernel(const DecodeParams p) {
  constexpr int V = D / 32, R = K / W;  // R rows a CTA
  __shared__ float s_m[K], s_l[K], s_o[K][D];  // (used where warps share a row)
  __shared__ int64_t s_row0[R];
  __shared__ int s_n[R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = warp / W, sub = warp % W;
  const int rows = p.num_seqs * p.hq;
  const int row = SHARE ? blockIdx.x + mine * gridDim.x : blockIdx.x * R + mine;
  if (!SHARE && row >= rows) return;
  const int b = row < rows ? row / p.hq : 0, h = row < rows ? row - b * p.hq : 0;
  const int kvh = h / p.group, hg = h - kvh * p.group, slc = hg / p.hs, g = kvh * p.nc + slc;
  // (context_lens is no output of the launch before: read, and for few sequences summed up,
  // while that runs)
  auto length = [&](int i) {
    return checked_context_len(__ldg(p.context_lens + i), p.capacity, p.max_ctx, p.err, false);
  };
  const int L = row < rows ? length(b) : 0;
  int total = 0, pref = 0;
  const bool sums = p.num_seqs <= kJoinSums;
  if (sums) {
    for (int i = lane; i < p.num_seqs; i += 32) {
      const int items = ceil32(length(i)) * p.vh;
      total += items;
      if (i < b) pref += items;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    pref = __reduce_add_sync(0xffffffffu, pref);
  }
  griddep_wait();
  griddep_launch_dependents();
  int n = 0;
  int64_t row0 = 0;
  if (!SHARE && L <= 0) return;
  if (L > 0) {
    if (!sums) {
      total = p.ws_pref[p.num_seqs];
      pref = p.ws_pref[b];
    }
    const int U = pref + g * ceil32(L);
    const int C = chunk_tokens(total, p.num_workers, p.chunk_cap);
    const int c0 = U / C;
    n = (U + ceil32(L) - 1) / C - c0 + 1;  // (one piece: written by the decode kernel itself)
    row0 = (static_cast<int64_t>(b) * p.vh + g + c0) * p.hs + hg - slc * p.hs;
  }
  auto leave = [&](const JoinState<V> &t) {
    s_m[warp] = t.m;
    s_l[warp] = t.l;
#pragma unroll
    for (int v = 0; v < V; ++v) s_o[warp][lane * V + v] = t.o[v];
  };
  auto collect = [&](int first, auto warps) {
    constexpr int count = decltype(warps)::value;
    JoinState<V> t;
#pragma unroll
    for (int w = 0; w < count; ++w) t.m = fmaxf(t.m, s_m[first + w]);
#pragma unroll
    for (int w = 0; w < count; ++w) {
      const float f = s_m[first + w] == -INFINITY ? 1.f : exp2f(s_m[first + w] - t.m);
      t.l += f * s_l[first + w];
#pragma unroll
      for (int v = 0; v < V; ++v) t.o[v] += f * s_o[first + w][lane * V + v];
    }
    return t;
  };
  auto store = [&](int to, const JoinState<V> &t) {
    const int q = to / p.hq;
    const float inv = t.l == 0.f ? 0.f : 1.f / t.l;
    typename E::T *dst = static_cast<typename E::T *>(p.out) + q * p.out_row_stride +
                         (to - q * p.hq) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<uint32_t *>(dst + v) = E::pack2(t.o[v] * inv, t.o[v + 1] * inv);
  };
  if (!SHARE && n <= 1) return;
  const bool joint = SHARE && n > kJoinOwn * W;
  if (SHARE && sub == 0 && lane == 0) {
    s_n[mine] = joint ? n : 0;
    s_row0[mine] = row0;
  }
  if (n > 1 && !joint) {
    JoinState<V> t;
    join_pieces<D>(p, row0, n, sub, W, lane, t);
    if constexpr (W > 1) {
      leave(t);
      asm volatile("bar.sync %0, %1;" ::"r"(mine + SHARE), "n"(32 * W) : "memory");
      if (sub == 0) t = collect(warp, std::integral_constant<int, W>{});
    }
    if (sub == 0) store(row, t);
  }
  if constexpr (SHARE) {
    __syncthreads();
    for (int r = 0; r < R; ++r) {
      if (s_n[r] == 0) continue;
      JoinState<V> t;
      join_pieces<D>(p, s_row0[r], s_n[r], warp, K, lane, t);
      leave(t);
      __syncthreads();
      if (warp == 0) store(blockIdx.x + r * gridDim.x, collect(0, std::integral_constant<int, K>{}));
      __syncthreads();
    }
  }
}

template <class E, int D, int NG>
cudaError_t launch(const DecodeArgs &a, const DecodeParams &p, int stages, cudaStream_t stream) {
  const int smem = fp4_decode_smem(D, stages, a.num_seqs);
  cudaError_t e = allow_dynamic_smem<decode_fp4_kernel<E, D, NG>>();
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_fp4_kernel<E, D, NG>, dim3(static_cast<unsigned>(a.grid)),
                 dim3(kWarps * 32), smem, stream, p, static_cast<const uint8_t *>(a.k_pool),
                 static_cast<const uint8_t *>(a.v_pool), stages);
  if (e != cudaSuccess) return e;
  // nothing to join: every piece is its unit's whole context, or every context is empty
  if (p.partition_size || a.max_context_len == 0) return cudaSuccess;
  // Many rows: a warp each.  Else by the pieces of a row, about workers / units (1, 2, 4 and
  // 16 warps a row, device us of the whole call; rows, pieces: 4096, 8 (32 of 2700 to 4000,
  // 128/8 heads) 48.4, 53.0, 54.9, 83.4; 2048, 4 (64 of them, 32/8) 54.8, 56.6, 57.8, 72.2;
  // 1024, 7 (32 of 50 to 2000, 32/8) 15.6, 14.4, 14.2, 21.6; 256, 8 (8 of 500 to 2000, 32/32)
  // 20.4, 19.6, 20.6, 20.7; 256, 19 (8 of 1500, 32/8) 13.0, 11.5, 10.7, 12.1; 256, 57 (4 of
  // 32000 to 131000, 64/8) 96.1, 89.2, 86.6, 85.6; 64, 228 (30000, 64/8) 46, 32, 24.4, 21.0).
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_q_heads;
  const int64_t units = static_cast<int64_t>(a.num_seqs) * p.vh;
  // The most pieces that a row can have decide whether a CTA's rows lie apart and its warps
  // share the long ones among them (one warp a row each for itself / four warps share / eight;
  // 64/8 heads: one of 131072 among 31 of 100 82 / 58 / 54, of 20000 among 40 47 / 24 / 20, of
  // 5000 among 80 26 / 19 / 20; but even lengths, 32 of 8000, 128/8, 82.5 / 82.4 / 84.7, 32 of
  // 5000, 64/8 heads of 64, 31.1 / 31.7 / 31.9, 64 of 8000, 32/8, 109 / 109 / 109; two
  // warps a row, one of 20000 among 24 26.6 / - / 19.5, 20 of 9000 49.9 / - / 48.4; four warps a
  // row keep to themselves: sharing by eight 25.4 -> 20.8 with one of 20000 among 12, but 16 of
  // 9000 41.1 -> 42.9).
  const int64_t by_length = (a.max_context_len + 31) / 32 + 1, by_worker = p.num_workers / p.vh + 2;
  const int64_t longest = by_length < by_worker ? by_length : by_worker;
  auto join = [&](auto kernel, int per_row, int warps) {
    const int per_cta = warps / per_row;
    return launch_pdl(kernel, dim3(static_cast<unsigned>((rows + per_cta - 1) / per_cta)),
                      dim3(32 * warps), 0, stream, p);
  };
  if (rows >= 2048)
    return longest <= 64    ? join(decode_fp4_join_kernel<E, D, 1, 4, false>, 1, 4)
           : longest <= 192 ? join(decode_fp4_join_kernel<E, D, 1, 4, true>, 1, 4)
                            : join(decode_fp4_join_kernel<E, D, 1, 8, true>, 1, 8);
  if (p.num_workers > 48 * units) return join(decode_fp4_join_kernel<E, D, 16, 16, false>, 16, 16);
  if (p.num_workers > 12 * units) return join(decode_fp4_join_kernel<E, D, 4, 4, false>, 4, 4);
  return longest <= 64    ? join(decode_fp4_join_kernel<E, D, 2, 4, false>, 2, 4)
         : longest <= 192 ? join(decode_fp4_join_kernel<E, D, 2, 4, true>, 2, 4)
                          : join(decode_fp4_join_kernel<E, D, 2, 8, true>, 2, 8);
}

template <class E>
cudaError_t launch_type(const DecodeArgs &a, const DecodeParams &p, int stages,
                        cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.slices.ng == 2 ? launch<E, 128, 2>(a, p, stages, stream)
                            : launch<E, 128, 1>(a, p, stages, stream);
  return a.slices.ng == 2 ? launch<E, 64, 2>(a, p, stages, stream)
                          : launch<E, 64, 1>(a, p, stages, stream);
}

}  // namespace fp4

cudaError_t launch_decode_fp4(const DecodeArgs &a, cudaStream_t stream) {
  dec::DecodeParams p = decode_params(a);
  const DecodeBalance d = fp4_balance(a.num_seqs, a.num_kv_heads * a.slices.nc, a.slices.ng,
                                      a.head_dim, a.max_context_len, a.num_sms);
  p.num_workers = d.workers;
  p.chunk_cap = kFp4ChunkCap;
  const int64_t units = static_cast<int64_t>(a.num_seqs) * p.vh;
  p.partition_size =
      fp4_whole_units(a.max_context_len, units) ? (a.max_context_len + 31) / 32 * 32 : 0;
  return a.dtype == PA_BF16 ? fp4::launch_type<BF16>(a, p, d.stages, stream)
                            : fp4::launch_type<F16>(a, p, d.stages, stream);
}

}  // namespace pa
