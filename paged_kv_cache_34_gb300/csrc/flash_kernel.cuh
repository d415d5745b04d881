// flash_kernel.cuh -- the attention tile engine behind pa_attention_varlen
// (packed prompts over plain K/V rows) and pa_decode_shared's prefix pass
// (all queries of a group over the group's shared prefix in the paged cache),
// on the sm_103a tensor cores (tcgen05 + TMEM, fed by TMA).
//
// Mathematics.  For a tile of query rows and the keys j its rows may see,
//     s_ij = scale q_i . k_j,   m_i = max_j s_ij,   l_i = sum_j 2^(s_ij - m_i),
//     o_i = sum_j 2^(s_ij - m_i) v_j / l_i          (base 2, scale * log2 e)
// is formed in one pass over 128-key tiles with a running reference m_i: the
// running sum and O are rescaled only when a tile's maximum exceeds the
// reference by more than 8 (log2), which keeps every weight <= 256 and the
// result exact up to rounding.  Scores, sums and O are fp32; the weights are
// rounded to the input's 16-bit type for the tensor core and the sum takes
// the same rounded values, so o_i is an exact mean under the rounded weights.
//
// What bounds it.  Per 128 x 128 tile step at head_dim 128 the tensor core
// needs 1024 cycles (16 MMAs of 64), the softmax of one warpgroup about as
// long, one after the other: the chain S -> softmax -> P V -> next S of one
// query tile keeps the tensor core busy half the time.  So two such chains
// ("streams" A and B, one softmax warpgroup and one half of TMEM each) run
// against each other.
//
// Why this shape:
//  * A work item is a pair of query tiles that share every K/V tile loaded
//    (A the first tile, B the second), or, where a sequence or group has only
//    one tile left, that tile on both streams with the keys split between
//    them by turns (their two states are joined in the epilogue), so neither
//    stream idles.  A tile's rows are (token, head) pairs of the query heads
//    of one KV head.
//  * The streams run through the items without a stop: K/V tiles are
//    numbered through all of a CTA's items ("ring positions"), and in the
//    round of position n the MMA warp issues P V of tile n for the streams
//    that use it, then Q K^T of tile n + 1, and for a stream that skips it
//    of tile n + 2 -- the next item's first.  A causal pair's A has one tile
//    less than its B, so A starts the next item while B finishes.  (A kernel
//    whose items start and end together measured 650 TFLOP/s on 16 prompts of
//    1000 tokens, 3 us lost per item.)  Three Q buffers let the next item's
//    A query load during the current item.
//  * Items are dealt out statically, heaviest first and in alternating
//    direction (packed prompts), or as equal runs of K/V tiles (prefix), so no
//    counter in global memory is shared between launches.
#pragma once

#include <math.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace flash {

// Warpgroups: 0 / 1 softmax of stream A / B, 2 epilogue, 3 producers.
constexpr int kThreads = 512;
constexpr int kEpiWarp0 = 8, kTmaWarp = 12, kMmaWarp = 13, kFixWarp = 14, kSchedWarp = 15;
// Registers per thread after the split (setmaxnreg, per warpgroup); they must
// fit in what the CTA is launched with (checked on the host).
constexpr int kSoftmaxRegs = 152, kEpilogueRegs = 104, kProducerRegs = 104;
constexpr int kRegPoolNeeded = 128 * (2 * kSoftmaxRegs + kEpilogueRegs + kProducerRegs);
constexpr int kHalf = 128 * 128;  // 128 rows x 64 elements x 2 B
constexpr uint32_t kTmemCols = 512;        // S_A | S_B | O_A | O_B (P_t overlays S_t)
constexpr float kRescaleThreshold = 8.0f;  // log2 of the largest weight allowed
constexpr int kKeys = 128;                 // keys per K/V tile
constexpr int kItemRing = 4;
constexpr int kItemTakers = 15;  // 8 softmax warps, 4 epilogue warps, TMA, MMA, fixer

template <int D>
struct Layout {
  static constexpr int kHalves = D / 64;         // 128-byte halves per tile row
  static constexpr int kTile = kHalves * kHalf;  // one Q, K or V tile
  // Three Q buffers and two each of K and V fill the 227 KB at head_dim 128.
  static constexpr int NQ = D == 128 ? 3 : 4, NK = D == 128 ? 2 : 4, NV = D == 128 ? 2 : 4;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = NQ * kTile;
  static constexpr int kVOff = kKOff + NK * kTile;
  static constexpr int kMlOff = kVOff + NV * kTile;   // float m[2][128], l[2][128]
  static constexpr int kBarOff = kMlOff + 4 * 128 * 4;
  enum {
    kQFull = 0,
    kQEmpty = kQFull + NQ,
    kKFull = kQEmpty + NQ,
    kKEmpty = kKFull + NK,
    kVFull = kKEmpty + NK,
    kVEmpty = kVFull + NV,
    kTailIn = kVEmpty + NV,      // per V buffer: the load of an item's partial tile is out
    kVFixed = kTailIn + NV,      // ... its rows past the last key are cleared
    kSFull = kVFixed + NV,
    kPFull = kSFull + 2,
    kOFull = kPFull + 2,         // per stream and item: its last P V is done
    kOFree = kOFull + 2,         // ... the epilogue has read O and (m, l)
    kMLFull = kOFree + 2,        // ... the softmax has left (m, l)
    kItemFull = kMLFull + 2,
    kItemEmpty = kItemFull + kItemRing,
    kFin = kItemEmpty + kItemRing,
    kNumBars = kFin + 1
  };
  static constexpr int kItemOff = kBarOff + kNumBars * 8;
  static constexpr int kItemWords = 20;
  static constexpr int kMiscOff = kItemOff + kItemRing * kItemWords * 4;  // TMEM base, abort
  static constexpr int kBytes = kMiscOff + 16;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// One work item as every role sees it.
struct Item {
  int live;      // 0 ends the list
  int q0;        // first query row (token or sequence) of the sequence or group
  int ntok;      // its query rows
  int tok0;      // first of them in the item's first tile
  int head0;     // first query head of the tile's rows
  int kvh;       // KV head
  int flags;     // kSingle | kTurns | kTail
  int nkv;       // K/V tiles
  int cnt[2];    // ... used by stream A, B
  int key0;      // first key
  int kend;      // end of the keys (exclusive)
  int kv0;       // packed: K/V row of key 0; paged: the block table's row
  int ws_row;    // prefix pass: first workspace row of the item's states
  int base;      // ring position of the first K/V tile
  int qbase;     // Q buffers taken by earlier items
  int bad;       // prefix pass: a block id was outside the pool
};
constexpr int kItemFields = 17;
static_assert(sizeof(Item) == kItemFields * 4, "item words");
enum { kSingle = 1, kTurns = 2, kTail = 4 };

struct Params {
  // queries and output rows
  void *out;                // packed: output
  int64_t out_row_stride;
  int32_t hq, group, pg, tpt;  // heads, per KV head, per tile row group; rows (tokens) per tile
  int32_t hu;               // head units: hq / pg
  float scale_log2;         // |scale| * log2 e
  uint32_t negate;          // 1: the scale is negative, Q enters the product negated
  int32_t causal;
  // packed prompts
  const int32_t *cu;
  int32_t num_seqs, total, max_seqlen;
  // prefix pass
  const int32_t *block_table;
  int64_t bt_stride;
  const int32_t *ctx;
  int32_t capacity, max_ctx;
  const int32_t *group_starts, *prefix_lens;
  int32_t num_groups, max_prefix;
  int32_t block_size;
  int64_t num_blocks;
  float *ws_o, *ws_ml;
  int32_t *ws_info;
  int32_t *err;
  uint64_t wait_ns;
};

// Query tiles of a sequence or group of n rows (tokens).
__device__ __forceinline__ int tiles_of(const Params &p, int n) {
  return n > 0 ? (n - 1) / p.tpt + 1 : 0;
}

// ------------------------------------------------------ work distribution --
// Packed prompts.  Item x of the launch: pairs of query tiles, the heaviest
// first over the whole batch (a causal pair's cost is its index, whatever the
// sequence), then by sequence and head unit; batches of more than 64
// sequences go sequence by sequence, heaviest pair first, which needs no
// counting over all sequences per step.  Item k of CTA c is x = k * grid + c,
// or counted from the far end in odd rounds, so that no CTA always gets a
// round's heaviest.  Warp-collective.
struct PackedSched {
  int pairs0, pairs1;  // pairs of sequences lane, lane + 32 (up to 64 sequences)
  int level;           // ... the current pair index
  int64_t base;        // items before the level (or before chunk c0)
  int c0;              // first sequence of the current 32 (more than 64 sequences)
  int k;

  __device__ int pairs(const Params &p, int s) const {
    if (s >= p.num_seqs) return 0;
    const int a = __ldg(p.cu + s), e = __ldg(p.cu + s + 1);  // a bad pair of entries: no items
    if (a < 0 || e <= a || e > p.total || e - a > p.max_seqlen) return 0;
    return (tiles_of(p, e - a) + 1) / 2;
  }
  __device__ void init(const Params &p, int lane) {
    k = 0;
    base = 0;
    c0 = 0;
    level = 0;
    pairs0 = pairs1 = 0;
    if (p.num_seqs <= 64) {
      pairs0 = pairs(p, lane);
      pairs1 = pairs(p, lane + 32);
      level = __reduce_max_sync(0xffffffffu, max(pairs0, pairs1)) - 1;
    }
  }
  // (sequence, pair, head unit) of this CTA's next item; false at the end.
  __device__ bool next(const Params &p, int lane, int *seq, int *pair, int *head) {
    const int64_t c = (k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    const int64_t x = static_cast<int64_t>(k) * gridDim.x + c;
    ++k;
    if (p.num_seqs <= 64) {
      for (; level >= 0; --level) {
        const unsigned b0 = __ballot_sync(0xffffffffu, pairs0 > level);
        const unsigned b1 = __ballot_sync(0xffffffffu, pairs1 > level);
        const int n0 = __popc(b0), n = n0 + __popc(b1);
        if (x < base + static_cast<int64_t>(n) * p.hu) {
          const int rem = static_cast<int>(x - base);
          const int i = rem / p.hu;
          *head = rem - i * p.hu;
          *seq = i < n0 ? __fns(b0, 0, i + 1) : 32 + __fns(b1, 0, i - n0 + 1);
          *pair = level;
          return true;
        }
        base += static_cast<int64_t>(n) * p.hu;
      }
      return false;
    }
    for (; c0 < p.num_seqs; c0 += 32) {
      const int n = pairs(p, c0 + lane);
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int64_t lo = base + static_cast<int64_t>(incl - n) * p.hu;
      const int64_t hi = base + static_cast<int64_t>(incl) * p.hu;
      const unsigned hit = __ballot_sync(0xffffffffu, x >= lo && x < hi);
      if (hit) {
        const int src = __ffs(hit) - 1;
        const int64_t first = __shfl_sync(0xffffffffu, lo, src);
        const int ns = __shfl_sync(0xffffffffu, n, src);
        const int rem = static_cast<int>(x - first);
        *seq = c0 + src;
        *pair = ns - 1 - rem / p.hu;
        *head = rem % p.hu;
        return true;
      }
      base = __shfl_sync(0xffffffffu, hi, 31);
    }
    return false;
  }
};

// cu_seqlens must start at 0, never decrease, end within the packed rows,
// and no sequence may exceed max_seqlen.
__device__ inline bool check_cu(const Params &p, int lane) {
  bool bad = false;
  if (lane == 0) bad = __ldg(p.cu) != 0 || __ldg(p.cu + p.num_seqs) > p.total;
  for (int s = lane; s < p.num_seqs; s += 32) {
    const int q = __ldg(p.cu + s + 1) - __ldg(p.cu + s);
    bad |= q < 0 || q > p.max_seqlen;
  }
  return !__any_sync(0xffffffffu, bad);
}

// Prefix pass.  The unit is a (group, head unit, pair of query tiles) with
// nkt K/V tiles; a tile of a pair costs 2, of a single query tile 1, so a
// group's cost is head units x query tiles x nkt.  The units are laid end to
// end and cut into runs of C cost, one per CTA; tile i of a unit that starts
// at U (cost w per tile) belongs to run (U + w i) / C.  C >= 2 leaves no run
// inside a unit without a tile, so a unit's states are those of runs
// U / C .. (U + w (nkt - 1)) / C.  Warp-collective.
struct GroupGeom {
  int first, n, nkt, prefix;
  int64_t cost;
};
__device__ __forceinline__ GroupGeom group_geom(const Params &p, int g) {
  GroupGeom r;
  r.first = r.n = r.nkt = r.prefix = 0;
  r.cost = 0;
  if (g >= p.num_groups) return r;
  r.first = __ldg(p.group_starts + g);
  r.n = __ldg(p.group_starts + g + 1) - r.first;
  const int len = __ldg(p.prefix_lens + g);
  if (len < 0 || len > p.max_prefix || len > p.capacity) return r;  // reported by check_groups
  r.prefix = len;
  r.nkt = (len + kKeys - 1) / kKeys;
  r.cost = static_cast<int64_t>(p.hu) * tiles_of(p, r.n) * r.nkt;
  return r;
}

// group_starts must start at 0, never decrease and end at num_seqs: anything
// else makes the whole call a plain decode (no prefix is shared).  A prefix
// length that does not fit is taken as none.  Returns whether the groups are
// usable; *total is the batch's cost.
__device__ inline bool check_groups(const Params &p, int lane, bool report, int64_t *total) {
  bool bad = false, bad_len = false;
  int64_t sum = 0;
  if (lane == 0)
    bad = __ldg(p.group_starts) != 0 || __ldg(p.group_starts + p.num_groups) != p.num_seqs;
  for (int g = lane; g < p.num_groups; g += 32) {
    const int a = __ldg(p.group_starts + g), e = __ldg(p.group_starts + g + 1);
    bad |= a < 0 || e < a || e > p.num_seqs;
    const int len = __ldg(p.prefix_lens + g);
    bad_len |= len < 0 || len > p.max_prefix || len > p.capacity;
    sum += group_geom(p, g).cost;
  }
  bad = __any_sync(0xffffffffu, bad);
  bad_len = __any_sync(0xffffffffu, bad_len);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  *total = bad ? 0 : sum;
  if (report && lane == 0) {
    if (bad) raise_error(p.err, PA_DEVERR_CU_SEQLENS);
    if (bad_len) raise_error(p.err, PA_DEVERR_CONTEXT);
  }
  return !bad;
}

__host__ __device__ __forceinline__ int64_t run_cost(int64_t total, int runs) {
  const int64_t c = (total + runs - 1) / runs;
  return c < 2 ? 2 : c;
}

// What the joining kernel needs: int32 words 0-1 the run cost C (int64), then
// from word 8 on 8 words per sequence: prefix length (0: none), the group's
// first sequence, its size, 0, and its first cost position (int64).
constexpr int kInfoWords = 8;

struct PrefixSched {
  int64_t x, xend, gbase;
  int g0;

  __device__ void init(const Params &p, int64_t total) {
    const int64_t C = run_cost(total, gridDim.x);
    x = min(static_cast<int64_t>(blockIdx.x) * C, total);
    xend = min(x + C, total);
    gbase = 0;
    g0 = 0;
  }
  // The next piece: tiles [i0, i1) of a unit.
  __device__ bool next(const Params &p, int lane, GroupGeom *geom, int *head, int *pair, int *i0,
                       int *i1) {
    while (x < xend) {
      for (; g0 < p.num_groups; g0 += 32) {
        const GroupGeom r = group_geom(p, g0 + lane);
        int64_t incl = r.cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const int64_t lo = gbase + incl - r.cost, hi = gbase + incl;
        const unsigned hit = __ballot_sync(0xffffffffu, x >= lo && x < hi);
        if (hit) {
          const int src = __ffs(hit) - 1;
          GroupGeom s;
          s.first = __shfl_sync(0xffffffffu, r.first, src);
          s.n = __shfl_sync(0xffffffffu, r.n, src);
          s.nkt = __shfl_sync(0xffffffffu, r.nkt, src);
          s.prefix = __shfl_sync(0xffffffffu, r.prefix, src);
          const int64_t start = __shfl_sync(0xffffffffu, lo, src);
          const int64_t per_head = static_cast<int64_t>(tiles_of(p, s.n)) * s.nkt;
          const int64_t rem = x - start;
          const int64_t h = rem / per_head;
          const int64_t in_head = rem - h * per_head;
          const int64_t q = in_head / (2 * static_cast<int64_t>(s.nkt));
          const int w = 2 * q + 1 < tiles_of(p, s.n) ? 2 : 1;
          const int64_t U = start + h * per_head + q * 2 * s.nkt;
          const int64_t a = (x - U + w - 1) / w;
          const int64_t b = min(static_cast<int64_t>(s.nkt), (xend - U + w - 1) / w);
          x = min(xend, U + static_cast<int64_t>(w) * s.nkt);
          if (a >= b) break;  // the rest of the unit's last tile lies in the run before
          *geom = s;
          *head = static_cast<int>(h);
          *pair = static_cast<int>(q);
          *i0 = static_cast<int>(a);
          *i1 = static_cast<int>(b);
          return true;
        }
        gbase = __shfl_sync(0xffffffffu, hi, 31);
      }
      if (g0 >= p.num_groups) return false;
    }
    return false;
  }
};

__device__ __forceinline__ void store_item(volatile int *w, const Item &it) {
  const int *f = reinterpret_cast<const int *>(&it);
#pragma unroll
  for (int i = 0; i < kItemFields; ++i) w[i] = f[i];
}
__device__ __forceinline__ Item load_item(const volatile int *w) {
  Item it;
  int *f = reinterpret_cast<int *>(&it);
#pragma unroll
  for (int i = 0; i < kItemFields; ++i) f[i] = w[i];
  return it;
}

// The ring positions at which stream t uses an item's tiles: first, step.
__device__ __forceinline__ int use_first(const Item &it, int t) {
  return it.base + ((it.flags & kTurns) ? t : 0);
}
__device__ __forceinline__ int use_step(const Item &it) { return (it.flags & kTurns) ? 2 : 1; }

// -------------------------------------------------------------- the kernel --
template <class E, int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    flash_kernel(const Params p, const __grid_constant__ CUtensorMap tmq,
                 const __grid_constant__ CUtensorMap tmk,
                 const __grid_constant__ CUtensorMap tmv) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
  float *s_m = reinterpret_cast<float *>(smem + L::kMlOff), *s_l = s_m + 256;
  volatile int *items = reinterpret_cast<volatile int *>(smem + L::kItemOff);
  volatile int *misc = reinterpret_cast<volatile int *>(smem + L::kMiscOff);  // TMEM base, abort
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Nothing is static in this kernel's shared memory, so the dynamic part
  // starts on the 1024 bytes the swizzled tiles need; no tile works otherwise.
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) raise_error(p.err, PA_DEVERR_TIMEOUT);
    return;
  }

  // Lane 0 waits, the warp learns the outcome.
  auto warp_wait = [&](int b, uint32_t parity) {
    bool ok = true;
    if (lane == 0) ok = mbar_wait_bounded(bar(b), parity, p.wait_ns);
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  };
  auto slot_words = [&](int j) { return items + (j % kItemRing) * L::kItemWords; };
  // Item j of this CTA's list, without giving its ring entry back.
  auto peek_item = [&](int j, Item *it) {
    const bool ok = warp_wait(L::kItemFull + j % kItemRing, (j / kItemRing) & 1);
    if (ok) *it = load_item(slot_words(j));
    else it->live = 0;
    return ok;
  };
  auto drop_item = [&](int j) {
    __syncwarp();  // every lane has read the entry
    if (lane == 0) mbar_arrive(bar(L::kItemEmpty + j % kItemRing));
  };
  auto give_up = [&]() {
    raise_error(p.err, PA_DEVERR_TIMEOUT);
    misc[1] = 1;
  };

  griddep_wait();  // inputs (e.g. this step's cache write) come from earlier kernels
  griddep_launch_dependents();
  if (warp == 0 && lane == 0) {
    misc[1] = 0;
    for (int i = 0; i < L::kNumBars; ++i) {
      uint32_t n = 1;
      if ((i >= L::kPFull && i < L::kPFull + 2) || (i >= L::kOFree && i < L::kOFree + 2)) n = 4;
      if (i >= L::kMLFull && i < L::kMLFull + 2) n = 128;
      if (i >= L::kItemEmpty && i < L::kItemEmpty + kItemRing) n = kItemTakers;
      mbar_init(bar(i), n);
    }
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(const_cast<int *>(misc)), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = static_cast<uint32_t>(misc[0]);

  if (warp >= kTmaWarp) {
    reg_dealloc<kProducerRegs>();
    if (warp == kSchedWarp) {
      // ----------------------------------------------------- scheduler --
      bool ok = true;
      int base = 0, qbase = 0;
      PackedSched ps;
      PrefixSched xs;
      if constexpr (PAGED) {
        int64_t total;
        check_groups(p, lane, blockIdx.x == 0, &total);
        xs.init(p, total);
      } else {
        if (blockIdx.x == 0 && !check_cu(p, lane) && lane == 0)
          raise_error(p.err, PA_DEVERR_CU_SEQLENS);
        ps.init(p, lane);
      }
      for (int j = 0;; ++j) {
        Item it;
        it.live = 0;
        it.flags = 0;
        it.bad = 0;
        it.base = base;
        it.qbase = qbase;
        if constexpr (PAGED) {
          GroupGeom g;
          int head, pair, i0, i1;
          if (xs.next(p, lane, &g, &head, &pair, &i0, &i1)) {
            it.live = 1;
            it.q0 = g.first;
            it.ntok = g.n;
            it.tok0 = pair * 2 * p.tpt;
            it.head0 = head * p.pg;
            it.nkv = i1 - i0;
            it.key0 = i0 * kKeys;
            it.kend = min(g.prefix, i1 * kKeys);
            it.kv0 = g.first;
            it.ws_row = g.first * p.hq + head * g.n * p.pg + pair * 2 * p.tpt * p.pg +
                        static_cast<int>(blockIdx.x) * 256;
            const bool single = 2 * pair + 1 >= tiles_of(p, g.n);
            it.cnt[0] = it.cnt[1] = it.nkv;
            if (single) it.flags |= kSingle;
          }
        } else {
          int seq, pair, head;
          if (ps.next(p, lane, &seq, &pair, &head)) {
            it.live = 1;
            it.q0 = __ldg(p.cu + seq);
            it.ntok = __ldg(p.cu + seq + 1) - it.q0;
            it.tok0 = pair * 2 * p.tpt;
            it.head0 = head * p.pg;
            it.key0 = 0;
            it.kend = it.ntok;
            it.kv0 = it.q0;
            it.ws_row = 0;
#pragma unroll
            for (int t = 0; t < 2; ++t) {  // keys up to those of the tile's last token
              const int first = it.tok0 + t * p.tpt;
              int keys = first < it.ntok ? it.ntok : 0;
              if (p.causal && keys > 0) keys = min(keys, first + p.tpt);
              it.cnt[t] = (keys + kKeys - 1) / kKeys;
            }
            it.nkv = max(it.cnt[0], it.cnt[1]);
            if (it.cnt[1] == 0) it.flags |= kSingle;
          }
        }
        if (it.live) {
          it.kvh = it.head0 / p.group;
          if (it.key0 + it.nkv * kKeys > it.kend) it.flags |= kTail;
          if (it.flags & kSingle) {
            // one query tile: its keys by turns on both streams; a single
            // K/V tile goes to either stream, by turns of the items
            if (it.nkv > 1) {
              it.flags |= kTurns;
              it.cnt[0] = (it.nkv + 1) / 2;
              it.cnt[1] = it.nkv / 2;
            } else {
              it.cnt[0] = 1 - (j & 1);
              it.cnt[1] = j & 1;
            }
          }
          base += it.nkv;
          qbase += (it.cnt[0] > 0 ? 1 : 0) + (it.cnt[1] > 0 ? 1 : 0);
        }
        if (j >= kItemRing)
          ok = warp_wait(L::kItemEmpty + j % kItemRing, ((j / kItemRing) - 1) & 1);
        if (!ok) it.live = 0;
        if (lane == 0) {
          if (it.live) store_item(slot_words(j), it);
          else slot_words(j)[0] = 0;
          mbar_arrive(bar(L::kItemFull + j % kItemRing));
        }
        __syncwarp();
        if (!it.live) break;
      }
      if (!ok && lane == 0) give_up();
    } else if (warp == kFixWarp) {
      // --------------------------------------------------------- fixer --
      // K/V rows past an item's last key may hold anything (another
      // sequence's rows, never-written pool rows, even NaN); their weights
      // are 0, but 0 * NaN is NaN: V's are cleared once the tile has landed,
      // before the P V that reads it (K's scores are masked).
      if constexpr (PAGED) {
        if (blockIdx.x == 0) {  // what the joining kernel needs
          int64_t total;
          const bool good = check_groups(p, lane, false, &total);
          if (lane == 0) *reinterpret_cast<int64_t *>(p.ws_info) = run_cost(total, gridDim.x);
          if (!good) {
            for (int b = lane; b < p.num_seqs; b += 32)
              p.ws_info[(b + 1) * kInfoWords] = 0;
          } else {
            int64_t gbase = 0;
            for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
              const GroupGeom r = group_geom(p, g0 + lane);
              int64_t incl = r.cost;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
              }
              const int64_t lo = gbase + incl - r.cost;
              gbase = __shfl_sync(0xffffffffu, gbase + incl, 31);
              for (int i = 0; i < 32; ++i) {
                const int first = __shfl_sync(0xffffffffu, r.first, i);
                const int n = __shfl_sync(0xffffffffu, r.n, i);
                const int pre = __shfl_sync(0xffffffffu, r.prefix, i);
                const int64_t at = __shfl_sync(0xffffffffu, lo, i);
                if (g0 + i >= p.num_groups) break;
                for (int b = lane; b < n; b += 32) {
                  int32_t *w = p.ws_info + static_cast<int64_t>(first + b + 1) * kInfoWords;
                  *reinterpret_cast<int4 *>(w) = make_int4(pre, first, n, 0);
                  *reinterpret_cast<int64_t *>(w + 4) = at;
                }
              }
            }
          }
        }
      }
      // The load is waited for only once it is out (an earlier phase of the
      // buffer would pass for it otherwise), one phase of kTailIn per tail
      // in the buffer: the next one there needs this one cleared and used.
      bool ok = true;
      uint32_t par = 0;
      for (int j = 0;; ++j) {
        Item it;
        ok = peek_item(j, &it);
        drop_item(j);
        if (!ok || !it.live) break;
        if (!(it.flags & kTail)) continue;
        const int n = it.base + it.nkv - 1, slot = n % L::NV;
        ok = warp_wait(L::kTailIn + slot, (par >> slot) & 1);
        par ^= 1u << slot;
        ok = ok && mbar_wait_bounded(bar(L::kVFull + slot), (n / L::NV) & 1, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t *vt = smem + L::kVOff + slot * L::kTile;
        const int first = it.kend - it.key0 - (it.nkv - 1) * kKeys;  // 1..127
        for (int i = lane; i < (kKeys - first) * (D / 8); i += 32) {
          const int row = first + i / (D / 8), c16 = i % (D / 8);
          *reinterpret_cast<uint4 *>(vt + (c16 >> 3) * kHalf + row * 128 + (c16 & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // generic writes before the tensor core reads
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kVFixed + slot));
      }
      if (!ok && lane == 0) give_up();
    } else if (warp == kTmaWarp) {
      // ----------------------------------------------------------- TMA --
      if (lane == 0) {
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
      }
      const int bs = PAGED ? p.block_size : kKeys;
      const int nbox = kKeys / bs;  // boxes per tile, lane k loads box k
      const uint32_t q_bytes = static_cast<uint32_t>(p.tpt) * p.pg * D * 2;
      bool ok = true;
      int nk = 0, nv = 0, nq = 0;   // loads issued
      // V runs one tile behind K, also from one item to the next
      int v_pos = -1, v_row = 0, v_kvh = 0;
      bool v_valid = false, v_tail = false;
      auto load_kv = [&](bool is_v, int pos, int row, int kvh, bool valid) {
        const int slot = is_v ? pos % L::NV : pos % L::NK;
        const int use = is_v ? pos / L::NV : pos / L::NK;  // earlier uses of the buffer
        const int full = (is_v ? L::kVFull : L::kKFull) + slot;
        const int empty = (is_v ? L::kVEmpty : L::kKEmpty) + slot;
        if (use > 0 && !warp_wait(empty, (use - 1) & 1)) return false;
        const unsigned vmask = __ballot_sync(0xffffffffu, valid);
        if (lane == 0)
          mbar_arrive_expect_tx(bar(full), static_cast<uint32_t>(__popc(vmask)) * bs * D * 2);
        __syncwarp();
        if (valid) {
          const uint32_t dst =
              smem_u32(smem + (is_v ? L::kVOff : L::kKOff) + slot * L::kTile) + lane * bs * 128;
          const CUtensorMap *map = is_v ? &tmv : &tmk;
#pragma unroll
          for (int h = 0; h < L::kHalves; ++h)
            tma_load_3d(dst + h * kHalf, map, bar(full), h * 64, kvh, row);
        }
        return true;
      };
      auto load_v = [&]() {  // the pending V tile
        if (!load_kv(true, v_pos, v_row, v_kvh, v_valid)) return false;
        __syncwarp();
        if (v_tail && lane == 0) mbar_arrive(bar(L::kTailIn + v_pos % L::NV));
        ++nv;
        return true;
      };
      auto load_q = [&](const Item &it, int t, int qi) {
        const int slot = qi % L::NQ, use = qi / L::NQ;
        if (use > 0 && !warp_wait(L::kQEmpty + slot, (use - 1) & 1)) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::kQFull + slot), q_bytes);
          const int tok = it.q0 + it.tok0 + ((it.flags & kSingle) ? 0 : t * p.tpt);
          const uint32_t dst = smem_u32(smem + L::kQOff + slot * L::kTile);
#pragma unroll
          for (int h = 0; h < L::kHalves; ++h)
            tma_load_3d(dst + h * kHalf, &tmq, bar(L::kQFull + slot), h * 64, it.head0, tok);
        }
        __syncwarp();
        ++nq;
        return true;
      };
      for (int j = 0; ok; ++j) {
        Item it;
        ok = peek_item(j, &it);
        if (!ok || !it.live || misc[1]) break;
        const int t_first = it.cnt[0] > 0 ? 0 : 1;
        const bool two = it.cnt[0] > 0 && it.cnt[1] > 0;
        // PAGED: this lane's block ids, the next tile's in flight
        const int32_t *bt = PAGED ? p.block_table + it.kv0 * p.bt_stride : nullptr;
        auto load_id = [&](int i) {
          const int key = it.key0 + i * kKeys + lane * bs;
          return (lane < nbox && i < it.nkv && key < it.kend) ? __ldg(bt + key / bs) : -1;
        };
        int id = PAGED ? load_id(0) : 0;
        ok = load_q(it, t_first, it.qbase);
        for (int i = 0; ok && i < it.nkv; ++i) {
          const int id_next = PAGED ? load_id(i + 1) : 0;
          int row;
          bool valid;
          if constexpr (PAGED) {
            const bool want = lane < nbox && it.key0 + i * kKeys + lane * bs < it.kend;
            valid = want && id >= 0 && id < p.num_blocks;
            row = valid ? id * bs : 0;
            if (__any_sync(0xffffffffu, want && !valid) && lane == 0) {
              raise_error(p.err, PA_DEVERR_BLOCK_ID);
              slot_words(j)[kItemFields - 1] = 1;  // its states are left empty
            }
          } else {
            valid = lane == 0;
            row = it.kv0 + it.key0 + i * kKeys;
          }
          ok = load_kv(false, it.base + i, row, it.kvh, valid);
          if (!ok) break;
          ++nk;
          if (v_pos >= 0) ok = load_v();
          if (ok && i == 0 && two) ok = load_q(it, 1, it.qbase + 1);
          v_tail = (it.flags & kTail) && i + 1 == it.nkv;
          v_pos = it.base + i;
          v_row = row;
          v_kvh = it.kvh;
          v_valid = valid;
          id = id_next;
          if (misc[1]) ok = false;
        }
        drop_item(j);
      }
      if (ok && !misc[1] && v_pos >= 0) ok = load_v();  // the last tile's
      if (!ok && lane == 0 && !misc[1]) give_up();
      // Do not leave while copies this CTA issued may still land.
      if (lane == 0) {
        for (int n = nq - 1; n >= 0 && n >= nq - L::NQ; --n)
          mbar_wait_bounded(bar(L::kQFull + n % L::NQ), (n / L::NQ) & 1);
        for (int n = nk - 1; n >= 0 && n >= nk - L::NK; --n)
          mbar_wait_bounded(bar(L::kKFull + n % L::NK), (n / L::NK) & 1);
        for (int n = nv - 1; n >= 0 && n >= nv - L::NV; --n)
          mbar_wait_bounded(bar(L::kVFull + n % L::NV), (n / L::NV) & 1);
      }
      __syncwarp();
    } else {
      // ----------------------------------------------------------- MMA --
      // The whole warp runs this loop; MMAs and commits are issued by one
      // elected lane.  The tensor core runs one thread's MMAs in order, so
      // Q K^T may overwrite the S columns that the P V before it reads.
      // Issuing runs at the tensor core's own pace, so every cycle this warp
      // spends between two issues is one the tensor core idles: a step's
      // bookkeeping and its waits for K and V are done before the wait for P,
      // and P V and the stream's next Q K^T go out in one block after it
      // (separate waits and blocks measured 2700 cycles per tile step
      // instead of 1024: 930 TFLOP/s on two prompts of 16384).
      const uint32_t id_qk = idesc_f16(E::kBF16, 128, 128, false) | (p.negate << 13);
      const uint32_t id_pv = idesc_f16(E::kBF16, 128, D, true);
      const uint64_t q_desc0 = sdesc_sw128(smem_u32(smem) + L::kQOff, 16, 1024);
      const uint64_t k_desc0 = sdesc_sw128(smem_u32(smem) + L::kKOff, 16, 1024);
      const uint64_t v_desc0 = sdesc_sw128(smem_u32(smem) + L::kVOff, kHalf, 1024);
      bool ok = true;
      // Every lane asks once; only a wait that is not over yet goes the long way.
      auto ready = [&](int b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar(b), parity)) != 0;
      };
      auto wait = [&](int b, uint32_t parity) {
        return ready(b, parity) || warp_wait(b, parity);
      };
      constexpr int kNone = 0x7fffffff;
      // Per stream: the step whose Q K^T is issued and whose P V is to come
      // (ring position pn, or kNone), the ring position np of the Q K^T after
      // it where that is known (kNone: the item is exhausted), and the place
      // in the item list.
      struct Stream {
        int pn, np;
        bool pfirst, plast;       // the pending step is its item's first / last
        int j, end;               // item the fields belong to, its end
        int step, left, q;        // ring step, Q K^T still to issue, Q buffer
        bool first, ended;        // the next Q K^T is the item's first
        int items, psteps;        // items begun (P V), P tiles taken
      } st[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        st[t].pn = st[t].np = kNone;
        st[t].pfirst = st[t].plast = st[t].first = st[t].ended = false;
        st[t].j = -1;
        st[t].end = st[t].left = st[t].q = st[t].items = st[t].psteps = 0;
        st[t].step = 1;
      }
      // An exhausted stream walks on to the items that begin by `limit`.
      auto advance = [&](Stream &s, int t, int limit) {
        while (!s.ended && s.left == 0 && s.end <= limit) {
          Item it;
          if (!peek_item(s.j + 1, &it)) ok = false;
          if (!ok || !it.live) {
            s.ended = true;
            return;
          }
          ++s.j;
          s.end = it.base + it.nkv;
          s.left = it.cnt[t];
          s.np = s.left > 0 ? use_first(it, t) : kNone;
          s.step = use_step(it);
          s.first = true;
          s.q = it.qbase + (t == 1 && it.cnt[0] > 0 ? 1 : 0);
        }
      };
      // The elected lane's part of S_t = Q_t K_n^T.
      auto issue_qk = [&](const Stream &s, int t, int n) {
        const int qs = s.q % L::NQ;
        const uint64_t qd = q_desc0 + static_cast<uint64_t>(qs) * (L::kTile >> 4);
        const uint64_t kd = k_desc0 + static_cast<uint64_t>(n % L::NK) * (L::kTile >> 4);
        // K step k: 16 columns = 32 bytes into a 128-byte swizzled row, the
        // second 64 columns in the tile's second half
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
          umma_f16_ss(tbase + t * 128, qd + off, kd + off, id_qk, k > 0 ? 1u : 0u);
        }
        umma_commit(bar(L::kSFull + t));
        if (s.left == 1) umma_commit(bar(L::kQEmpty + qs));
      };
      // ... and the bookkeeping after it.
      auto qk_issued = [&](Stream &s, int n) {
        s.pn = n;
        s.pfirst = s.first;
        s.first = false;
        s.plast = --s.left == 0;
        s.np = s.plast ? kNone : n + s.step;
      };
      auto wait_qk = [&](const Stream &s, int n) {  // the operands of Q K_n^T
        if (s.first && !wait(L::kQFull + s.q % L::NQ, (s.q / L::NQ) & 1)) return false;
        return wait(L::kKFull + n % L::NK, (n / L::NK) & 1);
      };
      int r = -1, r_end = 0;         // the item that holds ring position n
      bool r_tail = false;
      uint32_t fix_par = 0;          // parity of each V buffer's next clearing
      for (int n = -1; ok; ++n) {
        if (n == r_end) {            // the next item (or the end of the list)
          if (r >= 0) drop_item(r);
          Item it;
          ok = peek_item(++r, &it);
          if (!ok || !it.live) {
            if (ok) drop_item(r);
            break;
          }
          r_end = it.base + it.nkv;
          r_tail = (it.flags & kTail) != 0;
        }
        if (n >= 0) {
          ok = wait(L::kVFull + n % L::NV, (n / L::NV) & 1);
          if (ok && r_tail && n + 1 == r_end) {
            ok = wait(L::kVFixed + n % L::NV, (fix_par >> (n % L::NV)) & 1);
            fix_par ^= 1u << (n % L::NV);
          }
        }
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          Stream &s = st[t];
          if (!ok || s.pn != n || n < 0) continue;
          if (s.pfirst) {  // O of the stream's previous item has been read
            if (s.items > 0) ok = wait(L::kOFree + t, (s.items - 1) & 1);
            ++s.items;
          }
          // the stream's next Q K^T goes along if its K is there already
          const bool along = s.np == n + 1 &&
                             ready(L::kKFull + (n + 1) % L::NK, ((n + 1) / L::NK) & 1);
          const uint64_t vd = v_desc0 + static_cast<uint64_t>(n % L::NV) * (L::kTile >> 4);
          const uint32_t acc0 = s.pfirst ? 0u : 1u;
          const bool last = s.plast;
          if (!ok) continue;
          ok = wait(L::kPFull + t, s.psteps & 1);
          if (!ok) continue;
          tc_fence_after();
          if (elect_one()) {
            // O_t += P_t V_n, P_t from TMEM; K step k: 16 keys = 16 rows of
            // 128 bytes of the MN-major V tile
#pragma unroll
            for (int k = 0; k < 8; ++k)
              umma_f16_ts(tbase + 256 + t * 128, tbase + t * 128 + 8 * k, vd + ((k * 2048) >> 4),
                          id_pv, k > 0 ? 1u : acc0);
            if (last) umma_commit(bar(L::kOFull + t));
            if (along) issue_qk(s, t, n + 1);
          }
          __syncwarp();
          ++s.psteps;
          s.pn = kNone;
          if (along) qk_issued(s, n + 1);
        }
        if (!ok) break;
        // Streams without a Q K^T out: tile n + 1 (its K was late, or the
        // stream does not use tile n), then n + 2.
        if (st[0].pn == kNone || st[1].pn == kNone) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (st[t].pn == kNone) advance(st[t], t, n + 2);
#pragma unroll
          for (int m = 1; m <= 2; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              Stream &s = st[t];
              if (!ok || s.pn != kNone || s.np != n + m) continue;
              ok = wait_qk(s, n + m);
              if (!ok) continue;
              tc_fence_after();
              if (elect_one()) issue_qk(s, t, n + m);
              __syncwarp();
              qk_issued(s, n + m);
            }
          if (!ok) break;
        }
        // Tile n's V has been used, and every Q K^T of tile n + 1, if there is
        // one, has been issued (a stream still behind it has no use of it).
        const bool next_tile = n + 1 < r_end || st[0].end > n + 1 || st[1].end > n + 1;
        if (elect_one()) {
          if (n >= 0) umma_commit(bar(L::kVEmpty + n % L::NV));
          if (next_tile) umma_commit(bar(L::kKEmpty + (n + 1) % L::NK));
        }
        __syncwarp();
      }
      if (!ok && lane == 0) give_up();
      // Every MMA issued above has completed once this barrier fires (the
      // full bound: TMEM is freed after it).
      if (elect_one()) umma_commit(bar(L::kFin));
      __syncwarp();
      if (lane == 0) mbar_wait_bounded(bar(L::kFin), 0);
      __syncwarp();
    }
  } else if (warp >= kEpiWarp0) {
    // ----------------------------------------------------- epilogue --
    reg_dealloc<kEpilogueRegs>();
    const int q = warp - kEpiWarp0;  // TMEM lanes 32q .. 32q+31
    const int r = q * 32 + lane;     // row of the tile
    const uint32_t o_tm = tbase + (static_cast<uint32_t>(q * 32) << 16) + 256;
    const int tl = r / p.pg, hl = r - tl * p.pg;  // the row's token and head in the tile
    int done[2] = {0, 0};            // items of each stream taken
    bool ok = true;
    for (int j = 0;; ++j) {
      Item it;
      ok = peek_item(j, &it);
      if (!ok || !it.live) {
        drop_item(j);
        break;
      }
      const bool single = (it.flags & kSingle) != 0;
      // one pass per query tile: both streams' halves of a single tile, or
      // stream t's tile t
#pragma unroll 1
      for (int u = 0; u < (single ? 1 : 2); ++u) {
        const bool use[2] = {it.cnt[0] > 0 && (single || u == 0),
                             it.cnt[1] > 0 && (single || u == 1)};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!use[t]) continue;
          ok = ok && mbar_wait_bounded(bar(L::kOFull + t), done[t] & 1, p.wait_ns);
          ok = ok && mbar_wait_bounded(bar(L::kMLFull + t), done[t] & 1, p.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          m[t] = s_m[t * 128 + r];
          l[t] = s_l[t * 128 + r];
          ++done[t];
        }
        if (!ok) break;
        tc_fence_after();
        const bool bad = PAGED && slot_words(j)[kItemFields - 1] != 0;
        // join: weights of the two halves
        const float mm = bad ? -INFINITY : fmaxf(m[0], m[1]);
        float f[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) f[t] = m[t] > -INFINITY && !bad ? fast_exp2(m[t] - mm) : 0.f;
        const float ll = f[0] * l[0] + f[1] * l[1];
        if constexpr (!PAGED) {
          const float inv = ll > 0.f ? 1.f / ll : 0.f;
          f[0] *= inv;
          f[1] *= inv;
        }
        const int tok = it.tok0 + u * p.tpt + tl;
        const bool row_ok = tl < p.tpt && tok < it.ntok;
        typename E::T *orow = nullptr;
        float *wrow = nullptr;
        if constexpr (PAGED) {
          const int64_t ws = static_cast<int64_t>(it.ws_row) + u * p.tpt * p.pg + r;
          wrow = p.ws_o + ws * D;
          if (row_ok) *reinterpret_cast<float2 *>(p.ws_ml + ws * 2) = make_float2(mm, bad ? 0.f : ll);
        } else {
          orow = static_cast<typename E::T *>(p.out) +
                 static_cast<int64_t>(it.q0 + tok) * p.out_row_stride + (it.head0 + hl) * D;
        }
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!use[t]) continue;
            uint32_t v[32];
            tmem_ld32(o_tm + t * 128 + c * 32, v);
            tmem_wait_ld();
            // a row that saw no key (f = 0) adds nothing, whatever O holds
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = f[t] != 0.f ? fmaf(__uint_as_float(v[i]), f[t], o[i]) : o[i];
          }
          if (row_ok) {
            if constexpr (PAGED) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4 *>(wrow + c * 32 + i * 4) =
                    make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4 *>(orow + c * 32 + i * 8) = make_uint4(
                    E::pack2(o[8 * i], o[8 * i + 1]), E::pack2(o[8 * i + 2], o[8 * i + 3]),
                    E::pack2(o[8 * i + 4], o[8 * i + 5]), E::pack2(o[8 * i + 6], o[8 * i + 7]));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (use[t]) mbar_arrive(bar(L::kOFree + t));
        }
      }
      drop_item(j);
      if (!ok) break;
    }
    if (!ok && lane == 0) give_up();
  } else {
    // ------------------------------------------------------- softmax --
    reg_alloc<kSoftmaxRegs>();
    const int t = warp >> 2;  // stream
    const int r = tid & 127;  // row of the tile == TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tm = tbase + lane_addr + t * 128;
    const uint32_t o_tm = tbase + lane_addr + 256 + t * 128;
    const float sl = p.scale_log2;
    const int tl = r / p.pg;
    int n = 0;      // S tiles of this stream
    int items = 0;  // items of this stream
    bool ok = true;
    for (int j = 0;; ++j) {
      Item it;
      ok = peek_item(j, &it);
      drop_item(j);
      if (!ok || !it.live) break;
      const int cnt = it.cnt[t];
      if (cnt == 0) continue;
      const int tok = it.tok0 + ((it.flags & kSingle) ? 0 : t * p.tpt) + tl;
      // the row's last visible key (rows outside the batch see what there is)
      int lim = it.kend - 1;
      if constexpr (PAGED) {
        if (tl < p.tpt && tok < it.ntok)
          lim = min(lim, checked_context_len(__ldg(p.ctx + it.q0 + tok), p.capacity, p.max_ctx,
                                             p.err, false) - 1);
      } else {
        if (p.causal) lim = min(lim, tok);
      }
      int bound = lim - it.key0 - ((it.flags & kTurns) ? t * kKeys : 0);
      const int bstep = use_step(it) * kKeys;
      float m_ref = -INFINITY, l = 0.f;
      for (int i = 0; i < cnt; ++i, ++n, bound -= bstep) {
        ok = mbar_wait_bounded(bar(L::kSFull + t), n & 1, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        // The whole S row in one TMEM round trip.
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld32(s_tm + c * 32, *reinterpret_cast<uint32_t(*)[32]>(v + c * 32));
        tmem_wait_ld();
        if (bound < kKeys - 1) {  // columns 0..bound are visible
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > bound) v[c] = __float_as_uint(-INFINITY);
        }
        float mx[8];  // raw scores (the factor is positive), as a tree
#pragma unroll
        for (int c = 0; c < 8; ++c) mx[c] = __uint_as_float(v[c]);
#pragma unroll
        for (int c = 8; c < 128; ++c) mx[c & 7] = fmaxf(mx[c & 7], __uint_as_float(v[c]));
        const float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                               fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sl;
        const bool raise = mt > m_ref + kRescaleThreshold;  // false for a fully masked row
        const float m_new = raise ? mt : m_ref;
        const float corr = raise ? fast_exp2(m_ref - m_new) : 1.f;
        // P = 2^(s - m), rounded to the input type and packed, goes to TMEM
        // over S, 16 words at a time; S(n) being complete means the P V that
        // read these columns before is done.
        const float mu = m_new == -INFINITY ? 0.f : m_new;
        const uint64_t sl2 = f2_pack(sl, sl), nmu2 = f2_pack(-mu, -mu);
        float rs[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pw[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) {  // column pair
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), sl2,
                           nmu2),
                    x0, x1);
          pw[c] = E::pack2(fast_exp2(x0), fast_exp2(x1));  // 2^-inf = 0 where masked
          E::add_halves(pw[c], rs[(c & 1) * 2], rs[(c & 1) * 2 + 1]);
          if ((c & 15) == 15)
            tmem_st16(s_tm + (c >> 4) * 16, *reinterpret_cast<uint32_t(*)[16]>(pw + c - 15));
        }
        tmem_wait_st();
        if (i > 0 && __any_sync(0xffffffffu, raise)) {
          // O holds exactly the sum so far: S(n) being complete means Q K^T
          // of this tile ran, which was issued after the P V before it.
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_tm + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
            tmem_st32(o_tm + c * 32, o);
          }
          tmem_wait_st();
        }
        l = l * corr + ((rs[0] + rs[1]) + (rs[2] + rs[3]));
        m_ref = m_new;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kPFull + t));
      }
      if (!ok) break;
      // Hand (m, l) over once the epilogue has taken the previous item's.
      if (items > 0) ok = warp_wait(L::kOFree + t, (items - 1) & 1);
      if (!ok) break;
      ++items;
      s_m[t * 128 + r] = m_ref;
      s_l[t * 128 + r] = l;
      mbar_arrive(bar(L::kMLFull + t));
    }
    if (!ok) give_up();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// The register split must fit in what the CTA is launched with, or setmaxnreg
// would wait for registers that never come: refuse to launch such a build.
template <auto Kernel>
cudaError_t check_register_pool() {
  static const cudaError_t status = [] {
    cudaFuncAttributes attr;
    const cudaError_t e = cudaFuncGetAttributes(&attr, Kernel);
    if (e != cudaSuccess) return e;
    return attr.numRegs * kThreads >= kRegPoolNeeded ? cudaSuccess : cudaErrorInvalidConfiguration;
  }();
  return status;
}

template <class E, int D, bool PAGED>
cudaError_t launch(const Params &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                   const CUtensorMap &tmv, int grid, cudaStream_t stream) {
  constexpr auto kernel = flash_kernel<E, D, PAGED>;
  cudaError_t e = allow_dynamic_smem<kernel>();
  if (e == cudaSuccess) e = check_register_pool<kernel>();
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), Layout<D>::kBytes,
                    stream, p, tmq, tmk, tmv);
}

}  // namespace flash
}  // namespace pa
