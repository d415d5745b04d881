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
// rounded to the input's 16-bit type for the tensor core, and the sum takes
// them in fp32 before that.  (Summing the rounded values, which makes o_i an
// exact mean under them, costs one or two instructions a weight instead of a half:
// 16384 tokens 32/8 heads 1390 us against 1285, 16 x 1000 32/32 146 against 144.  On
// values far from 0, with a mean of 4, the error is by 0.5 % smaller then as a root
// mean square, by 20 % at its largest; on centred ones by 1 % and 0.)
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
//    one tile left or a launch has few, one tile on both streams with the keys
//    split between them by turns (their two states are joined in the epilogue),
//    so neither stream idles.  A tile's rows are (token, head) pairs of the query heads
//    of one KV head.
//  * The streams run through the items without a stop: K/V tiles are
//    numbered through all of a CTA's items ("ring positions") and each stream,
//    with an MMA warp of its own, goes on to the next tile it uses whatever
//    item that is in.  A causal pair's A has one tile less than its B, so A
//    starts the next item while B finishes; three Q buffers let the next
//    item's first query tile load during the current item.
//  * Items are handed out by the hardware's launch queue (packed prompts) or
//    as equal runs of K/V tiles (prefix), so no counter in global memory is
//    shared between launches.
//
// Measured (causal, head_dim 128, rates of the visible pairs; a 16-bit library
// product reaches 1945 TFLOP/s): 16384 tokens 32/8 heads 1650 to 1790 TFLOP/s (by
// the card's power), 4 x 4096 32/8 1540, 24 prompts of up to 2700 tokens 40/8 1170,
// 16 of up to 2000 32/32 1000, 16 x 1000 32/32 910; not causal 1730, 1670, -, 1240,
// 1210; head_dim 64, 8192 tokens 1020, where the softmax bounds it.  Prefix pass: 256
// sequences x 64/8 heads over 32768 tokens 1640 (170 us).  In the long run a
// step's length is one stream's chain (softmax and its own MMAs, 2400 cycles,
// 2048 of them with the tensor core busy); around items, where both streams'
// softmaxes run at once, it is the fetching of their instructions and the pipes
// they share (ncu: 1.0 warps an issue wait for an instruction on the 24 prompts,
// with the compact softmax 0.4 on the 16 of up to 2000; 0.6 on 2 x 8192).
#pragma once

#include <math.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace flash {

// Warpgroups: 0 / 1 softmax of stream A / B, 2 epilogue, 3 producers.
constexpr int kThreads = 512;
constexpr int kEpiWarp0 = 8, kTmaWarp = 12, kMmaWarp0 = 13, kSchedWarp = 15;  // MMA: 13 A, 14 B
// Registers per thread after the split (setmaxnreg, per warpgroup); they must
// fit in what the CTA is launched with (checked on the host).
constexpr int kSoftmaxRegs = 168, kEpilogueRegs = 88, kProducerRegs = 88;
constexpr int kRegPoolNeeded = 128 * (2 * kSoftmaxRegs + kEpilogueRegs + kProducerRegs);
constexpr int kHalf = 128 * 128;  // 128 rows x 64 elements x 2 B
constexpr uint32_t kTmemCols = 512;        // S_A | S_B | O_A | O_B (P_t overlays S_t)
constexpr float kRescaleThreshold = 8.0f;  // log2 of the largest weight allowed
constexpr int kKeys = 128;                 // keys per K/V tile
constexpr int kItemRing = 4;
constexpr int kItemTakers = 15;  // 8 softmax warps, 4 epilogue warps, TMA, 2 MMA

// What a launch is built for.
enum Mode {
  kPacked = 0,       // packed prompts over plain rows
  kPaged = 1,        // prefix pass
  kPagedSingle = 2,  // ... where no group has more rows than one query tile
  kPackedSingle = 3  // packed prompts, one query tile per item
};
template <int MODE>
constexpr bool kIsPaged = MODE == kPaged || MODE == kPagedSingle;
template <int MODE>
constexpr bool kIsSingle = MODE == kPagedSingle || MODE == kPackedSingle;

template <int D, int MODE>
struct Layout {
  static constexpr int kHalves = D / 64;         // 128-byte halves per tile row
  static constexpr int kTile = kHalves * kHalf;  // one Q, K or V tile
  // Buffers of 32 KB (16 at head_dim 64), in what the 227 KB hold.  Packed
  // prompts run through many items: a third Q buffer lets the next one's first
  // query tile load early.  The prefix pass, and a launch of single tiles, have
  // few items and wait for K and V: these get the room (8 sequences behind 16384
  // tokens, 32/32 heads: 67 us against 82 with the pairs' split; one prompt of
  // 2000 tokens 8/2: 21.5 against 30.0).
  static constexpr int kUnit = D == 128 ? 1 : 2;
  // Q buffers of stream A and B; a single-tile launch's streams share theirs.
  static constexpr int kQA = (MODE == kPacked ? 2 : 1) * kUnit;
  static constexpr int kQB = (kIsSingle<MODE> ? 0 : 1) * kUnit;
  static constexpr int NQ = kQA + kQB;
  static constexpr int NK = (kIsSingle<MODE> ? 3 : 2) * kUnit;
  static constexpr int NV = (MODE == kPacked ? 2 : 3) * kUnit;
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
    kBegun = kItemEmpty + kItemRing,  // the TMA warp has begun an item
    kNext = kBegun + 1,               // the launch's next item has come
    kFin = kNext + 1,                 // per stream: every MMA issued is done
    kNumBars = kFin + 2
  };
  static constexpr int kNextOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;  // the answer, 16 B
  // Buffer and use count of a stream's query tile number q (counted by stream,
  // or, where they share, by item).
  static __device__ __forceinline__ int q_slot(int t, int q) {
    return t == 0 || kQB == 0 ? q % kQA : kQA + q % (kQB > 0 ? kQB : 1);
  }
  static __device__ __forceinline__ int q_use(int t, int q) {
    return t == 0 || kQB == 0 ? q / kQA : q / (kQB > 0 ? kQB : 1);
  }
  static constexpr int kItemOff = kNextOff + 16;
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
  int flags;     // kSingle | kTurns | kTail | kTailOdd (parity of the tail in its V buffer)
  int nkv;       // K/V tiles
  int cnt[2];    // ... used by stream A, B
  int key0;      // first key
  int kend;      // end of the keys (exclusive)
  int kv0;       // packed: K/V row of key 0; paged: the block table's row
  int ws_row;    // prefix pass: first workspace row of the item's states
  int base;      // ring position of the first K/V tile
  int bad;       // prefix pass: a block id was outside the pool
};
constexpr int kItemFields = 16;
static_assert(sizeof(Item) == kItemFields * 4, "item words");
enum { kSingle = 1, kTurns = 2, kTail = 4, kTailOdd = 8 };

struct Params {
  // queries and output rows
  void *out;                // packed: output
  int64_t out_row_stride;
  int32_t hq, group, pg, tpt;  // heads, per KV head, per tile row group; rows (tokens) per tile
  int32_t hu;               // head units: hq / pg
  bool out_wide;            // packed: output rows are 32-byte aligned
  int32_t pair_log2;        // packed: log2 of an item's query tiles, 1 or 0
  float scale_log2;         // |scale| * log2 e, > 0
  int32_t q_off;            // 0; at scale 0 the query's rows: its tiles are read as zeros
  uint32_t negate;          // 1: the scale is negative, Q enters the product negated
  int32_t causal;
  // packed prompts
  const int32_t *cu;
  int32_t num_seqs, total, max_seqlen;
  int32_t kv_bytes;         // of one token's K and V, one KV head
  // prefix pass
  const int32_t *block_table;
  int64_t bt_stride;
  const int32_t *ctx;
  int32_t capacity, max_ctx;
  const int32_t *group_starts, *prefix_lens;
  int32_t num_groups, max_prefix;
  bool blocks;              // a group may have more than two query tiles
  int32_t block_size;
  int64_t num_blocks;
  float *ws_o, *ws_ml;
  int32_t *ws_info;
  int32_t *err;
  uint32_t wait_ns;
};

// The full bound, for what must have ended before a CTA leaves, and a launch's.
constexpr uint32_t kFullWait = static_cast<uint32_t>(kWaitLimitNs);
inline uint32_t wait_limit(uint64_t ns) {
  return static_cast<uint32_t>(ns < kWaitLimitNs ? ns : kWaitLimitNs);
}

// Query tiles of a sequence or group of n rows (tokens).
__device__ __forceinline__ int tiles_of(const Params &p, int n) {
  return n > 0 ? (n - 1) / p.tpt + 1 : 0;
}

// A pipeline wait, bounded in time.  In few instructions (a 32-bit timer; the
// bound is at most 2 s): this kernel has some 25 waits, its roles run their
// parts of it side by side, and what does not fit in the SM's instruction
// cache is paid for at every item.
__device__ __forceinline__ uint32_t timer_lo_ns() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, uint32_t limit_ns) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint32_t start = timer_lo_ns();
    do {
      ok = mbar_try_wait(bar, parity);
    } while (!ok && timer_lo_ns() - start <= limit_ns);
  }
  return ok;
}

// Whether the phase is over, without waiting (try_wait suspends the thread for
// microseconds where it is not).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// ------------------------------------------------------ work distribution --
// Packed prompts.  The launch has (at least) one CTA per item; the ones that
// run take over the items of those still waiting (cluster launch control), so
// items are handed out in order as CTAs become free, without a counter in
// memory.  The order keeps K and V in L2 and the last items light: sequences
// by falling length (up to 64 of them, else as they come), within one the
// head units in blocks whose K and V stay in L2, within a block the tile pairs
// from the last, heaviest one down, then the block's head units.  (All
// sequences' heaviest pairs first would read K and V from memory again for
// each pair.)
constexpr int64_t kBlockBytes = 40 << 20;  // K and V of a head block: a third of L2

// Warp-collective; each call goes on from the one before while x grows.
struct PackedSched {
  unsigned key0, key1;  // sequences lane, lane + 32: pairs << 6 | (63 - index), 0 once passed
  int seq, n;           // the current sequence and its pairs
  int64_t base;         // items before it

  // Query tile pairs of sequence s; none where its two entries are bad.
  static __device__ int pairs_of(const Params &p, int s) {
    if (s >= p.num_seqs) return 0;
    const int a = __ldg(p.cu + s), e = __ldg(p.cu + s + 1);
    if (a < 0 || e <= a || e > p.total || e - a > p.max_seqlen) return 0;
    return (tiles_of(p, e - a) + p.pair_log2) >> p.pair_log2;
  }
  // The next sequence by length (up to 64).
  __device__ void longest(int lane) {
    const unsigned top = __reduce_max_sync(0xffffffffu, max(key0, key1));
    n = static_cast<int>(top >> 6);
    seq = 63 - static_cast<int>(top & 63u);
    if (key0 == top) key0 = 0;
    if (key1 == top) key1 = 0;
  }
  __device__ void init(const Params &p, int lane) {
    base = 0;
    seq = 0;  // more than 64 sequences: first of the current 32
    if (p.num_seqs <= 64) {
      const int n0 = pairs_of(p, lane), n1 = pairs_of(p, lane + 32);
      key0 = n0 ? static_cast<unsigned>(n0) << 6 | (63 - lane) : 0u;
      key1 = n1 ? static_cast<unsigned>(n1) << 6 | (31 - lane) : 0u;
      longest(lane);
    }
  }
  // (sequence, pair, head unit) of item x; false beyond the last.
  __device__ bool find(const Params &p, int64_t x, int lane, int *seq_out, int *pair, int *head) {
    int pairs, rem;
    if (p.num_seqs <= 64) {
      while (n > 0 && x >= base + static_cast<int64_t>(n) * p.hu) {
        base += static_cast<int64_t>(n) * p.hu;
        longest(lane);
      }
      if (n == 0) return false;
      *seq_out = seq;
      pairs = n;
      rem = static_cast<int>(x - base);
    } else {
      for (;; seq += 32) {
        if (seq >= p.num_seqs) return false;
        const int m = pairs_of(p, seq + lane);
        int incl = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const int64_t lo = base + static_cast<int64_t>(incl - m) * p.hu;
        const int64_t hi = base + static_cast<int64_t>(incl) * p.hu;
        const unsigned hit = __ballot_sync(0xffffffffu, x >= lo && x < hi);
        if (hit) {
          const int src = __ffs(hit) - 1;
          *seq_out = seq + src;
          pairs = __shfl_sync(0xffffffffu, m, src);
          rem = static_cast<int>(x - __shfl_sync(0xffffffffu, lo, src));
          break;
        }
        base = __shfl_sync(0xffffffffu, hi, 31);
      }
    }
    // head units per block: pairs * 2 * tpt tokens of K and V per KV head
    const int64_t kv = (static_cast<int64_t>(pairs) << p.pair_log2) * p.tpt * p.kv_bytes;
    const int per_kv = p.group / p.pg;
    const int hb = static_cast<int>(
        min(static_cast<int64_t>(p.hu), max(kBlockBytes / kv, static_cast<int64_t>(1)) * per_kv));
    const int blk = rem / (pairs * hb);
    rem -= blk * pairs * hb;
    const int hn = min(hb, p.hu - blk * hb);
    const int q = rem / hn;
    *pair = pairs - 1 - q;
    *head = blk * hb + rem - q * hn;
    return true;
  }
};

// The launch's next item for this CTA: a request that the hardware answers
// with the index of a waiting CTA, which it then does not start, or with none.
__device__ __forceinline__ void clc_request(uint32_t dst, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(dst),
      "r"(bar)
      : "memory");
}
// The answer's CTA index, or -1.
__device__ __forceinline__ int clc_answer(uint32_t src) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(src)
      : "memory");
  return got ? static_cast<int>(x) : -1;
}

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

// Prefix pass.  A group of n rows with T query tiles per head unit and nkt K/V
// tiles has a line of (head units x nkt) K/V tiles, each needed by its pairs of
// query tiles; a tile costs a pair 2, a single query tile 1.  The line is cut
// into blocks; within a block the pairs follow one another, each with the
// block's tiles ("row").  All rows are laid end to end and cut into runs of C
// cost, one per CTA; tile i of a row that starts at U (cost w per tile) belongs
// to run (U + w i) / C.  C >= 2 leaves no run inside a row without a tile, so
// the runs of its tiles i .. k are (U + w i) / C .. (U + w k) / C.
//
// A block is as long as a run of a pair: the CTAs that work beside each other
// are then a block's pairs over the same K and V, which come from memory once
// (256 sequences over 32768 tokens, 64/8 heads, 8 pairs: 142 MB read where whole
// lines one after the other read 850, the pass 170 us against 198).  Two query
// tiles or less are one pair, whose line is one block.  Of full blocks a run holds
// no two rows of one pair (three tiles' other row is a run long with blocks of C);
// where a line's last block is shorter, a run may.
//
// A work item is a row's tiles of one head unit in one run; its states start at
// a workspace row that grows along the line by at least its rows (item_row, which
// counts every block) plus 256 per run, so no two items share one, nor do a
// pair's rows of two blocks in one run.  Warp-collective.
struct GroupGeom {
  int first, n, nkt, prefix, cost;
};
// K/V tiles per block of a line for T query tiles and runs of C.
__device__ __forceinline__ int block_tiles(int T, int C, int line) {
  return T <= 2 ? line : min(line, T == 3 ? C : (C + 1) >> 1);
}
// Workspace rows of a group (its runs' 256 aside): rows of a head unit x
// (blocks + head units), as item_row counts.
__device__ __forceinline__ int group_rows(const Params &p, const GroupGeom &g, int C) {
  if (g.cost == 0) return 0;
  const int line = p.hu * g.nkt, ks = block_tiles(tiles_of(p, g.n), C, line);
  return g.n * p.pg * ((line + ks - 1) / ks + p.hu);
}
// ... and of the item of block `blk` (first tile at, len tiles), pair q and head
// unit h, from the group's first on.
__device__ __forceinline__ int item_row(int n, int pg, int tpt, int nkt, int blk, int at, int len,
                                        int q, int h) {
  const int h0 = at / nkt, heads = (at + len - 1) / nkt - h0 + 1;
  return n * pg * (blk + h0) + q * 2 * tpt * pg * heads +
         (h - h0) * min(2 * tpt, n - q * 2 * tpt) * pg;
}
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
  r.cost = p.hu * tiles_of(p, r.n) * r.nkt;
  return r;
}

// group_starts must start at 0, never decrease and end at num_seqs: anything
// else makes the whole call a plain decode (no prefix is shared).  A prefix
// length that does not fit is taken as none.  Returns whether the groups are
// usable; *total is the batch's cost.
__device__ inline bool check_groups(const Params &p, int lane, bool report, int *total) {
  bool bad = false, bad_len = false;
  int sum = 0;
  if (lane == 0)
    bad = __ldg(p.group_starts) != 0 || __ldg(p.group_starts + p.num_groups) != p.num_seqs;
  for (int g = lane; g < p.num_groups; g += 32) {
    const int a = __ldg(p.group_starts + g), e = __ldg(p.group_starts + g + 1);
    const int len = __ldg(p.prefix_lens + g);
    const bool odd = a < 0 || e < a || e > p.num_seqs;
    bad |= odd;
    bad_len |= len < 0 || len > p.max_prefix || len > p.capacity;
    if (!odd) sum += group_geom(p, g).cost;
  }
  bad = __any_sync(0xffffffffu, bad);
  bad_len = __any_sync(0xffffffffu, bad_len);
  *total = bad ? 0 : __reduce_add_sync(0xffffffffu, sum);
  if (report && lane == 0) {
    if (bad) raise_error(p.err, PA_DEVERR_CU_SEQLENS);
    if (bad_len) raise_error(p.err, PA_DEVERR_CONTEXT);
  }
  return !bad;
}

__device__ __forceinline__ int run_cost(int total, int runs) {
  const int c = static_cast<int>((static_cast<unsigned>(total) + runs - 1) / runs);
  return c < 2 ? 2 : c;
}

// Sum of v over the lanes up to this one.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// What the joining kernel needs, in kInfoWords words: first the run cost C, then
// for each sequence its prefix length (0: none), the group's first sequence, its
// size, its first cost position and workspace row.  Warp-collective.
constexpr int kInfoWords = 8;
__device__ inline void write_info(const Params &p, int lane, bool good, int total) {
  const int C = run_cost(total, gridDim.x);
  if (lane == 0) p.ws_info[0] = C;
  if (!good) {
    for (int b = lane; b < p.num_seqs; b += 32)
      p.ws_info[static_cast<int64_t>(b + 1) * kInfoWords] = 0;
    return;
  }
  int gbase = 0, rbase = 0;
  for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
    const GroupGeom r = group_geom(p, g0 + lane);
    const int incl = warp_scan(r.cost, lane);
    const int lo = gbase + incl - r.cost;
    gbase += __shfl_sync(0xffffffffu, incl, 31);
    int row = r.first * p.hq;
    if (p.blocks) {
      const int rows = group_rows(p, r, C), rincl = warp_scan(rows, lane);
      row = rbase + rincl - rows;
      rbase += __shfl_sync(0xffffffffu, rincl, 31);
    }
    for (int i = 0; i < 32 && g0 + i < p.num_groups; ++i) {
      const int first = __shfl_sync(0xffffffffu, r.first, i);
      const int n = __shfl_sync(0xffffffffu, r.n, i);
      const int pre = __shfl_sync(0xffffffffu, r.prefix, i);
      const int at = __shfl_sync(0xffffffffu, lo, i);
      const int ws = __shfl_sync(0xffffffffu, row, i);
      for (int b = lane; b < n; b += 32) {
        int32_t *w = p.ws_info + static_cast<int64_t>(first + b + 1) * kInfoWords;
        *reinterpret_cast<int4 *>(w) = make_int4(pre, first, n, at);
        w[4] = ws;
      }
    }
  }
}

template <bool BLOCKS>  // false: no group has more than one query tile
struct PrefixSched {
  int x, xend, gbase, rbase, g0, C;

  __device__ void init(const Params &p, int total) {
    C = run_cost(total, gridDim.x);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * C;
    x = at < total ? static_cast<int>(at) : total;
    xend = total - x > C ? x + C : total;
    gbase = 0;
    rbase = 0;
    g0 = 0;
  }
  // The next piece: tiles [i0, i1) of a head unit for a pair, and the workspace
  // row of its states.
  __device__ bool next(const Params &p, int lane, GroupGeom *geom, int *head, int *pair, int *i0,
                       int *i1, int *ws_row) {
    while (x < xend) {
      for (; g0 < p.num_groups; g0 += 32) {
        const GroupGeom r = group_geom(p, g0 + lane);
        const int incl = warp_scan(r.cost, lane);
        const int hi = gbase + incl, lo = hi - r.cost;
        int rincl = 0, row = r.first * p.hq;  // workspace rows, the group's first
        if (BLOCKS && p.blocks) {
          const int rows = group_rows(p, r, C);
          rincl = warp_scan(rows, lane);
          row = rbase + rincl - rows;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, x >= lo && x < hi);
        if (hit) {
          const int src = __ffs(hit) - 1;
          GroupGeom s;
          s.first = __shfl_sync(0xffffffffu, r.first, src);
          s.n = __shfl_sync(0xffffffffu, r.n, src);
          s.nkt = __shfl_sync(0xffffffffu, r.nkt, src);
          s.prefix = __shfl_sync(0xffffffffu, r.prefix, src);
          const int start = __shfl_sync(0xffffffffu, lo, src);
          const int row0 = __shfl_sync(0xffffffffu, row, src);
          const int T = tiles_of(p, s.n), line = p.hu * s.nkt;
          int t0 = 0, blk = 0, len = line, q = 0, U = start;
          if (BLOCKS && T > 2) {
            const int ks = block_tiles(T, C, line);
            blk = (x - start) / (ks * T);
            t0 = blk * ks;
            len = min(ks, line - t0);
            q = (x - start - t0 * T) / (2 * len);
            U = start + t0 * T + q * 2 * len;
          }
          const int w = 2 * q + 1 < T ? 2 : 1;
          const int a = (x - U + w - 1) >> (w - 1);
          const int b = min(len, (xend - U + w - 1) >> (w - 1));
          if (a >= b) {  // the rest of the row's last tile lies in the run before
            x = min(xend, U + w * len);
            break;
          }
          const int at = t0 + a, h = at / s.nkt;
          *geom = s;
          *head = h;
          *pair = q;
          *i0 = at - h * s.nkt;
          *i1 = min(s.nkt, *i0 + b - a);
          x = min(xend, U + w * (a + *i1 - *i0));
          *ws_row = row0 + 256 * static_cast<int>(blockIdx.x) +
                    (BLOCKS && T > 2 ? item_row(s.n, p.pg, p.tpt, s.nkt, blk, t0, len, q, h)
                                     : h * s.n * p.pg);
          return true;
        }
        gbase = __shfl_sync(0xffffffffu, hi, 31);
        if (BLOCKS && p.blocks) rbase += __shfl_sync(0xffffffffu, rincl, 31);
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
// (without a runtime index, which would put the item into local memory)
__device__ __forceinline__ int use_count(const Item &it, int t) {
  return t ? it.cnt[1] : it.cnt[0];
}
__device__ __forceinline__ int use_step(const Item &it) { return (it.flags & kTurns) ? 2 : 1; }

// -------------------------------------------------------------- the kernel --
// COMPACT: P is formed by a loop over 32 columns at a time, their S read once
// more from TMEM, instead of 128 columns unrolled: a third of the softmax's
// instructions, but each of its steps fills and drains the pipelines.  While
// both streams' softmaxes run at once, as at the start of an item, they wait
// for instructions, in the steady state for each other: see the launchers.
template <class E, int D, int MODE, bool COMPACT>
__global__ void __launch_bounds__(kThreads, 1)
    flash_kernel(const Params p, const __grid_constant__ CUtensorMap tmq,
                 const __grid_constant__ CUtensorMap tmk,
                 const __grid_constant__ CUtensorMap tmv) {
  using L = Layout<D, MODE>;
  constexpr bool PAGED = kIsPaged<MODE>, SINGLE = kIsSingle<MODE>;
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
    if (lane == 0) ok = wait_for(bar(b), parity, p.wait_ns);
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
      if (i >= L::kQEmpty && i < L::kQEmpty + L::NQ) n = SINGLE ? 2 : 1;
      if (i >= L::kKEmpty && i < L::kKEmpty + L::NK) n = 2;    // either stream
      if (i >= L::kVEmpty && i < L::kVEmpty + L::NV) n = 2;
      if (i >= L::kVFixed && i < L::kVFixed + L::NV) n = 4;    // the epilogue's warps
      if (i >= L::kItemEmpty && i < L::kItemEmpty + kItemRing) n = kItemTakers;
      mbar_init(bar(i), n);
    }
    fence_barrier_init();
  }
  if (warp == kMmaWarp0) {
    tmem_alloc(smem_u32(const_cast<int *>(misc)), kTmemCols);
    tmem_relinquish();
  }
  // The prefix pass's scheduler reads the batch while the others set up.
  PrefixSched<MODE == kPaged> xs;
  bool groups_ok = true;
  int groups_cost = 0;
  if constexpr (PAGED) {
    if (warp == kSchedWarp) {
      groups_ok = check_groups(p, lane, blockIdx.x == 0, &groups_cost);
      xs.init(p, groups_cost);
    }
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
      int base = 0;
      uint32_t tails = 0;  // parity of each V buffer's tails so far
      PackedSched ps;
      if constexpr (!PAGED) {
        if (blockIdx.x == 0 && !check_cu(p, lane) && lane == 0)
          raise_error(p.err, PA_DEVERR_CU_SEQLENS);
        ps.init(p, lane);
      }
      int x = blockIdx.x;  // packed prompts: the item in hand
      int asked = 0;       // ... and requests made for the next
      for (int j = 0;; ++j) {
        Item it;
        it.live = 0;
        it.flags = 0;
        it.bad = 0;
        it.base = base;
        if constexpr (PAGED) {
          GroupGeom g;
          int head, pair, i0, i1;
          if (xs.next(p, lane, &g, &head, &pair, &i0, &i1, &it.ws_row)) {
            it.live = 1;
            it.q0 = g.first;
            it.ntok = g.n;
            it.tok0 = pair * 2 * p.tpt;
            it.head0 = head * p.pg;
            it.nkv = i1 - i0;
            it.key0 = i0 * kKeys;
            it.kend = min(g.prefix, i1 * kKeys);
            it.kv0 = g.first;
            const bool single = 2 * pair + 1 >= tiles_of(p, g.n);
            it.cnt[0] = it.cnt[1] = it.nkv;
            if (single) it.flags |= kSingle;
          }
        } else {
          int seq, pair, head;
          bool found = false;
          // Item j is taken when item j - 1 begins to load: early enough, and
          // no CTA holds items that an idle one could run.
          if (j > 0) ok = warp_wait(L::kBegun, (j - 1) & 1);
          while (!found && x >= 0 && ok) {  // (a CTA beyond the last item has none)
            if (j > 0) {
              if (lane == 0) {
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(bar(L::kNext), 16);
                clc_request(smem_u32(smem + L::kNextOff), bar(L::kNext));
              }
              ok = __all_sync(0xffffffffu,
                              wait_for(bar(L::kNext), asked & 1, p.wait_ns));
              ++asked;
              if (!ok) break;
              x = clc_answer(smem_u32(smem + L::kNextOff));
              __syncwarp();  // read by every lane before it is asked again
              if (x < 0) break;
            }
            if (x < ps.base) ps.init(p, lane);
            found = ps.find(p, x, lane, &seq, &pair, &head);
            if (!found && j == 0) break;
          }
          if (found && ok) {
            it.live = 1;
            it.q0 = __ldg(p.cu + seq);
            it.ntok = __ldg(p.cu + seq + 1) - it.q0;
            it.tok0 = (pair << p.pair_log2) * p.tpt;
            it.head0 = head * p.pg;
            it.key0 = 0;
            it.kend = it.ntok;
            it.kv0 = it.q0;
            it.ws_row = 0;
#pragma unroll
            for (int t = 0; t < 2; ++t) {  // keys up to those of the tile's last token
              const int first = it.tok0 + t * p.tpt;
              int keys = first < it.ntok && t <= p.pair_log2 ? it.ntok : 0;
              if (p.causal && keys > 0) keys = min(keys, first + p.tpt);
              it.cnt[t] = (keys + kKeys - 1) / kKeys;
            }
            it.nkv = max(it.cnt[0], it.cnt[1]);
            if (it.cnt[1] == 0) it.flags |= kSingle;
          }
        }
        if (it.live) {
          it.kvh = it.head0 / p.group;
          if (it.key0 + it.nkv * kKeys > it.kend) {
            const int slot = (base + it.nkv - 1) % L::NV;
            it.flags |= kTail | ((tails >> slot) & 1u ? kTailOdd : 0);
            tails ^= 1u << slot;
          }
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
      // a request that was given up on still lands before the CTA leaves
      if (asked > 0 && lane == 0) wait_for(bar(L::kNext), (asked - 1) & 1, kFullWait);
      if (!ok && lane == 0) give_up();
      if constexpr (PAGED) {
        if (blockIdx.x == 0) write_info(p, lane, groups_ok, groups_cost);
      }
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
      int nk = 0, nv = 0;           // loads issued
      int nq0 = 0, nq1 = 0;         // ... of query tiles, by stream
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
      auto load_q = [&](const Item &it, int t) {
        const int qi = t ? nq1 : nq0;
        const int slot = L::q_slot(t, qi), use = L::q_use(t, qi);
        if (use > 0 && !warp_wait(L::kQEmpty + slot, (use - 1) & 1)) return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::kQFull + slot), q_bytes);
          const int tok = p.q_off + it.q0 + it.tok0 + ((it.flags & kSingle) ? 0 : t * p.tpt);
          const uint32_t dst = smem_u32(smem + L::kQOff + slot * L::kTile);
#pragma unroll
          for (int h = 0; h < L::kHalves; ++h)
            tma_load_3d(dst + h * kHalf, &tmq, bar(L::kQFull + slot), h * 64, it.head0, tok);
        }
        __syncwarp();
        if (t) ++nq1;
        else ++nq0;
        return true;
      };
      for (int j = 0; ok; ++j) {
        Item it;
        ok = peek_item(j, &it);
        if (!ok || !it.live || misc[1]) break;
        if (lane == 0) mbar_arrive(bar(L::kBegun));
        // the streams' query tiles: the first one's before the item's first K
        // (a shared one counts as stream A's)
        const bool two = !SINGLE && it.cnt[0] > 0 && it.cnt[1] > 0;
        const int t_first = SINGLE || it.cnt[0] > 0 ? 0 : 1;
        // PAGED: this lane's block ids, the next tile's in flight
        const int32_t *bt = PAGED ? p.block_table + it.kv0 * p.bt_stride : nullptr;
        auto load_id = [&](int i) {
          const int key = it.key0 + i * kKeys + lane * bs;
          return (lane < nbox && i < it.nkv && key < it.kend) ? __ldg(bt + key / bs) : -1;
        };
        int id = PAGED ? load_id(0) : 0;
        // (the last item's V tail first: nothing of this item holds it back)
        if (v_pos >= 0) {
          ok = load_v();
          v_pos = -1;
        }
        if (ok) ok = load_q(it, t_first);
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
          if (ok && i == 0 && two) ok = load_q(it, 1);
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
        for (int n = nq0 - 1; n >= 0 && n >= nq0 - L::kQA; --n)
          wait_for(bar(L::kQFull + L::q_slot(0, n)), L::q_use(0, n) & 1, kFullWait);
        for (int n = nq1 - 1; n >= 0 && n >= nq1 - L::kQB; --n)
          wait_for(bar(L::kQFull + L::q_slot(1, n)), L::q_use(1, n) & 1, kFullWait);
        for (int n = nk - 1; n >= 0 && n >= nk - L::NK; --n)
          wait_for(bar(L::kKFull + n % L::NK), (n / L::NK) & 1, kFullWait);
        for (int n = nv - 1; n >= 0 && n >= nv - L::NV; --n)
          wait_for(bar(L::kVFull + n % L::NV), (n / L::NV) & 1, kFullWait);
      }
      __syncwarp();
    } else {
      // ----------------------------------------------------------- MMA --
      // One warp per stream.  The whole warp runs the loop; MMAs and commits
      // are issued by one elected lane.  The tensor core runs one thread's
      // MMAs in order, so Q K^T may overwrite the S columns that the P V
      // before it reads.  Issuing runs at the tensor core's own pace, so a
      // step's waits and bookkeeping stand between its issues; with a warp per
      // stream the other stream's MMAs run meanwhile (one warp for both
      // measured 1740 cycles per tile step on long prompts, 1064 of them
      // issuing), and P V and the stream's next Q K^T go out in one block.
      //
      // Each stream accounts for every use of a K or V buffer (and of a Q
      // buffer, where the streams share it), in order: by a commit after the
      // MMAs that read it, or, for a tile it does not use, by an arrival once
      // the tile has landed (an earlier one would count towards the buffer's
      // use before).  So a stream sees every phase of the buffers it waits
      // for, and no wait can take an older phase for its own.
      const int t = warp - kMmaWarp0;
      const uint32_t id_qk = idesc_f16(E::kBF16, 128, 128, false) | (p.negate << 13);
      const uint32_t id_pv = idesc_f16(E::kBF16, 128, D, true);
      const uint64_t q_desc0 = sdesc_sw128(smem_u32(smem) + L::kQOff, 16, 1024);
      const uint64_t k_desc0 = sdesc_sw128(smem_u32(smem) + L::kKOff, 16, 1024);
      const uint64_t v_desc0 = sdesc_sw128(smem_u32(smem) + L::kVOff, kHalf, 1024);
      const uint32_t s_tm = tbase + t * 128, o_tm = tbase + 256 + t * 128;
      bool ok = true;
      // Every lane asks once; only a wait that is not over yet goes the long way.
      auto ready = [&](int b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar(b), parity)) != 0;
      };
      auto wait = [&](int b, uint32_t parity) {
        return ready(b, parity) || warp_wait(b, parity);
      };
      constexpr int kNone = 0x7fffffff;
      int j = -1;              // the item whose tiles are being issued ...
      int end = 0, left = 0;   // ... its end, its Q K^T still to issue
      int np = kNone;          // ring position of the next Q K^T, where it is known
      int step = 1;            // the item's ring step
      int q = -1;              // the stream's current query tile
      bool first = false, tail = false, odd = false, ended = false, unused = false;
      int kdone = 0, vdone = 0;  // K and V uses accounted for
      int items = 0, psteps = 0; // items begun (P V), P tiles taken
      // the step whose Q K^T is out and whose P V is to come
      int pn = kNone;
      bool pfirst = false, plast = false, ptail = false, podd = false;

      // Moves on to item j + 1 (exhausted stream).
      auto next_item = [&]() {
        Item it;
        ok = peek_item(j + 1, &it);
        if (j >= 0) drop_item(j);
        ++j;
        if (!ok || !it.live) {
          ended = true;
          if (ok) drop_item(j);
          np = kNone;
          return;
        }
        end = it.base + it.nkv;
        left = use_count(it, t);
        np = left > 0 ? use_first(it, t) : kNone;
        step = use_step(it);
        first = true;
        tail = (it.flags & kTail) != 0;
        odd = (it.flags & kTailOdd) != 0;
        if (left > 0 || SINGLE) ++q;
        unused = left == 0;
      };
      // Accounts for the tiles before ring position m that this stream does
      // not use.
      auto skip_to = [&](int m) {
        while (ok && kdone < m) {
          ok = wait(L::kKFull + kdone % L::NK, (kdone / L::NK) & 1);
          if (lane == 0) mbar_arrive(bar(L::kKEmpty + kdone % L::NK));
          ++kdone;
        }
        while (ok && vdone < m) {
          ok = wait(L::kVFull + vdone % L::NV, (vdone / L::NV) & 1);
          if (lane == 0) mbar_arrive(bar(L::kVEmpty + vdone % L::NV));
          ++vdone;
        }
      };
      // The elected lane's part of S = Q K_n^T.
      auto issue_qk = [&](int n) {
        const int qs = L::q_slot(t, q);
        const uint64_t qd = q_desc0 + static_cast<uint64_t>(qs) * (L::kTile >> 4);
        const uint64_t kd = k_desc0 + static_cast<uint64_t>(n % L::NK) * (L::kTile >> 4);
        // K step k: 16 columns = 32 bytes into a 128-byte swizzled row, the
        // second 64 columns in the tile's second half
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
          umma_f16_ss(s_tm, qd + off, kd + off, id_qk, k > 0 ? 1u : 0u);
        }
        umma_commit(bar(L::kSFull + t));
        umma_commit(bar(L::kKEmpty + n % L::NK));
        if (left == 1) umma_commit(bar(L::kQEmpty + qs));
      };
      // ... and the bookkeeping after it.
      auto qk_issued = [&](int n) {
        pn = n;
        pfirst = first;
        first = false;
        plast = --left == 0;
        ptail = tail && n + 1 == end;
        podd = odd;
        np = plast ? kNone : n + step;
      };

      while (ok) {
        // P V of the pending step, and the next Q K^T with it where its
        // operands are there already.
        if (pn != kNone) {
          const int n = pn;
          if (left == 0) next_item();  // where the stream goes on, if at once
          bool along = false;
          if (ok && np <= n + 2) {
            const int kb = L::kKFull + np % L::NK;
            const uint32_t kp = (np / L::NK) & 1;
            // By turns the load of K is what the stream waits for: only look.
            // Else K is about to land, and waiting for it keeps P V and Q K^T
            // in one block (prefix pass, looking / waiting: 64 / 72 us on 64
            // sequences in 6 groups, 365 / 351 on 256 of one).
            along = MODE != kPacked && step == 2
                        ? __all_sync(0xffffffffu, mbar_test(bar(kb), kp)) != 0
                        : ready(kb, kp);
            if (along && first) along = ready(L::kQFull + L::q_slot(t, q), L::q_use(t, q) & 1);
          }
          if (ok && pfirst) {  // O of the stream's previous item has been read
            if (items > 0) ok = wait(L::kOFree + t, (items - 1) & 1);
            ++items;
          }
          if (ok) ok = wait(L::kVFull + n % L::NV, (n / L::NV) & 1);
          if (ok && ptail) {
            // (the buffer's tails before it have been cleared and used)
            ok = wait(L::kVFixed + n % L::NV, podd ? 1 : 0);
          }
          if (ok) ok = wait(L::kPFull + t, psteps & 1);
          if (!ok) break;
          ++psteps;
          tc_fence_after();
          const uint64_t vd = v_desc0 + static_cast<uint64_t>(n % L::NV) * (L::kTile >> 4);
          const uint32_t acc0 = pfirst ? 0u : 1u;
          if (elect_one()) {
            // O += P V_n, P from TMEM; K step k: 16 keys = 16 rows of 128
            // bytes of the MN-major V tile
#pragma unroll
            for (int k = 0; k < 8; ++k)
              umma_f16_ts(o_tm, s_tm + 8 * k, vd + ((k * 2048) >> 4), id_pv, k > 0 ? 1u : acc0);
            if (plast) umma_commit(bar(L::kOFull + t));
            umma_commit(bar(L::kVEmpty + n % L::NV));
            if (along) issue_qk(np);
          }
          __syncwarp();
          vdone = n + 1;
          pn = kNone;
          if (along) {
            const int m = np;
            qk_issued(m);
            skip_to(m);       // the tiles in between
            kdone = m + 1;
            continue;
          }
        }
        // Otherwise walk to the next tile the stream uses.
        while (ok && !ended && left == 0) {
          skip_to(end);
          if (SINGLE && unused && ok) {
            ok = wait(L::kQFull + L::q_slot(t, q), L::q_use(t, q) & 1);
            if (lane == 0) mbar_arrive(bar(L::kQEmpty + L::q_slot(t, q)));
          }
          if (ok) next_item();
        }
        if (ended) {
          skip_to(end);       // of the last item, which is over
          break;
        }
        if (!ok) break;
        const int m = np;
        skip_to(m);
        if (ok && first) ok = wait(L::kQFull + L::q_slot(t, q), L::q_use(t, q) & 1);
        if (ok) ok = wait(L::kKFull + m % L::NK, (m / L::NK) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) issue_qk(m);
        __syncwarp();
        qk_issued(m);
        kdone = m + 1;
      }
      if (!ok && lane == 0) give_up();
      // Every MMA issued above has completed once this barrier fires (the
      // full bound: TMEM is freed after it).
      if (elect_one()) umma_commit(bar(L::kFin + t));
      __syncwarp();
      if (lane == 0) wait_for(bar(L::kFin + t), 0, kFullWait);
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
      if (it.flags & kTail) {
        // V rows past the item's last key may hold anything (another
        // sequence's rows, never-written pool rows, even NaN); their weights
        // are 0, but 0 * NaN is NaN: they are cleared once the tile has
        // landed, before the P V that reads it (K's scores are masked).  The
        // load is waited for only once it is out (an earlier phase of the
        // buffer would pass for it otherwise), one phase of kTailIn per tail
        // in the buffer: the next one there needs this one cleared and used.
        const int n = it.base + it.nkv - 1, slot = n % L::NV;
        ok = wait_for(bar(L::kTailIn + slot), (it.flags & kTailOdd) ? 1 : 0, p.wait_ns);
        ok = ok && wait_for(bar(L::kVFull + slot), (n / L::NV) & 1, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          drop_item(j);
          break;
        }
        uint8_t *vt = smem + L::kVOff + slot * L::kTile;
        const int first = it.kend - it.key0 - (it.nkv - 1) * kKeys;  // 1..127
        for (int i = r; i < (kKeys - first) * (D / 8); i += 128) {
          const int row = first + i / (D / 8), c16 = i % (D / 8);
          *reinterpret_cast<uint4 *>(vt + (c16 >> 3) * kHalf + row * 128 + (c16 & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // generic writes before the tensor core reads
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kVFixed + slot));
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
          ok = ok && wait_for(bar(L::kOFull + t), done[t] & 1, p.wait_ns);
          ok = ok && wait_for(bar(L::kMLFull + t), done[t] & 1, p.wait_ns);
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
          const float inv = ll == 0.f ? 0.f : 1.f / ll;
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
          if (row_ok)
            *reinterpret_cast<float2 *>(p.ws_ml + ws * 2) = make_float2(mm, bad ? 0.f : ll);
        } else {
          orow = static_cast<typename E::T *>(p.out) +
                 static_cast<int64_t>(it.q0 + tok) * p.out_row_stride + (it.head0 + hl) * D;
        }
        const int t0 = use[0] ? 0 : 1;
        const bool both = use[0] && use[1];
        const uint64_t fa = f2_pack(t0 ? f[1] : f[0], t0 ? f[1] : f[0]);
        const uint64_t fb = f2_pack(f[1], f[1]);
        // rows that saw no key are 0, whatever O holds; a sum that is NaN (a query
        // or a visible key was) is passed on
        const bool none = ll == 0.f || bad;
        const bool any_none = __any_sync(0xffffffffu, none && row_ok);
        // 32 bytes a lane and store where rows allow it: a store's 32 rows are
        // 32 lines to the load/store unit either way (24 prompts of 2691 tokens
        // on average, 40/8: 497 us, with 16 bytes 515)
        const bool wide = PAGED || p.out_wide;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32];
          tmem_ld32(o_tm + t0 * 128 + c, v);
          uint64_t o[16];  // column pairs
          if (both) {
            uint32_t x[32];
            tmem_ld32(o_tm + 128 + c, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = f2_fma(f2_words(x[2 * i], x[2 * i + 1]), fb,
                            f2_mul(f2_words(v[2 * i], v[2 * i + 1]), fa));
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = f2_mul(f2_words(v[2 * i], v[2 * i + 1]), fa);
          }
          if (any_none) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = none ? 0ull : o[i];
          }
          constexpr int kWords = PAGED ? 32 : 16;
          uint32_t w[kWords];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            f2_unpack(o[i], a, b);
            if constexpr (PAGED) {
              w[2 * i] = __float_as_uint(a);
              w[2 * i + 1] = __float_as_uint(b);
            } else {
              w[i] = E::pack2(a, b);
            }
          }
          if (row_ok) {
            uint32_t *dst = PAGED ? reinterpret_cast<uint32_t *>(wrow + c)
                                  : reinterpret_cast<uint32_t *>(orow + c);
            if (wide) {
#pragma unroll
              for (int i = 0; i < kWords; i += 8) store_32b(dst + i, w + i);
            } else {
#pragma unroll
              for (int i = 0; i < kWords; i += 4)
                *reinterpret_cast<uint4 *>(dst + i) =
                    make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
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
      const int cnt = use_count(it, t);
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
        ok = wait_for(bar(L::kSFull + t), n & 1, p.wait_ns);
        tc_fence_after();
        // Columns past `bound` are hidden: where a tile has any, its S goes
        // through a loop (not unrolled, for the instruction cache's sake).
        // (A wait that ran out in any lane ends the whole warp here.)
        if (__any_sync(0xffffffffu, bound < kKeys - 1 || !ok)) {
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 32) {
            if (!__any_sync(0xffffffffu, bound < c + 31)) continue;
            uint32_t h[32];
            tmem_ld32(s_tm + c, h);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (k > bound - c) h[k] = __float_as_uint(-INFINITY);
            tmem_st32(s_tm + c, h);
          }
          tmem_wait_st();
        }
        // The whole S row in one TMEM round trip.
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld32(s_tm + c * 32, *reinterpret_cast<uint32_t(*)[32]>(v + c * 32));
        tmem_wait_ld();
        float mx[4];  // raw scores (the factor is positive), as a tree
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mx[c] = max3(__uint_as_float(v[c]), __uint_as_float(v[4 + c]), __uint_as_float(v[8 + c]));
#pragma unroll
        for (int c = 12; c + 7 < 128; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = max3(mx[k], __uint_as_float(v[c + k]), __uint_as_float(v[c + 4 + k]));
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(v[124 + k]));
        const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sl;
        const bool raise = mt > m_ref + kRescaleThreshold;  // false for a fully masked row
        const float m_new = raise ? mt : m_ref;
        const float corr = raise ? fast_exp2(m_ref - m_new) : 1.f;
        // P = 2^(s - m), rounded to the input type and packed, goes to TMEM
        // over S, 8 words at a time; S(n) being complete means the P V that
        // read these columns before is done.
        const float mu = m_new == -INFINITY ? 0.f : m_new;
        const uint64_t sl2 = f2_pack(sl, sl), nmu2 = f2_pack(-mu, -mu);
        uint64_t rs[2] = {0, 0};  // the row's sum, in four parts
        auto form = [&](const uint32_t *y, int pairs, uint32_t dst) {  // column pairs of S to P
          uint32_t pw[8];
#pragma unroll
          for (int c = 0; c < pairs; ++c) {
            float x0, x1;
            f2_unpack(f2_fma(f2_words(y[2 * c], y[2 * c + 1]), sl2, nmu2), x0, x1);
            x0 = fast_exp2(x0);  // 2^-inf = 0 where masked
            x1 = fast_exp2(x1);
            pw[c & 7] = E::pack2(x0, x1);
            rs[c & 1] = f2_add(rs[c & 1], f2_pack(x0, x1));
            if ((c & 7) == 7) tmem_st8(dst + c - 7, pw);
          }
        };
        if constexpr (COMPACT) {
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t y[32];
            tmem_ld32(s_tm + c, y);
            tmem_wait_ld();
            form(y, 16, s_tm + c / 2);
          }
        } else {
          form(v, 64, s_tm);
        }
        tmem_wait_st();
        if (i > 0 && __any_sync(0xffffffffu, raise)) {
          // O holds exactly the sum so far: S(n) being complete means Q K^T
          // of this tile ran, which was issued after the P V before it.
#pragma unroll 1
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
        float r0, r1;
        f2_unpack(f2_add(rs[0], rs[1]), r0, r1);
        l = l * corr + (r0 + r1);
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
  if (warp == kMmaWarp0) {
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

template <class E, int D, int MODE, bool COMPACT>
cudaError_t launch(const Params &p, const CUtensorMap &tmq, const CUtensorMap &tmk,
                   const CUtensorMap &tmv, int grid, cudaStream_t stream) {
  constexpr auto kernel = flash_kernel<E, D, MODE, COMPACT>;
  cudaError_t e = allow_dynamic_smem<kernel>();
  if (e == cudaSuccess) e = check_register_pool<kernel>();
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                    Layout<D, MODE>::kBytes, stream, p, tmq, tmk, tmv);
}

}  // namespace flash
}  // namespace pa
