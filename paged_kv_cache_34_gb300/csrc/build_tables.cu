// build_tables.cu -- a serving step's metadata from request lengths, on the
// GPU: cumulative query lengths, token positions, cache slots, and the block
// table entries of the blocks the step takes off the free list.
//
// Operation (cannbot-skills "model-infer-kvcache" skill page §3.1-3.3: the
// logical block of a token is pos / block_size, its slot is
// block * block_size + pos % block_size; lqnn.cn article §3.1 cu_seqlens):
// request b holds c_b cached tokens and gets n_b new ones.  With
//     have_b = ceil(c_b / bs),  need_b = ceil((c_b + n_b) / bs),
//     t_b = need_b - have_b,    U_b = t_0 + ... + t_b,
// its new blocks are the free list's entries F - 1 - (U_b - t_b) downwards,
// and token i of request b sits at cu_b + i, position c_b + i.
//
// Everything follows from two prefix sums over the requests (tokens and
// blocks).  One launch: every CTA forms both sums over all requests in shared
// memory (a few KB of input that stays in L2), so no CTA waits for another
// and nothing is kept in a workspace; then the CTAs share the tokens out in
// runs, four per thread.  A warp finds the requests of its first and last token
// in the shared sums, 32 probes at a time, and its lanes theirs between them.
// A new block's table entry is written by the thread that holds the block's
// first token, which is always a new token.
//
// Bound by latency, not by bytes: launch, lengths, sums, search, block ids,
// stores follow one another.  Measured (graph replay, GB300): 3.0 us for one
// token of one request, 4.7 us for 1024 requests of 16 tokens, 11.2 us for
// 1024 prompts of up to 2000 tokens (a million in all, 12.6 MB written).  Two
// CTAs per SM at most, in several steps: a third repeats the sums more often
// and takes registers from the token loop (1024 x 1000 tokens: 12.4 us against
// 8.7), one alone leaves no room for the next launch's start beside it
// (back-to-back calls 15.0 us against 11.2).
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 2;
constexpr int kGroup = 4;       // tokens per thread and step: one 16-byte store of
                                // positions, two of slots
constexpr int kMaxEntries = 4096;  // most sums kept per CTA (32 KB: no opt-in size)

struct TablesParams {
  int32_t *block_table;
  int64_t bt_stride;
  const int32_t *ctx, *query;
  const int32_t *free_blocks, *num_free;
  int32_t free_capacity;
  int32_t *ctx_out, *cu, *positions, *num_free_out;
  int64_t *slots;
  int32_t num_seqs, max_tokens, bs_log2;
  uint32_t capacity;  // tokens a block-table row can hold, below 2^31
  int64_t num_blocks;
  int32_t entries;    // sums kept in shared memory, one per `gran` requests
  int32_t gran;
  bool vec;           // slots and positions are 16-byte aligned
  int32_t *err;
};

__device__ __forceinline__ int32_t sat32(int64_t x) {
  return x > 0x7fffffff ? 0x7fffffff : static_cast<int32_t>(x);
}

struct Request {
  int32_t c, n;     // cached and new tokens (0, 0 when not valid)
  int32_t have, t;  // blocks held, blocks to take
  bool valid;
};

__device__ __forceinline__ Request load_request(const TablesParams &p, int b) {
  Request r;
  r.c = __ldg(p.ctx + b);
  r.n = __ldg(p.query + b);
  // c + n as unsigned cannot wrap for c, n >= 0; capacity < 2^31
  const uint32_t both = static_cast<uint32_t>(r.c) + static_cast<uint32_t>(r.n);
  r.valid = (r.c | r.n) >= 0 && both <= p.capacity;
  if (!r.valid) r.c = r.n = 0;
  const uint32_t mask = (1u << p.bs_log2) - 1;
  r.have = static_cast<int32_t>((static_cast<uint32_t>(r.c) + mask) >> p.bs_log2);
  r.t = static_cast<int32_t>(((r.valid ? both : 0u) + mask) >> p.bs_log2) - r.have;
  return r;
}

// The last entry in [lo, hi) of the ascending `sums` whose sum is <= t; the
// first one's is (warp-collective, 32 probes a round).
__device__ __forceinline__ int warp_find(const int32_t *sums, int lo, int hi, int64_t t, int lane) {
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && sums[at] <= t);
    const int k = 31 - __clz(le);  // the last probe that is <= t
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm) build_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t s_sums[];  // cu[entries], first block[entries]
  int32_t *s_cu = s_sums, *s_first = s_sums + p.entries;
  __shared__ int64_t s_warp_tok[kWarps], s_warp_blk[kWarps];
  __shared__ int32_t s_taken[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();  // lengths and free list may come from earlier kernels
  griddep_launch_dependents();

  const int32_t nfree_in = __ldg(p.num_free);
  const int32_t nfree = min(max(nfree_in, 0), p.free_capacity);
  if (blockIdx.x == 0 && tid == 0 && nfree != nfree_in) raise_error(p.err, PA_DEVERR_NO_BLOCKS);

  // Thread i sums requests [i * per, (i + 1) * per); per is a multiple of
  // gran, so that shared entries start where a thread's count does.
  const int chunks = (p.entries + kThreads - 1) / kThreads;  // shared entries per thread
  const int64_t per = static_cast<int64_t>(chunks) * p.gran;
  const int b0 = static_cast<int>(min(tid * per, static_cast<int64_t>(p.num_seqs)));
  const int b1 = static_cast<int>(min(b0 + per, static_cast<int64_t>(p.num_seqs)));
  int64_t tok = 0, blk = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    const Request r = load_request(p, b);
    tok += r.n;
    blk += r.t;
  }
  int64_t itok = tok, iblk = blk;  // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t vt = __shfl_up_sync(0xffffffffu, itok, o);
    const int64_t vb = __shfl_up_sync(0xffffffffu, iblk, o);
    if (lane >= o) {
      itok += vt;
      iblk += vb;
    }
  }
  if (lane == 31) {
    s_warp_tok[warp] = itok;
    s_warp_blk[warp] = iblk;
  }
  __syncthreads();
  int64_t base_tok = 0, base_blk = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      base_tok += s_warp_tok[w];
      base_blk += s_warp_blk[w];
    }
    total += s_warp_tok[w];
  }
  tok = base_tok + itok - tok;  // exclusive: before this thread's requests
  blk = base_blk + iblk - blk;

  // Second walk: the shared sums and, shared out over the CTAs by warp, the
  // per-request outputs.  CTA 0 also finds how many blocks are taken.
  const bool writes = warp % gridDim.x == blockIdx.x;
  int32_t taken = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    const Request r = load_request(p, b);
    if (p.gran == 1 || b % p.gran == 0) {
      s_cu[b / p.gran] = sat32(tok);
      s_first[b / p.gran] = sat32(blk);
    }
    const bool fits = r.n == 0 || tok + r.n <= p.max_tokens;
    const bool blocks = r.t == 0 || blk + r.t <= nfree;
    if (fits && blocks && r.t > 0) taken = static_cast<int32_t>(blk + r.t);
    if (writes) {
      p.cu[b] = sat32(tok);
      p.ctx_out[b] = r.valid && fits && blocks ? r.c + r.n : 0;
      if (!r.valid) raise_error(p.err, PA_DEVERR_CONTEXT);
      if (!fits) raise_error(p.err, PA_DEVERR_CU_SEQLENS);
      if (!blocks) raise_error(p.err, PA_DEVERR_NO_BLOCKS);
    }
    tok += r.n;
    blk += r.t;
  }
  if (blockIdx.x == 0) {
    taken = __reduce_max_sync(0xffffffffu, taken);
    if (lane == 0) s_taken[warp] = taken;
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    p.cu[p.num_seqs] = sat32(total);
    int32_t m = 0;
    for (int w = 0; w < kWarps; ++w) m = max(m, s_taken[w]);
    *p.num_free_out = nfree - m;
  }

  // Tokens.
  const int32_t real = static_cast<int32_t>(min(total, static_cast<int64_t>(p.max_tokens)));
  const int32_t bmask = (1 << p.bs_log2) - 1;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads * kGroup;
  // The physical block (-1: none) of logical block lb of request b, which
  // keeps `have` blocks and takes its first new one at list place `first`; the
  // holder of a taken block's first token writes its table entry.
  auto block_of = [&](int b, int32_t have, int32_t first, int32_t lb, bool opens) {
    int32_t *entry = p.block_table + b * p.bt_stride + lb;
    const bool taken_now = lb >= have;
    int32_t id = taken_now ? __ldg(p.free_blocks + (nfree - 1 - (first + lb - have))) : *entry;
    if (id < 0 || id >= p.num_blocks) {
      raise_error(p.err, PA_DEVERR_BLOCK_ID);
      id = -1;
    }
    if (taken_now && opens) *entry = id;
    return id;
  };
  auto slot_of = [&](int32_t id, int32_t pos) {
    return id < 0 ? static_cast<int64_t>(-1)
                  : (static_cast<int64_t>(id) << p.bs_log2) + (pos & bmask);
  };
  for (int64_t w0 = (static_cast<int64_t>(blockIdx.x) * kThreads + (tid & ~31)) * kGroup;
       w0 < p.max_tokens; w0 += stride) {
    const int64_t t0 = w0 + lane * kGroup;
    int64_t slot[kGroup];
    int32_t pos[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      slot[k] = -1;
      pos[k] = 0;
    }
    if (w0 < real) {
      // the entries that hold the warp's first and last token, then each
      // lane's own between them
      int lo = warp_find(s_cu, 0, p.entries, w0, lane);
      int hi = warp_find(s_cu, lo, p.entries,
                         min(w0 + 32 * kGroup, static_cast<int64_t>(real)) - 1, lane) + 1;
      if (t0 < real) {
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_cu[mid] <= t0) lo = mid;
          else hi = mid;
        }
        int b = lo * p.gran;
        int32_t cu = s_cu[lo], first = s_first[lo];
        Request r = load_request(p, b);
        auto next_request = [&](int64_t t) {  // on to the one that holds t < real
          while (t >= static_cast<int64_t>(cu) + r.n) {
            cu += r.n;
            first = sat32(static_cast<int64_t>(first) + r.t);
            r = load_request(p, ++b);
          }
        };
        auto served = [&]() {
          return static_cast<int64_t>(cu) + r.n <= p.max_tokens &&
                 (r.t == 0 || static_cast<int64_t>(first) + r.t <= nfree);
        };
        next_request(t0);
        if (t0 + kGroup <= real && t0 + kGroup <= static_cast<int64_t>(cu) + r.n) {
          // all of one request: at most two blocks (block_size >= 8)
          const int32_t p0 = r.c + static_cast<int32_t>(t0 - cu), p3 = p0 + kGroup - 1;
#pragma unroll
          for (int k = 0; k < kGroup; ++k) pos[k] = p0 + k;
          if (served()) {
            const int32_t lb0 = p0 >> p.bs_log2, lb1 = p3 >> p.bs_log2;
            const int32_t id0 = block_of(b, r.have, first, lb0, (p0 & bmask) == 0);
            const int32_t id1 = lb1 != lb0 ? block_of(b, r.have, first, lb1, true) : id0;
#pragma unroll
            for (int k = 0; k < kGroup; ++k)
              slot[k] = slot_of((p0 + k) >> p.bs_log2 == lb0 ? id0 : id1, p0 + k);
          }
        } else {
#pragma unroll 1
          for (int k = 0; k < kGroup && t0 + k < real; ++k) {
            next_request(t0 + k);
            const int32_t at = r.c + static_cast<int32_t>(t0 + k - cu);
            const int64_t sl =
                served() ? slot_of(block_of(b, r.have, first, at >> p.bs_log2, (at & bmask) == 0),
                                   at)
                         : -1;
#pragma unroll
            for (int q = 0; q < kGroup; ++q)
              if (q == k) {
                pos[q] = at;
                slot[q] = sl;
              }
          }
        }
      }
    }
    if (p.vec && t0 + kGroup <= p.max_tokens) {
      longlong2 *s = reinterpret_cast<longlong2 *>(p.slots + t0);
      s[0] = make_longlong2(slot[0], slot[1]);
      s[1] = make_longlong2(slot[2], slot[3]);
      if (p.positions)
        *reinterpret_cast<int4 *>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        if (t0 + k >= p.max_tokens) break;
        p.slots[t0 + k] = slot[k];
        if (p.positions) p.positions[t0 + k] = pos[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_build_tables(const BuildTablesArgs &a, cudaStream_t stream) {
  TablesParams p;
  p.block_table = a.block_table;
  p.bt_stride = a.block_table_stride;
  p.ctx = a.context_lens;
  p.query = a.query_lens;
  p.free_blocks = a.free_blocks;
  p.num_free = a.num_free;
  p.free_capacity = a.free_capacity;
  p.ctx_out = a.context_lens_out;
  p.cu = a.cu_seqlens_q;
  p.positions = a.positions;
  p.num_free_out = a.num_free_out;
  p.slots = a.slot_mapping;
  p.num_seqs = a.num_seqs;
  p.max_tokens = a.max_tokens;
  p.bs_log2 = 0;
  while ((1 << p.bs_log2) < a.block_size) ++p.bs_log2;
  const int64_t capacity = static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size;
  p.capacity = static_cast<uint32_t>(capacity < 0x7fffffff ? capacity : 0x7fffffff);
  p.num_blocks = a.num_blocks;
  p.gran = (a.num_seqs + kMaxEntries - 1) / kMaxEntries;
  if (p.gran < 1) p.gran = 1;
  p.entries = (a.num_seqs + p.gran - 1) / p.gran;
  if (p.entries < 1) p.entries = 1;
  p.vec = (reinterpret_cast<uintptr_t>(a.slot_mapping) & 15u) == 0 &&
          (reinterpret_cast<uintptr_t>(a.positions) & 15u) == 0;
  p.err = a.d_error;
  const size_t smem = static_cast<size_t>(p.entries) * 2 * sizeof(int32_t);
  // At most one wave of CTAs, each thread taking the same number of steps.
  const int64_t blocks =
      (static_cast<int64_t>(a.max_tokens) + kThreads * kGroup - 1) / (kThreads * kGroup);
  const int64_t wave = static_cast<int64_t>(kCtasPerSm) * a.num_sms;
  const int64_t steps = (blocks + wave - 1) / wave;
  const int64_t grid = blocks > 0 ? (blocks + steps - 1) / steps : 1;
  return launch_pdl(build_tables_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem,
                    stream, p);
}

}  // namespace pa
