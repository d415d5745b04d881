// attention_varlen.cu -- causal attention of packed prompts straight from
// their K and V rows: the launcher and instantiations of the tile engine in
// flash_kernel.cuh over plain rows.
//
// Operation (lqnn.cn article §3.1 cu_seqlens, §4.4 packed attention;
// cannbot-skills page App. C sparse_mode 3): sequence b owns rows
// cu_seqlens[b] .. cu_seqlens[b+1]-1 of query, key and value; row i of it
// sees its keys 0..i (all of them without `causal`).
#include <type_traits>

#include "flash_kernel.cuh"

namespace pa {

// Prompts up to this long take the compact softmax: their items are few tiles
// each (16 x 1000 tokens 32/32 heads: 144 us against 156, 200 x 100 32/8: 93
// against 98, 16 of 50..2000 32/32: 274 against 276; but 24 of up to 2700 40/8:
// 483 against 473, 4 x 4096 32/8: 423 against 374).
constexpr int kCompactLen = 2048;

cudaError_t launch_attention_varlen(const AttentionVarlenArgs &a, cudaStream_t stream) {
  flash::Params p = {};
  p.out = a.out;
  p.out_row_stride = a.out_row_stride;
  p.hq = a.num_q_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.pg = a.packed_heads;
  p.tpt = 128 / a.packed_heads;
  p.hu = p.hq / p.pg;
  p.scale_log2 = a.scale_log2;
  p.negate = a.negate ? 1u : 0u;
  p.q_off = a.q_off;
  p.causal = a.causal;
  p.cu = a.cu_seqlens;
  p.num_seqs = a.num_seqs;
  p.total = a.total;
  p.max_seqlen = a.max_seqlen;
  p.err = a.d_error;
  p.wait_ns = flash::wait_limit(a.wait_ns);
  p.out_wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_row_stride % 16 == 0;
  p.kv_bytes = 4 * a.head_dim;
  p.pair_log2 = a.tiles == 2 ? 1 : 0;
  const int grid = static_cast<int>(a.grid);
  const bool compact = a.max_seqlen <= kCompactLen, bf = a.dtype == PA_BF16;
  auto launch = [&](auto e, auto d) {
    using E = decltype(e);
    constexpr int D = decltype(d)::value;
    if (a.tiles == 1)
      return flash::launch<E, D, flash::kPackedSingle, true>(p, a.tm_q, a.tm_k, a.tm_v, grid,
                                                             stream);
    return compact ? flash::launch<E, D, flash::kPacked, true>(p, a.tm_q, a.tm_k, a.tm_v, grid,
                                                               stream)
                   : flash::launch<E, D, flash::kPacked, false>(p, a.tm_q, a.tm_k, a.tm_v, grid,
                                                                stream);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (a.head_dim == 64) return bf ? launch(BF16{}, D64{}) : launch(F16{}, D64{});
  return bf ? launch(BF16{}, D128{}) : launch(F16{}, D128{});
}

}  // namespace pa
