// attention_varlen.cu -- causal attention of packed prompts straight from
// their K and V rows: the launcher and instantiations of the tile engine in
// flash_kernel.cuh over plain rows.
//
// Operation (lqnn.cn article §3.1 cu_seqlens, §4.4 packed attention;
// cannbot-skills page App. C sparse_mode 3): sequence b owns rows
// cu_seqlens[b] .. cu_seqlens[b+1]-1 of query, key and value; row i of it
// sees its keys 0..i (all of them without `causal`).
#include "flash_kernel.cuh"

namespace pa {

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
  p.causal = a.causal;
  p.cu = a.cu_seqlens;
  p.num_seqs = a.num_seqs;
  p.total = a.total;
  p.max_seqlen = a.max_seqlen;
  p.err = a.d_error;
  p.wait_ns = flash::wait_limit(a.wait_ns);
  p.out_wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_row_stride % 16 == 0;
  p.kv_bytes = 4 * a.head_dim;
  const int grid = static_cast<int>(a.grid);
  const bool bf = a.dtype == PA_BF16;
  if (a.head_dim == 64)
    return bf ? flash::launch<BF16, 64, flash::kPacked>(p, a.tm_q, a.tm_k, a.tm_v, grid, stream)
              : flash::launch<F16, 64, flash::kPacked>(p, a.tm_q, a.tm_k, a.tm_v, grid, stream);
  return bf ? flash::launch<BF16, 128, flash::kPacked>(p, a.tm_q, a.tm_k, a.tm_v, grid, stream)
            : flash::launch<F16, 128, flash::kPacked>(p, a.tm_q, a.tm_k, a.tm_v, grid, stream);
}

}  // namespace pa
