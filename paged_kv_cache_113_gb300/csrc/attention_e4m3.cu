// Decode attention over the 8-bit cache (pk_paged_attention_decode_e4m3).
//
// With K_t = 2^ek_t kc_t and V_t = 2^ev_t vc_t (e4m3 codes kc, vc):
//     x_t = scale * 2^ek_t <q, kc_t>
//     out = sum_t 2^(x_t - m) 2^ev_t vc_t / sum_t 2^(x_t - m)     (x in log2)
// Bound by memory: a token and KV head cost 2 (d + 1) bytes, half of bf16.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_rows.cuh"
#include "pagedkv.h"

using namespace pk;

extern "C" int pkx_take_attention_e4m3_error(cudaStream_t stream) {
  return take_error_word(g_rows_error, stream);
}

extern "C" int pkx_e4m3_resident_ctas(int, int) { return 3; }

namespace {

template <typename IO, int D>
pk_status run(const RowsParams &p, cudaStream_t stream) {
  pk_status st = launch_rows<E4M3, IO, D, 1>(p, stream);
  if (st != PK_OK || p.num_partitions == 1) return st;
  return launch_rows_merge<IO, D>(p, stream);
}

}  // namespace

extern "C" pk_status pk_paged_attention_decode_e4m3(
    void *out, const void *q, pk_dtype io_dtype, const void *k_cache, const void *v_cache,
    const uint8_t *kv_exp, const int32_t *block_tables, const int32_t *context_lens, float scale,
    int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks_per_seq, int32_t max_context_len,
    int32_t partition_size, const int32_t *work_items, int32_t num_items, void *workspace,
    size_t workspace_bytes, const pk_cache_desc *desc, void *stream) {
  if (!desc) return PK_ERR_INVALID_ARG;
  if (desc->dtype != PK_E4M3 || (io_dtype != PK_F32 && io_dtype != PK_BF16))
    return PK_ERR_UNSUPPORTED;
  const int32_t part = pk_paged_attention_resolve_partition(num_seqs, num_q_heads, max_context_len,
                                                            partition_size, desc);
  if (part < 0) return PK_ERR_INVALID_ARG;
  if (desc->block_size != 8 && desc->block_size != 16 && desc->block_size != 32)
    return PK_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PK_OK;
  if (!kv_exp || !aligned16(kv_exp)) return PK_ERR_INVALID_ARG;
  RowsParams p{};
  pk_status st = rows_params(p, out, q, k_cache, v_cache, block_tables, context_lens, scale, num_seqs,
                             num_seqs, 1, num_q_heads, max_blocks_per_seq, max_context_len, part,
                             work_items, num_items, workspace, workspace_bytes, *desc);
  if (st != PK_OK) return st;
  p.kv_exp = kv_exp;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (io_dtype == PK_F32) return desc->head_dim == 128 ? run<float, 128>(p, s) : run<float, 64>(p, s);
  return desc->head_dim == 128 ? run<__nv_bfloat16, 128>(p, s) : run<__nv_bfloat16, 64>(p, s);
}
