// Attention of each sequence's drafted tokens over its cached context
// (pk_paged_attention_tree), for verifying a tree or a chain of drafts in one
// pass: the n drafted tokens are the last n of the context, their K/V already
// in the cache, and a 64-bit mask per token says which drafts it sees.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_rows.cuh"
#include "pagedkv.h"

namespace pk {

extern "C" int pkx_take_tree_attention_error(cudaStream_t stream) {
  return take_error_word(g_rows_error, stream);
}

namespace {

template <typename T, int D>
pk_status run(const RowsParams &p, cudaStream_t stream) {
  pk_status st = p.max_draft * p.group <= 8 ? launch_rows<T, T, D, 1>(p, stream)
                                            : launch_rows<T, T, D, 8>(p, stream);
  if (st != PK_OK || p.num_partitions == 1) return st;
  return launch_rows_merge<T, D>(p, stream);
}

pk_status check_tree(const pk_cache_desc *d, int32_t num_q_heads, int32_t max_context_len,
                     int32_t partition_size) {
  if (!d || d->num_blocks <= 0 || d->block_size <= 0 || d->num_kv_heads <= 0 || num_q_heads <= 0 ||
      max_context_len <= 0 || partition_size < 0)
    return PK_ERR_INVALID_ARG;
  if (d->dtype != PK_F32 && d->dtype != PK_BF16) return PK_ERR_UNSUPPORTED;
  if (num_q_heads % d->num_kv_heads != 0 || partition_size % d->block_size != 0)
    return PK_ERR_INVALID_ARG;
  if (num_q_heads / d->num_kv_heads > 8 || (d->head_dim != 64 && d->head_dim != 128))
    return PK_ERR_UNSUPPORTED;
  if (int64_t(d->num_blocks) * d->block_size > INT32_MAX) return PK_ERR_UNSUPPORTED;
  return PK_OK;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
    return n;
  cudaGetLastError();  // clear a failed query on a machine without a GPU
  return 152;
}

}  // namespace

extern "C" {

pk_status pk_tree_masks(const int32_t *parents, int32_t num_drafts, uint64_t *masks_out,
                        int32_t *depths_out) {
  if (num_drafts < 0 || num_drafts > PK_MAX_DRAFT) return PK_ERR_INVALID_ARG;
  if (num_drafts > 0 && (!parents || !masks_out)) return PK_ERR_INVALID_ARG;
  for (int32_t i = 0; i < num_drafts; ++i)
    if (parents[i] < -1 || parents[i] >= i) return PK_ERR_INVALID_ARG;
  int32_t depth[PK_MAX_DRAFT];
  for (int32_t i = 0; i < num_drafts; ++i) {
    masks_out[i] = (1ull << i) | (parents[i] >= 0 ? masks_out[parents[i]] : 0);
    depth[i] = parents[i] >= 0 ? depth[parents[i]] + 1 : 0;
    if (depths_out) depths_out[i] = depth[i];
  }
  return PK_OK;
}

size_t pk_tree_workspace_size(int32_t num_q_tokens, int32_t num_q_heads, int32_t max_context_len,
                              int32_t partition_size, const pk_cache_desc *desc) {
  if (num_q_tokens < 0 || check_tree(desc, num_q_heads, max_context_len, partition_size) != PK_OK ||
      partition_size == 0)
    return 0;
  const int64_t P = (int64_t(max_context_len) + partition_size - 1) / partition_size;
  if (P <= 1) return 0;
  return size_t(num_q_tokens) * num_q_heads * size_t(P) * (size_t(desc->head_dim) + 2) * sizeof(float);
}

pk_status pk_tree_plan(const int32_t *context_lens, int32_t num_seqs, int32_t max_draft_len,
                       int32_t num_q_heads, int32_t partition_size, const pk_cache_desc *desc,
                       int32_t *partition_out, int32_t *items_out, int32_t cap,
                       int32_t *num_items_out) {
  if (!partition_out || !num_items_out || num_seqs <= 0 || !context_lens || max_draft_len < 1 ||
      max_draft_len > PK_MAX_DRAFT || partition_size < -1)
    return PK_ERR_INVALID_ARG;
  *partition_out = 0;
  *num_items_out = 0;
  int32_t longest = 1;
  int64_t total = 0;
  for (int32_t s = 0; s < num_seqs; ++s) {
    longest = std::max(longest, context_lens[s]);
    total += std::max(context_lens[s], 1);
  }
  const pk_status st = check_tree(desc, num_q_heads, longest, std::max(partition_size, 0));
  if (st != PK_OK) return st;
  int32_t part = partition_size > 0 && partition_size < longest ? partition_size : 0;
  if (partition_size == -1) {
    const int64_t rows = int64_t(max_draft_len) * (num_q_heads / desc->num_kv_heads);
    const int64_t units = desc->num_kv_heads * ((rows + 127) / 128);
    const int64_t slots = int64_t(sm_count()) * 2;
    const int64_t W = std::max<int64_t>(1, (total * units + slots - 1) / slots);
    if (longest > 2 * W && longest > 1024) {
      const int64_t k = std::max<int64_t>(1, longest / W);
      int64_t n = (longest + k - 1) / k;
      n = std::max<int64_t>(512, (n + 63) / 64 * 64);
      n = (n + desc->block_size - 1) / desc->block_size * desc->block_size;
      part = n < longest ? int32_t(n) : 0;
    }
  }
  *partition_out = part;
  return pk_attention_work_items(context_lens, num_seqs, part, items_out, cap, num_items_out);
}

pk_status pk_paged_attention_tree(void *out, const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *block_tables, const int32_t *context_lens,
                                  const int32_t *q_offsets, const uint64_t *tree_mask, float scale,
                                  int32_t num_seqs, int32_t num_q_tokens, int32_t max_draft_len,
                                  int32_t num_q_heads, int32_t max_blocks_per_seq,
                                  int32_t max_context_len, int32_t partition_size,
                                  const int32_t *work_items, int32_t num_items, void *workspace,
                                  size_t workspace_bytes, const pk_cache_desc *desc, void *stream) {
  pk_status st = check_tree(desc, num_q_heads, max_context_len, partition_size);
  if (st != PK_OK) return st;
  if (num_seqs < 0 || num_q_tokens < 0 || max_draft_len < 0) return PK_ERR_INVALID_ARG;
  if (max_draft_len > PK_MAX_DRAFT) return PK_ERR_UNSUPPORTED;
  if (num_seqs == 0 || num_q_tokens == 0 || max_draft_len == 0) return PK_OK;
  if (!q_offsets || (tree_mask && (reinterpret_cast<uintptr_t>(tree_mask) & 7u)))
    return PK_ERR_INVALID_ARG;
  if (int64_t(num_q_tokens) * num_q_heads > INT32_MAX) return PK_ERR_UNSUPPORTED;
  RowsParams p{};
  st = rows_params(p, out, q, k_cache, v_cache, block_tables, context_lens, scale, num_seqs,
                   num_q_tokens, max_draft_len, num_q_heads, max_blocks_per_seq, max_context_len,
                   partition_size, work_items, num_items, workspace, workspace_bytes, *desc);
  if (st != PK_OK) return st;
  p.q_offsets = q_offsets;
  p.tree_mask = tree_mask;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (desc->dtype == PK_F32)
    return desc->head_dim == 128 ? run<float, 128>(p, s) : run<float, 64>(p, s);
  return desc->head_dim == 128 ? run<__nv_bfloat16, 128>(p, s) : run<__nv_bfloat16, 64>(p, s);
}

}  // extern "C"

}  // namespace pk
