// Shared by the attention kernels over 8-bit caches and over drafted tokens:
// the launch parameters, a sequence's place in the batch, and the log-sum-exp
// merge of split rows.
//
// A sequence s has n_s query tokens (1 without q_offsets), the last n_s of its
// context. With base = ctx - n_s, query i of it sees every token t < base and
// the token base + j where bit j of its mask is set (a chain without masks:
// j <= i). Per KV head the sequence is n_s * G rows of query, row r being token
// r / G, query head kvh * G + r % G.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pagedkv.h"
#include "pk_device.cuh"

namespace pk {
namespace {

// The device error word of the including translation unit.
__device__ int g_rows_error;

struct RowsParams {
  void *out;                  // [num_rows, Hq, D]
  const void *q;              // [num_rows, Hq, D]
  const void *k_cache, *v_cache;  // [N, B, Hk, D]
  const uint8_t *kv_exp;      // [N, Hk, B, 2] (8-bit caches)
  const int32_t *tables;      // [S, max_blocks]
  const int32_t *ctx_lens;    // [S]
  const int32_t *q_offsets;   // [S + 1], or null: row s is sequence s's only query
  const uint64_t *tree_mask;  // [num_rows], or null: a chain
  float *ws_acc, *ws_m, *ws_l;  // split-K partials [num_rows, Hq, P, D], [.., P], [.., P]
  const int32_t *items;       // [num_items][2] (sequence, partition), or null
  float scale_log2;           // scale * log2(e)
  int32_t num_seqs, num_rows, max_draft, num_q_heads, num_kv_heads, group;
  int32_t block_size, max_blocks, num_blocks;
  int32_t partition, num_partitions, num_items;
  int32_t max_context;        // the longest context that the call allows and a table holds
  int32_t row_tiles;          // CTAs that share a (sequence, KV head)'s rows
};

struct SeqRows {
  int q0, n;     // query rows q0 .. q0 + n - 1 (n = 0: nothing to do)
  int ctx;       // context length (0: the rows are zero)
  int np;        // partitions with tokens
};

// Sequence s's context length c, n of its tokens being queries: clamped to
// max_context, 0 where c is below n; either is recorded when asked.
__device__ __forceinline__ int checked_context(const RowsParams &p, int s, int n, int c, bool record) {
  const int cap = p.max_context;
  if (c >= n && c <= cap) return c;
  if (record) record_error(&g_rows_error, PK_DEVERR_CONTEXT, s);
  return c < n || cap < n ? 0 : cap;
}

// Partitions with tokens of a context of c.
__device__ __forceinline__ int partitions_of(const RowsParams &p, int c) {
  return int((int64_t(c) + p.partition - 1) / p.partition);
}

// Sequence s's rows and length, checked; bad entries are recorded when asked.
__device__ __forceinline__ SeqRows seq_rows(const RowsParams &p, int s, bool record) {
  SeqRows r{s, 1, 0, 0};
  if (p.q_offsets) {
    const int a = __ldg(p.q_offsets + s), b = __ldg(p.q_offsets + s + 1);
    if (a < 0 || b < a || b > p.num_rows || b - a > p.max_draft) {
      if (record) record_error(&g_rows_error, PK_DEVERR_OFFSETS, s);
      r.n = 0;
      return r;
    }
    r.q0 = a;
    r.n = b - a;
    if (r.n == 0) return r;
  }
  r.ctx = checked_context(p, s, r.n, __ldg(p.ctx_lens + s), record);
  r.np = partitions_of(p, r.ctx);
  return r;
}

// The (sequence, partition) of work y: an item of the list, or the grid's.
__device__ __forceinline__ bool checked_item(const RowsParams &p, int y, int s, int part, bool record) {
  if (s >= 0 && s < p.num_seqs && part >= 0 && part < p.num_partitions) return true;
  if (record) record_error(&g_rows_error, PK_DEVERR_ORDER, y);
  return false;
}
__device__ __forceinline__ bool work_item(const RowsParams &p, int y, int z, bool record,
                                          int &s, int &part) {
  s = p.items ? __ldg(p.items + 2 * y) : y;
  part = p.items ? __ldg(p.items + 2 * y + 1) : z;
  return checked_item(p, y, s, part, record);
}

// Which drafted tokens row q0 + i of a sequence of n sees, one bit each.
__device__ __forceinline__ uint64_t draft_mask(const RowsParams &p, int q0, int i, int n) {
  const uint64_t all = n >= 64 ? ~0ull : (1ull << n) - 1;
  if (p.tree_mask) return __ldg(reinterpret_cast<const unsigned long long *>(p.tree_mask) + q0 + i) & all;
  return i >= 63 ? all : ((2ull << i) - 1) & all;
}

// Which of the 64 tokens t0 .. t0 + 63 a row sees: those before base, and the
// drafted ones of its mask (bits past the last draft are clear).
__device__ __forceinline__ uint64_t see64(uint64_t mask, int base, int t0) {
  const int cut = base - t0;  // tokens of these that everyone sees
  if (cut >= 64) return ~0ull;
  if (cut <= -64) return 0;
  if (cut >= 0) return (mask << cut) | ((1ull << cut) - 1);
  return mask >> -cut;
}

// The m of a state as it is kept for a merge: maxima leave NaN out, sums do not.
__device__ __forceinline__ float merge_max(float m, float l) { return l == l ? m : l; }

// What a row's accumulator is divided by. A sum of 0 is a row that sees nothing (its
// result is 0), or one that sees scores of -inf alone (NaN).
__device__ __forceinline__ float denominator(float l, bool sees) {
  return l != 0.0f ? l : (sees ? __uint_as_float(0x7fc00000u) : INFINITY);
}

// sum + x f for a state's factor f; with f 0 only what is not finite counts.
__device__ __forceinline__ float merge_add(float sum, float x, float f) {
  return f != 0.0f ? fmaf(x, f, sum) : (fabsf(x) <= 3.402823466e38f ? sum : sum + x);
}

// Four consecutive elements as fp32 values.
template <typename T>
__device__ __forceinline__ float4 load4(const T *p) {
  return widen4(raw4(p));
}
// ---------------------------------------------------------------------------
// Merge of split rows: M = max_q m_q, out = sum_q acc_q 2^(m_q - M) /
// sum_q l_q 2^(m_q - M). What is not finite survives it: a state whose sum is NaN
// (a NaN score, which no maximum shows) has NaN for its m, so that its factor is
// NaN, and an infinite or NaN acc counts even where its factor is 0. A row (grid.y = sequence, so that it needs no search
// for its sequence) gets wpr warps, enough that a warp merges at most eight
// partials, all loaded at once; the row's first warp joins the warps' states.
// ---------------------------------------------------------------------------
template <typename IO, int D>
__global__ void __launch_bounds__(256) rows_merge_kernel(RowsParams p, int wpr) {
  constexpr int EPL = D / 32, U = 8;
  __shared__ float sm_acc[8][D], sm_m[8], sm_l[8];
  const int s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqRows sr = seq_rows(p, s, false);
  const int row = blockIdx.x * (8 / wpr) + warp / wpr, sub = warp % wpr;  // row: token * Hq + head
  wait_prerequisites();
  const bool live = row < sr.n * p.num_q_heads && sr.np > 1;
  const size_t at = size_t(sr.q0) * p.num_q_heads + row;
  const int chunk = (sr.np + wpr - 1) / wpr;
  const int q_end = live ? min(sr.np, (sub + 1) * chunk) : 0;
  float M, L, acc[EPL];
  // Whether a result is not finite although its sum is: then the states are joined
  // again with care for what a factor of 0 would hide (see merge_add), which costs
  // registers and a fifth of the time in a loop that has it for every state.
  auto odd = [&] {
    float o = 0.0f;  // NaN once an element is not finite
#pragma unroll
    for (int e = 0; e < EPL; ++e) o = fmaf(acc[e], 0.0f, o);
    return __any_sync(0xffffffffu, o != 0.0f) && fabsf(L) <= 3.402823466e38f;
  };
  auto partitions = [&](auto care) {
    constexpr bool CARE = decltype(care)::value;
    M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.0f;
    for (int q0 = sub * chunk; q0 < q_end; q0 += U) {
      float m[U], l[U], x[U][EPL];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const size_t q = at * p.num_partitions + min(q0 + u, q_end - 1);
        // Past the end the last one again, at a factor of 0: what is not finite in it
        // counts already.
        m[u] = q0 + u < q_end ? __ldcg(p.ws_m + q) : -INFINITY;
        l[u] = __ldcg(p.ws_l + q);
        const float *src = p.ws_acc + q * D + lane * EPL;
        if (EPL == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
          x[u][0] = v.x, x[u][1] = v.y, x[u][EPL - 2] = v.z, x[u][EPL - 1] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
          x[u][0] = v.x, x[u][1] = v.y;
        }
      }
      float top = M;
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, m[u]);
      const float ref = top == -INFINITY ? 0.0f : top, f = exp2f(M - ref);
      M = top;
      L *= f;  // NaN stays
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = CARE ? merge_add(0.0f, acc[e], f) : acc[e] * f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = exp2f(m[u] - ref);
        L = fmaf(l[u], w, L);
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] = CARE ? merge_add(acc[e], x[u][e], w) : fmaf(x[u][e], w, acc[e]);
      }
    }
  };
  partitions(std::false_type());
  if (odd()) partitions(std::true_type());
  if (wpr > 1) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) sm_acc[warp][lane * EPL + e] = acc[e];
    if (lane == 0) sm_m[warp] = merge_max(M, L), sm_l[warp] = L;
    __syncthreads();
    if (sub != 0) return;
    for (int w = 1; w < wpr; ++w) M = fmaxf(M, sm_m[warp + w]);
    const float ref = M == -INFINITY ? 0.0f : M;
    auto warps = [&](auto care) {
      L = 0.0f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = 0.0f;
      for (int w = 0; w < wpr; ++w) {
        const float f = exp2f(sm_m[warp + w] - ref);
        L = fmaf(sm_l[warp + w], f, L);
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
          const float x = sm_acc[warp + w][lane * EPL + e];
          acc[e] = decltype(care)::value ? merge_add(acc[e], x, f) : fmaf(x, f, acc[e]);
        }
      }
    };
    warps(std::false_type());
    if (odd()) warps(std::true_type());
  }
  if (!live) return;
  const float inv = 1.0f / denominator(L, sr.ctx > sr.n || draft_mask(p, sr.q0, row / p.num_q_heads, sr.n) != 0);
#pragma unroll
  for (int e = 0; e < EPL; ++e)
    store_elem(static_cast<IO *>(p.out) + at * D + lane * EPL + e, acc[e] * inv);
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Host: the checks and parameters that both attentions share, from the call's
// arguments. `part` is the resolved partition size (0: no split).
inline pk_status rows_params(RowsParams &p, void *out, const void *q, const void *k_cache,
                             const void *v_cache, const int32_t *block_tables,
                             const int32_t *context_lens, float scale, int32_t num_seqs,
                             int32_t num_rows, int32_t max_draft, int32_t num_q_heads,
                             int32_t max_blocks_per_seq, int32_t max_context_len, int32_t part,
                             const int32_t *items, int32_t num_items, void *workspace,
                             size_t workspace_bytes, const pk_cache_desc &d) {
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || max_blocks_per_seq <= 0)
    return PK_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PK_ERR_INVALID_ARG;
  if (!(scale == scale)) return PK_ERR_INVALID_ARG;
  if (int64_t(max_blocks_per_seq) * d.block_size > INT32_MAX) return PK_ERR_UNSUPPORTED;
  const int64_t P = part > 0 ? (int64_t(max_context_len) + part - 1) / part : 1;
  if (num_seqs > 65535 || P > 65535) return PK_ERR_UNSUPPORTED;
  if (items ? (num_items <= 0 || num_items > 65535) : num_items != 0) return PK_ERR_UNSUPPORTED;
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.tables = block_tables;
  p.ctx_lens = context_lens;
  p.items = items;
  p.num_items = num_items;
  p.scale_log2 = float(double(scale) * 1.4426950408889634);
  p.num_seqs = num_seqs;
  p.num_rows = num_rows;
  p.max_draft = max_draft;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = d.num_kv_heads;
  p.group = num_q_heads / d.num_kv_heads;
  p.block_size = d.block_size;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = d.num_blocks;
  p.partition = P > 1 ? part : max_blocks_per_seq * d.block_size;
  p.num_partitions = int32_t(P);
  p.max_context = std::min(max_context_len, max_blocks_per_seq * d.block_size);
  p.row_tiles = 1;
  if (workspace && !aligned16(workspace)) return PK_ERR_WORKSPACE;
  if (P > 1) {
    const size_t slots = size_t(num_rows) * num_q_heads * size_t(P);
    if (!workspace || workspace_bytes < slots * (size_t(d.head_dim) + 2) * sizeof(float))
      return PK_ERR_WORKSPACE;
    p.ws_acc = static_cast<float *>(workspace);
    p.ws_m = p.ws_acc + slots * d.head_dim;
    p.ws_l = p.ws_m + slots;
  }
  return PK_OK;
}

inline dim3 rows_grid(const RowsParams &p) {
  return dim3(unsigned(p.num_kv_heads * p.row_tiles), unsigned(p.items ? p.num_items : p.num_seqs),
              unsigned(p.items ? 1 : p.num_partitions));
}

// Opts a kernel into its dynamic shared memory, once per device (the attribute
// belongs to the device that is current).
template <typename Kernel>
bool smem_ready(Kernel kern, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return false;
  if (dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

// The merge, as the attention's programmatic dependent (an ordinary launch
// where that is refused).
template <typename IO, int D>
pk_status launch_rows_merge(const RowsParams &p, cudaStream_t stream) {
  int wpr = 1;
  while (wpr < 8 && wpr * 8 < p.num_partitions) wpr *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(p.max_draft) * p.num_q_heads + 8 / wpr - 1) / (8 / wpr)),
                     unsigned(p.num_seqs));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, rows_merge_kernel<IO, D>, p, wpr) == cudaSuccess) return PK_OK;
  cudaGetLastError();
  rows_merge_kernel<IO, D><<<cfg.gridDim, cfg.blockDim, 0, stream>>>(p, wpr);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // namespace
}  // namespace pk
