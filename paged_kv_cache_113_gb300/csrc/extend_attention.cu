// Attention of each sequence's new tokens over its paged context, with changed scores
// (pk_paged_attention_extend): a prompt, a chunk of one, or one decoded token.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <new>
#include <tuple>
#include <vector>

#include "attn_extend.cuh"
#include "extend_prompt.cuh"
#include "extend_few.cuh"
#include "pagedkv.h"

namespace pk {

extern "C" int *pkx_extend_attention_error_word() { return error_word(g_rows_error); }

namespace {

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
    return n;
  cudaGetLastError();  // clear a failed query on a machine without a GPU
  return 152;
}

// The kernel of sequences of at most `rows` rows, and the rows of its units.
enum class Path { kFew, kPrompt, kSplit };
Path path_of(const pk_cache_desc &d, int64_t rows) {
  if (d.dtype != PK_BF16 || (d.block_size != 8 && d.block_size != 16 && d.block_size != 32)) return Path::kSplit;
  return rows <= kFewRows ? Path::kFew : Path::kPrompt;
}
int unit_rows(const pk_cache_desc &d, int64_t rows) {
  switch (path_of(d, rows)) {
    case Path::kFew: return kFewRows;
    case Path::kPrompt: return kPromptRows;
    default: return split_rows(int(std::min<int64_t>(rows, 64)));
  }
}

template <typename T, int D>
pk_status launch_extend_merge(const ExtendParams &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(p.num_rows) * p.num_q_heads + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, extend_merge_kernel<T, D>, p) == cudaSuccess) return PK_OK;
  cudaGetLastError();
  extend_merge_kernel<T, D><<<cfg.gridDim, cfg.blockDim, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

template <typename T, int D>
pk_status run(ExtendParams p, const pk_cache_desc &d, cudaStream_t stream) {
  const int64_t rows = int64_t(p.max_draft) * p.group;
  const int R = unit_rows(d, rows);
  const int64_t tiles = rows <= R ? p.num_seqs
                                  : (int64_t(p.num_rows) * p.group + R - 1) / R + p.num_seqs;
  const int64_t units = (p.items ? p.num_items : tiles * p.num_partitions) * int64_t(p.num_kv_heads);
  if (units > INT32_MAX) return PK_ERR_UNSUPPORTED;
  p.tiles = int32_t(tiles);
  const dim3 grid = dim3(unsigned(units));
  pk_status st;
  const Path path = path_of(d, rows);
  if (path == Path::kPrompt) {
    st = launch_prompt<D>(p, d, unsigned(units), stream);
  } else if (path == Path::kFew) {
    st = launch_few<D>(p, d, unsigned(units), stream);
  } else {
    switch (R) {
      case 8: st = launch_split<T, D, 1, ExtendView>(p, grid, stream); break;
      case 16: st = launch_split<T, D, 2, ExtendView>(p, grid, stream); break;
      default: st = launch_split<T, D, 4, ExtendView>(p, grid, stream);
    }
  }
  if (st != PK_OK || p.num_partitions == 1) return st;
  return launch_extend_merge<T, D>(p, stream);
}

pk_status check_extend(const pk_cache_desc *d, int32_t num_q_heads, int32_t max_context_len,
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

// Whether a cap and what it makes of the scale are numbers that the kernels can work with: far
// enough from fp32's ends that their products with queries, in parts too, are normal numbers.
bool cap_fits(float softcap, float scale) {
  if (softcap == 0.0f) return true;
  constexpr double least = 0x1p-100, most = 0x1p100;
  const double c = softcap, f = std::fabs(double(scale)) / c;
  return c >= least && c <= most && (f == 0.0 || (f >= least && f <= most));
}

// Units of work without a split: the tokens that a unit's rows see between them (a
// prefix or documents are not known here), and the first of them.
struct Tile {
  int32_t s, r0, rows, lo, hi, ctx;
};
void tiles_of(const int32_t *lens, const int32_t *query_lens, int32_t num_seqs, int group, int32_t window,
              int R, std::vector<Tile> &out) {
  for (int32_t s = 0; s < num_seqs; ++s) {
    const int64_t n = query_lens ? query_lens[s] : 1, c = std::max<int64_t>(lens[s], n), rows = n * group;
    for (int64_t r0 = 0; r0 < rows; r0 += R) {
      const int64_t k = std::min<int64_t>(R, rows - r0), first = c - n + r0 / group;
      const int64_t lo = window > 0 ? std::max<int64_t>(0, first - window + 1) : 0;
      out.push_back(Tile{s, int32_t(r0), int32_t(k), int32_t(lo), int32_t(c - n + (r0 + k - 1) / group + 1),
                         int32_t(c)});
    }
  }
}

// The partition size that the planner chooses (0: none). Units go longest first to the CTA
// that is free first, so a launch lasts about as long as its longest unit or as the mean
// share of a CTA with what the last round leaves idle (of the shortest units' length),
// whichever is more; a unit costs `extra` tokens more than its own, each part of a row that
// is split d + 2 floats, written and read, and the merge a launch.
int32_t choose_partition(const std::vector<Tile> &tiles, const pk_cache_desc &d, Path path) {
  int64_t longest = 0;
  for (const Tile &t : tiles) longest = std::max<int64_t>(longest, t.hi - t.lo);
  if (longest <= 1024) return 0;
  // CTAs at once, the time of a token of one, and a unit's own cost in tokens.
  const int64_t slots = int64_t(sm_count()) * (path == Path::kPrompt ? 1 : (path == Path::kFew ? 3 : 2));
  const double token = path == Path::kPrompt ? 10e-9 : (path == Path::kFew ? 35e-9 : 22e-9);
  const double extra = path == Path::kPrompt ? 400 : 128;
  constexpr int64_t kBin = 128;
  std::vector<int64_t> count;  // parts by length
  int32_t best = 0;
  double least = 0;
  for (int c = 1; c <= 32; ++c) {
    int64_t n = ((longest + c - 1) / c + kBin - 1) / kBin * kBin;
    n = (n + d.block_size - 1) / d.block_size * d.block_size;
    if (c > 1 && n < 512) break;
    count.assign(size_t(std::max(n, longest) / kBin + 2), 0);
    double work = 0, partials = 0;
    int64_t units = 0, most = 0;
    for (const Tile &t : tiles) {
      const int64_t first = c == 1 ? 0 : t.lo / n, last = c == 1 ? 0 : (t.hi - 1) / n;
      for (int64_t q = first; q <= last; ++q) {
        const int64_t len = c == 1 ? t.hi - t.lo
                                   : std::min<int64_t>(t.hi, (q + 1) * n) - std::max<int64_t>(t.lo, q * n);
        ++count[size_t((len + kBin - 1) / kBin)];
        work += double(len) + extra;
        most = std::max(most, len);
      }
      units += last - first + 1;
      if (last > first) partials += double(last - first + 1) * t.rows;
    }
    units *= d.num_kv_heads;
    work *= d.num_kv_heads;
    int64_t tail = 0;  // the longest of the last `slots` units
    for (int64_t left = std::min(units, slots); left > 0 && tail + 1 < int64_t(count.size()); ++tail)
      left -= count[size_t(tail)] * d.num_kv_heads;
    const double idle = double((slots - units % slots) % slots) / double(slots) * (double(tail * kBin) + extra);
    const double merge = partials * d.num_kv_heads * (d.head_dim + 2) * 8 / 6e12 / token;
    const double cost = merge + (c > 1 ? 5e-6 / token : 0) +
                        std::max(double(most) + extra, work / double(slots) + idle);
    if (c == 1 || cost < (best ? 0.97 : 0.92) * least) least = cost, best = c == 1 ? 0 : int32_t(n);
  }
  return best;
}

}  // namespace

extern "C" {

size_t pk_extend_workspace_size(int32_t num_q_tokens, int32_t num_q_heads, int32_t max_context_len,
                                int32_t partition_size, const pk_cache_desc *desc) {
  if (num_q_tokens < 0 || check_extend(desc, num_q_heads, max_context_len, partition_size) != PK_OK ||
      partition_size == 0)
    return 0;
  const int64_t P = (int64_t(max_context_len) + partition_size - 1) / partition_size;
  if (P <= 1) return 0;
  return size_t(num_q_tokens) * num_q_heads * size_t(P) * (size_t(desc->head_dim) + 2) * sizeof(float);
}

pk_status pk_extend_plan(const int32_t *context_lens, const int32_t *query_lens, int32_t num_seqs,
                         int32_t max_query_len, int32_t num_q_heads, int32_t window, int32_t partition_size,
                         const pk_cache_desc *desc, int32_t *partition_out, int32_t *items_out, int32_t cap,
                         int32_t *num_items_out) {
  if (!partition_out || !num_items_out || num_seqs <= 0 || !context_lens || max_query_len < 1 || window < 0 ||
      partition_size < -1 || cap < 0)
    return PK_ERR_INVALID_ARG;
  *partition_out = 0;
  *num_items_out = 0;
  int32_t longest = 1;
  for (int32_t s = 0; s < num_seqs; ++s) {
    const int32_t n = query_lens ? query_lens[s] : 1;
    if (n < 0 || n > max_query_len) return PK_ERR_INVALID_ARG;
    longest = std::max(longest, std::max(context_lens[s], n));
  }
  const pk_status st = check_extend(desc, num_q_heads, longest, std::max(partition_size, 0));
  if (st != PK_OK) return st;
  const int group = num_q_heads / desc->num_kv_heads;
  const int R = unit_rows(*desc, int64_t(max_query_len) * group);
  try {
    std::vector<Tile> tiles;
    tiles_of(context_lens, query_lens, num_seqs, group, window, R, tiles);
    int32_t part = partition_size > 0 && partition_size < longest ? partition_size : 0;
    if (partition_size == -1) part = choose_partition(tiles, *desc, path_of(*desc, int64_t(max_query_len) * group));
    // Every partition that a row of the unit may see: a prefix lets it see all of the
    // context. Those of expected work first, longest first.
    std::vector<std::tuple<int64_t, int64_t, int32_t, int32_t>> order;  // -length, -context, tile, partition
    for (size_t i = 0; i < tiles.size(); ++i) {
      const Tile &t = tiles[i];
      const int32_t first = part ? t.lo / part : 0, last = part ? (t.ctx - 1) / part : 0;
      for (int32_t q = first; q <= last; ++q) {
        const int64_t a = part ? std::max<int64_t>(t.lo, int64_t(q) * part) : t.lo;
        const int64_t b = part ? std::min<int64_t>(t.hi, int64_t(q + 1) * part) : t.hi;
        order.emplace_back(-std::max<int64_t>(b - a, 0), -int64_t(t.ctx), int32_t(i), q);
      }
    }
    std::sort(order.begin(), order.end());
    if (order.size() > size_t(INT32_MAX) / 4) return PK_ERR_UNSUPPORTED;
    *partition_out = part;
    *num_items_out = int32_t(order.size());
    if (int64_t(order.size()) > cap || (!items_out && !order.empty())) return PK_ERR_INVALID_ARG;
    for (size_t k = 0; k < order.size(); ++k) {
      const Tile &t = tiles[size_t(std::get<2>(order[k]))];
      int32_t *item = items_out + 4 * k;
      item[0] = t.s, item[1] = t.r0, item[2] = t.rows, item[3] = std::get<3>(order[k]);
    }
  } catch (const std::bad_alloc &) {
    return PK_ERR_NOMEM;
  }
  return PK_OK;
}

pk_status pk_paged_attention_extend(void *out, const void *q, const void *k_cache, const void *v_cache,
                                    const int32_t *block_tables, const int32_t *context_lens,
                                    const int32_t *q_offsets, float scale, const pk_score_desc *scores,
                                    int32_t num_seqs, int32_t num_q_tokens, int32_t max_query_len,
                                    int32_t num_q_heads, int32_t max_blocks_per_seq, int32_t max_context_len,
                                    int32_t partition_size, const int32_t *work_items, int32_t num_items,
                                    void *workspace, size_t workspace_bytes, const pk_cache_desc *desc,
                                    void *stream) {
  pk_status st = check_extend(desc, num_q_heads, max_context_len, partition_size);
  if (st != PK_OK) return st;
  if (num_seqs < 0 || num_q_tokens < 0 || max_query_len < 0 || num_items < 0) return PK_ERR_INVALID_ARG;
  if (scores && (!cap_fits(scores->softcap, scale) || scores->window < 0)) return PK_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_q_tokens == 0 || max_query_len == 0) return PK_OK;
  if (!q_offsets && (num_q_tokens < num_seqs || max_query_len != 1)) return PK_ERR_INVALID_ARG;
  if (work_items ? (num_items == 0 || !aligned16(work_items)) : num_items != 0) return PK_ERR_INVALID_ARG;
  if (int64_t(num_q_tokens) * num_q_heads > INT32_MAX) return PK_ERR_UNSUPPORTED;
  ExtendParams p{};
  st = rows_params(p, out, q, k_cache, v_cache, block_tables, context_lens, scale, num_seqs, num_q_tokens,
                   max_query_len, num_q_heads, max_blocks_per_seq, max_context_len, partition_size, nullptr, 0,
                   workspace, workspace_bytes, *desc);
  if (st != PK_OK) return st;
  p.q_offsets = q_offsets;
  p.items = work_items;
  p.num_items = num_items;
  p.factor = p.scale_log2;
  if (scores) {
    p.slopes = scores->slopes;
    p.prefix_lens = scores->prefix_lens;
    p.first_tokens = scores->first_tokens;
    p.window = scores->window;
    if (scores->softcap > 0.0f) {
      p.factor = float(double(scale) / double(scores->softcap));
      p.cap_log2 = float(double(scores->softcap) * 1.4426950408889634);
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (desc->dtype == PK_F32)
    return desc->head_dim == 128 ? run<float, 128>(p, *desc, s) : run<float, 64>(p, *desc, s);
  return desc->head_dim == 128 ? run<__nv_bfloat16, 128>(p, *desc, s) : run<__nv_bfloat16, 64>(p, *desc, s);
}

}  // extern "C"

}  // namespace pk
