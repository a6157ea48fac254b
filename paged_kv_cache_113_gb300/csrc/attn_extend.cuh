// Attention of new tokens with changed scores (pk_paged_attention_extend): what
// its kernels share.
//
// Row r of a (sequence, KV head) is token i = r / G of the sequence's n new ones and
// query head kvh G + r % G, at position pos = ctx - n + i. It sees the tokens of one
// interval [lo, hi): hi = max(pos + 1, min(prefix, ctx)), lo the largest of 0, its
// document's first token and pos - window + 1. Its scores, in the exponent's scale
// (base 2): x = scale <q, k>; x = cap tanh(x / cap); x -= slope |pos - t|.
//
// A split call cuts every sequence's tokens at multiples of `partition`. A row whose
// interval lies in one partition gets its result from there; another's states are
// merged over the partitions that its interval meets, and every one of them has been
// visited by the row's unit. So no list of what was written is needed.
#pragma once

#include "attn_split.cuh"

namespace pk {
namespace {

struct ExtendParams : RowsParams {
  const float *slopes;          // [Hq] or null
  const int32_t *prefix_lens;   // [S] or null
  const int32_t *first_tokens;  // [num_rows] or null
  int32_t window;               // 0: none
  float factor;                 // of a product: scale log2(e), or scale / cap
  float cap_log2;               // cap log2(e), 0: none
  int32_t tiles;                // units of a KV head and partition without a list
};

// For |y| <= kTanhSmall tanh(y) = y (c0 + c1 y^2 + .. + c4 y^8) to 2^-20.6 of itself: like
// extend_prompt.cuh's shorter one, the polynomial of least largest relative error, by linear
// programming over 2000 points.
constexpr float kTanhSmall = 0.75f;
constexpr float kTanh0 = 0.999999463558197f, kTanh1 = -0.3332850933074951f, kTanh2 = 0.13261185586452484f,
                kTanh3 = -0.05011745169758797f, kTanh4 = 0.012983138673007488f;

struct RowSpan {
  int pos, lo, hi;  // position, and the tokens that the row sees (lo >= hi: none)
};

__device__ __forceinline__ RowSpan row_span(const ExtendParams &p, const SeqRows &sr, int s, int i) {
  RowSpan r;
  r.pos = sr.ctx - sr.n + i;
  r.hi = r.pos + 1;
  if (p.prefix_lens) r.hi = max(r.hi, min(__ldg(p.prefix_lens + s), sr.ctx));
  r.lo = p.window > 0 ? max(0, r.pos - p.window + 1) : 0;
  if (p.first_tokens) r.lo = max(r.lo, __ldg(p.first_tokens + sr.q0 + i));
  return r;
}

// Where the state of a row goes from partition `part`.
__device__ __forceinline__ Place row_place(const ExtendParams &p, int lo, int hi, int part) {
  if (p.num_partitions == 1) return Place::kOut;
  if (lo >= hi) return Place::kNowhere;  // the merge writes zeros
  const int first = lo / p.partition, last = (hi - 1) / p.partition;
  if (part < first || part > last) return Place::kNowhere;
  return first == last ? Place::kOut : Place::kWorkspace;
}

// Rows of a sequence, 0 where its offsets are no range of the query rows.
__device__ __forceinline__ int query_len(const ExtendParams &p, int s) {
  if (!p.q_offsets) return 1;
  const int a = __ldg(p.q_offsets + s), b = __ldg(p.q_offsets + s + 1);
  return a < 0 || b < a || b > p.num_rows || b - a > p.max_draft ? 0 : b - a;
}

// The unit of CTA `cta`: KV heads fastest, then units, then partitions, units and
// partitions last first (the last rows of a prompt see most). All threads of a warp
// call. False: none.
__device__ __forceinline__ bool extend_unit(const ExtendParams &p, int cta, int R, bool first_thread, SplitUnit &u) {
  const int lane = threadIdx.x & 31;
  u.kvh = cta % p.num_kv_heads;
  const int y = cta / p.num_kv_heads;
  const bool record = u.kvh == 0 && first_thread;
  if (p.items) {  // (sequence, first row, rows, partition)
    const int4 item = __ldg(reinterpret_cast<const int4 *>(p.items) + y);
    if (item.y < 0 || item.z < 1 || item.z > R || !checked_item(p, y, item.x, item.w, false)) {
      if (record) record_error(&g_rows_error, PK_DEVERR_ORDER, y);
      return false;
    }
    u.s = item.x, u.r0 = item.y, u.rows = item.z, u.part = item.w;
  } else {
    int tile = p.tiles - 1 - y % p.tiles;
    u.part = p.num_partitions - 1 - y / p.tiles;
    u.rows = R;
    if (int64_t(p.max_draft) * p.group <= R) {  // a unit is a sequence
      u.s = tile, u.r0 = 0;
    } else {
      // Sequences' units one after the other: the one that unit `tile` belongs to.
      bool found = false;
      for (int s0 = 0; s0 < p.num_seqs && !found; s0 += 32) {
        const int s = s0 + lane;
        const int mine = s < p.num_seqs ? (query_len(p, s) * p.group + R - 1) / R : 0;
        int sum = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, sum, off);
          if (lane >= off) sum += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, tile < sum);
        if (past) {
          const int at = __ffs(past) - 1;
          u.s = s0 + at;
          u.r0 = (tile - __shfl_sync(0xffffffffu, sum - mine, at)) * R;
          found = true;
        } else {
          tile -= __shfl_sync(0xffffffffu, sum, 31);
        }
      }
      if (!found) {
        // There are fewer units than `tiles`, so the first CTAs come here: they look at
        // every sequence's entries, to record bad ones of sequences without units.
        if (y == 0 && record)
          for (int s = 0; s < p.num_seqs; ++s) seq_rows(p, s, true);
        return false;
      }
    }
  }
  u.sr = seq_rows(p, u.s, record);
  u.rows = int(min(int64_t(u.rows), int64_t(u.sr.n) * p.group - u.r0));
  if (u.rows <= 0) {
    // An item behind its sequence's rows (of a sequence whose offsets are bad that is recorded).
    if (p.items && record && (u.sr.n > 0 || __ldg(p.q_offsets + u.s) == __ldg(p.q_offsets + u.s + 1)))
      record_error(&g_rows_error, PK_DEVERR_ORDER, y);
    return false;
  }
  u.void_rows = u.sr.ctx == 0;  // of a split call, the merge writes them
  if (u.void_rows) return p.num_partitions == 1;
  return true;
}

// Narrows a unit's tokens to those that its rows see ([from, to) of them all) within
// its partition; false: none. Their beginning is a block's.
__device__ __forceinline__ bool extend_tokens(const ExtendParams &p, SplitUnit &u, int from, int to) {
  const int64_t p0 = int64_t(u.part) * p.partition;
  u.start = int(max(int64_t(from / p.block_size) * p.block_size, p0));
  u.end = int(min(int64_t(to), p0 + p.partition));
  return from < to && u.start < u.end;
}

struct ExtendView {
  using Params = ExtendParams;
  static constexpr bool SCORES = true;
  template <int R>
  struct Shared {
    int lo[R], hi[R], pos[R];
    float slope[R];
    int from, to, all_from, all_to;
  };
  int all_from, all_to;

  static __device__ __forceinline__ bool unit(const ExtendParams &p, int R, bool, SplitUnit &u) {
    return extend_unit(p, blockIdx.x, R, threadIdx.x == 0, u);
  }
  template <int R>
  __device__ __forceinline__ bool rows(const ExtendParams &p, SplitUnit &u, Shared<R> &sh) {
    static_assert(R <= 32, "one warp sets the rows up");
    if (threadIdx.x < 32) {
      const int r = threadIdx.x;
      RowSpan x{0, 0, 0};
      if (r < u.rows) x = row_span(p, u.sr, u.s, (u.r0 + r) / p.group);
      const bool some = x.lo < x.hi;
      if (r < R) {
        sh.lo[r] = x.lo, sh.hi[r] = x.hi, sh.pos[r] = x.pos;
        sh.slope[r] = p.slopes && r < u.rows
                          ? __ldg(p.slopes + u.kvh * p.group + (u.r0 + r) % p.group) * 1.44269504f
                          : 0.0f;
      }
      // A row that sees nothing leaves no token seen by all.
      const int from = __reduce_min_sync(0xffffffffu, some ? x.lo : INT32_MAX);
      const int to = __reduce_max_sync(0xffffffffu, some ? x.hi : 0);
      const int af = __reduce_max_sync(0xffffffffu, r >= u.rows ? 0 : (some ? x.lo : INT32_MAX));
      const int at = __reduce_min_sync(0xffffffffu, r >= u.rows ? INT32_MAX : (some ? x.hi : 0));
      if (r == 0) sh.from = from, sh.to = to, sh.all_from = af, sh.all_to = at;
    }
    __syncthreads();
    if (!extend_tokens(p, u, sh.from, sh.to)) {
      u.void_rows = p.num_partitions == 1;
      return u.void_rows;
    }
    all_from = max(u.start, min(sh.all_from, u.end)), all_to = min(sh.all_to, u.end);
    return true;
  }
  static __device__ __forceinline__ float factor(const ExtendParams &p) { return p.factor; }
  template <int R>
  static __device__ __forceinline__ float score(const ExtendParams &p, const Shared<R> &sh, int r, int t, float x) {
    if (p.cap_log2 != 0.0f) x = p.cap_log2 * tanhf(x);
    if (p.slopes) x = fmaf(-sh.slope[r], float(abs(sh.pos[r] - t)), x);
    return x;
  }
  template <int R>
  static __device__ __forceinline__ bool sees(const SplitUnit &u, const Shared<R> &sh, int r, int t) {
    return t >= sh.lo[r] && t < min(sh.hi[r], u.end);
  }
  template <int R>
  static __device__ __forceinline__ Place place(const ExtendParams &p, const SplitUnit &u, const Shared<R> &sh, int r) {
    return row_place(p, sh.lo[r], sh.hi[r], u.part);
  }
  template <int R>
  static __device__ __forceinline__ bool nonzero(const SplitUnit &, const Shared<R> &, int) {
    return false;  // no weight at all: zeros
  }
};

// Joins the states of rows whose interval meets several partitions, and writes zeros
// for rows that see nothing: M = max m, out = sum acc 2^(m - M) / sum l 2^(m - M). A
// warp has a row (token, query head) and finds its sequence by bisection, so that the
// grid is as large as the rows, however uneven the sequences.
template <typename IO, int D>
__global__ void __launch_bounds__(256) extend_merge_kernel(ExtendParams p) {
  constexpr int EPL = D / 32, U = 8;
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const bool some = row < int64_t(p.num_rows) * p.num_q_heads;
  const int tok = some ? int(row / p.num_q_heads) : 0;
  int s = tok;
  if (p.q_offsets) {  // the last sequence that begins at or before the row
    int a = 0, b = p.num_seqs;
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (__ldg(p.q_offsets + mid) <= tok) a = mid;
      else b = mid;
    }
    s = a;
  }
  RowSpan x{0, 0, 0};
  int first = 0, last = -1;
  bool mine = some && s < p.num_seqs;
  if (mine) {
    const SeqRows sr = seq_rows(p, s, false);
    mine = tok >= sr.q0 && tok < sr.q0 + sr.n;
    if (mine && sr.ctx > 0) x = row_span(p, sr, s, tok - sr.q0);
    if (x.lo < x.hi) {
      first = x.lo / p.partition, last = (x.hi - 1) / p.partition;
      mine = first != last;
    }
  }
  // Every warp waits for the attention, those with nothing to do too: what comes after this
  // grid on the stream or in a graph waits for it alone, and the attention has written the rows
  // that lie in one partition to `out` itself.
  wait_prerequisites();
  if (!mine) return;
  float M = -INFINITY, L = 0.0f, acc[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.0f;
  for (int q0 = first; q0 <= last; q0 += U) {
    float m[U], l[U], v[U][EPL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // Past the end the last one again, at a factor of 0.
      const size_t q = size_t(row) * p.num_partitions + min(q0 + u, last);
      m[u] = q0 + u <= last ? __ldcg(p.ws_m + q) : -INFINITY;
      l[u] = q0 + u <= last ? __ldcg(p.ws_l + q) : 0.0f;
      const float *src = p.ws_acc + q * D + lane * EPL;
      if (EPL == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4 *>(src));
        v[u][0] = y.x, v[u][1] = y.y, v[u][EPL - 2] = y.z, v[u][EPL - 1] = y.w;
      } else {
        const float2 y = __ldcg(reinterpret_cast<const float2 *>(src));
        v[u][0] = y.x, v[u][1] = y.y;
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, m[u]);
    const float ref = top == -INFINITY ? 0.0f : top, f = exp2f(M - ref);
    M = top;
    L *= f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = merge_add(0.0f, acc[e], f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = exp2f(m[u] - ref);
      L = fmaf(l[u], w, L);
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = merge_add(acc[e], v[u][e], w);
    }
  }
  const float inv = 1.0f / denominator(L, false);
#pragma unroll
  for (int e = 0; e < EPL; ++e)
    store_elem(static_cast<IO *>(p.out) + size_t(row) * D + lane * EPL + e, acc[e] * inv);
}

}  // namespace
}  // namespace pk
