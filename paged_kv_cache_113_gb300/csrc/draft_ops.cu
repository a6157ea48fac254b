// What follows the attention of drafted tokens: which drafts are kept, by the target's
// probabilities and given random numbers (pk_verify_drafts), and their keys and values
// moved together in the cache (pk_compact_drafts).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pagedkv.h"
#include "pk_device.cuh"

namespace pk {

__device__ int g_draft_ops_error;

extern "C" int *pkx_draft_ops_error_word() { return error_word(g_draft_ops_error); }

namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 512;
constexpr int kMaxCluster = 8;

struct VerifyParams {
  int32_t *num_accepted;   // [S]
  int32_t *accepted;       // [num_rows]
  int64_t *next_tokens;    // [S]
  const void *p, *q;       // [num_rows] rows of V probabilities, q or null
  int64_t p_stride, q_stride;
  const int64_t *tokens;   // [num_rows]
  const float *uniforms;   // [num_rows]
  const int32_t *q_offsets;
  const int32_t *parents;  // [num_rows] or null: a chain
  int32_t num_rows, max_rows, vocab;
};

// A probability as it counts: what is not a positive finite number is 0.
__device__ __forceinline__ float weight(float x) { return x > 0.0f && x <= 3.402823466e38f ? x : 0.0f; }

// A number in two floats, hi + lo: the error of each addition is kept (Knuth's two-sum). The sum
// of the errors is rounded itself, by more the longer it is not brought in order: of 32 768 values
// 2^-34 of their sum in bad cases. So a thread sums 64 values at a time and adds those sums, in
// order each time: 2^-44 at worst, 2^-47 as a rule. Sums, products and comparisons go this way
// because of 64-bit operations this chip does two a clock and SM (with those, and sums in one
// pass over each thread's part, 256 chains of 8 drafts took 59 us; now 30).
struct Pair {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float x, float err) {
    const float t = __fadd_rn(hi, x), b = __fsub_rn(t, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(x, b)), err));
    hi = t;
  }
  __device__ __forceinline__ void add(const Pair &x) { add(x.hi, x.lo); }
  // In order: lo is at most half a unit in hi's last place.
  __device__ __forceinline__ void settle() {
    const float t = __fadd_rn(hi, lo);
    lo = __fsub_rn(lo, __fsub_rn(t, hi));
    hi = t;
  }
  __device__ __forceinline__ void sub(const Pair &x) { add(-x.hi, -x.lo); }
  __device__ __forceinline__ Pair times(float f) const {
    const float h = __fmul_rn(hi, f);
    return Pair{h, __fmaf_rn(lo, f, __fmaf_rn(hi, f, -h))};
  }
  // (Of values that are close the difference of the upper parts is exact.)
  __device__ __forceinline__ bool above(const Pair &x) const {
    return __fadd_rn(__fsub_rn(hi, x.hi), __fsub_rn(lo, x.lo)) > 0.0f;
  }
  __device__ __forceinline__ Pair shuffled_xor(int off) const {
    return Pair{__shfl_xor_sync(0xffffffffu, hi, off), __shfl_xor_sync(0xffffffffu, lo, off)};
  }
  __device__ __forceinline__ Pair shuffled_up(int off) const {
    return Pair{__shfl_up_sync(0xffffffffu, hi, off), __shfl_up_sync(0xffffffffu, lo, off)};
  }
};

// The weights that the next token is drawn by, element by element.
template <typename T>
struct Weights {
  const T *p, *q;           // q: the refused draft's distribution, or null
  int vocab, shift;         // elements of p before a multiple of four
  bool aligned_q;           // q's multiples of four are p's
  const int64_t *refused;   // tokens that do not count
  uint64_t mine;            // those that are this thread's

  // Elements 4 g - shift ..  + 3 of a row; zeros outside it.
  __device__ __forceinline__ float4 raw(const T *row, bool aligned, int g) const {
    const int e0 = 4 * g - shift;
    if (aligned && e0 >= 0 && e0 + 4 <= vocab) return widen4(raw4(row + e0));
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = e0 + i >= 0 && e0 + i < vocab ? load_elem(row + e0 + i) : 0.0f;
    return make_float4(x[0], x[1], x[2], x[3]);
  }
  // Calls f(element, weight, its error (of the difference from q)) for the groups g, g + step,
  // .. below `end`, in order; false from f ends it. Four groups' loads are under way at once.
  template <typename F>
  __device__ __forceinline__ void each(int g, int end, int step, F f) const {
    constexpr int U = 4;
    for (; g < end; g += U * step) {
      float4 x[U], y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[u] = y[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (g + u * step < end) {
          x[u] = raw(p, true, g + u * step);
          if (q) y[u] = raw(q, aligned_q, g + u * step);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int e0 = 4 * (g + u * step) - shift;
        const float a4[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, b4[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a = weight(a4[i]), err = 0.0f;
          if (q) {
            const float b = -weight(b4[i]), t = __fadd_rn(a, b), c = __fsub_rn(t, a);
            err = t > 0.0f ? __fadd_rn(__fsub_rn(a, __fsub_rn(t, c)), __fsub_rn(b, c)) : 0.0f;
            a = t > 0.0f ? t : 0.0f;
          }
          for (uint64_t m = mine; m; m &= m - 1)
            if (refused[__ffsll(m) - 1] == e0 + i) a = 0.0f;
          if (!f(e0 + i, a, err)) return;
        }
      }
    }
  }
};

// A cluster has a sequence: every CTA walks down from its root (a few loads, all nodes'
// at once), then sums its share of the weights of the row where the walk ended; the
// totals go round, and the CTA that the drawn number falls into finds the token: which
// warp's part, which of sixteen parts of that, and there 128 elements at a time. Only that
// row (and with q the refused draft's) is read whole: a vocabulary of V values a sequence,
// two with q.
//
// Measured: 256 chains of 8 drafts, 2 x 32 000 fp32 values each (66 MB, 9.7 us at the rate of a
// copy) 30 us; 64 trees of 16, 128 000 values (33 MB) 30 us; 4 x 4 drafts 13 us, of which the
// three reads that the walk waits for, one after the other, are the most. Beyond those an
// element's eight operations and the two passes behind the first bound it, not memory (23% busy).
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_drafts_kernel(VerifyParams a) {
  constexpr int NT = kVerifyThreads, NW = NT / 32;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int s = blockIdx.x / C, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ Pair totals[2][kMaxCluster], warp_sum[NW], part_sum[NW];
  __shared__ float pc[PK_MAX_DRAFT], lim[PK_MAX_DRAFT], un[PK_MAX_DRAFT];
  __shared__ int parent[PK_MAX_DRAFT];
  __shared__ int64_t token[PK_MAX_DRAFT];
  __shared__ uint64_t sh_refused;
  __shared__ int sh_cur;

  const int r0 = __ldg(a.q_offsets + s), r1 = __ldg(a.q_offsets + s + 1);
  const int64_t len = int64_t(r1) - r0;
  if (r0 < 0 || len <= 0 || r1 > a.num_rows || len > a.max_rows) {
    if (rank == 0 && threadIdx.x == 0) {
      if (len != 0 || r0 < 0 || r1 > a.num_rows) record_error(&g_draft_ops_error, PK_DEVERR_OFFSETS, s);
      a.num_accepted[s] = 0;
      a.next_tokens[s] = -1;
    }
    return;  // the whole cluster does
  }
  // Another CTA's shared memory is written only once that CTA is known to run: all say so here,
  // and are waited for ahead of the first totals.
  cluster.barrier_arrive();
  const int n = int(len);
  const T *const p = static_cast<const T *>(a.p), *const q = static_cast<const T *>(a.q);
  if (warp == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h;
      if (i >= n) continue;
      int up = i == 0 ? -1 : (a.parents ? __ldg(a.parents + r0 + i) : i - 1);
      int64_t t = i == 0 ? 0 : __ldg(reinterpret_cast<const long long *>(a.tokens) + r0 + i);
      if (i > 0 && (up < 0 || up >= i || t < 0 || t >= a.vocab)) {  // never reached
        if (rank == 0) record_error(&g_draft_ops_error, PK_DEVERR_DRAFT, s);
        up = -1, t = 0;
      }
      parent[i] = up;
      token[i] = t;
      un[i] = __ldg(a.uniforms + r0 + i);
      pc[i] = up >= 0 ? weight(load_elem(p + (r0 + up) * a.p_stride + t)) : 0.0f;
      lim[i] = up >= 0 && q ? weight(load_elem(q + (r0 + i) * a.q_stride + t)) : 0.0f;
    }
    __syncwarp();
    // A node comes after its parent, so one pass over the nodes is the walk.
    int cur = 0;
    uint64_t refused = 0, path = 1;
    Pair mass{1.0f, 0.0f};  // what the refused siblings leave
    for (int j = 1; j < n; ++j) {
      if (parent[j] != cur) continue;
      float pj = pc[j];
      if (!q && refused) {  // the same token again has nothing left
        const int64_t t = token[j];
        const bool again = (((refused >> lane) & 1) && token[lane] == t) ||
                           (((refused >> (lane + 32)) & 1) && token[lane + 32] == t);
        if (__any_sync(0xffffffffu, again)) pj = 0.0f;
      }
      if (Pair{pj, 0.0f}.above((q ? Pair{lim[j], 0.0f} : mass).times(un[j]))) {
        cur = j;
        path |= 1ull << j;
        refused = 0;
        mass = Pair{1.0f, 0.0f};
      } else {
        refused |= 1ull << j;
        mass.sub(Pair{pj, 0.0f});
      }
    }
    if (lane == 0) sh_cur = cur, sh_refused = refused;
    if (rank == 0) {
      const int count = __popcll(path);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        if (i < n && ((path >> i) & 1)) a.accepted[r0 + __popcll(path & ((1ull << i) - 1))] = i;
        if (i < n && i >= count) a.accepted[r0 + i] = -1;
      }
      if (lane == 0) a.num_accepted[s] = count - 1;
    }
  }
  __syncthreads();
  const uint64_t refused = sh_refused;
  Weights<T> w;
  w.p = p + (r0 + sh_cur) * a.p_stride;
  w.vocab = a.vocab;
  w.shift = int(reinterpret_cast<uintptr_t>(w.p) / sizeof(T) & 3);
  w.refused = token;
  // This CTA's groups of four elements, a contiguous part of them for each warp.
  const int groups = (a.vocab + w.shift + 3) / 4, share = (groups + C - 1) / C;
  const int g0 = min(groups, rank * share), g1 = min(groups, g0 + share);
  auto part_of = [](int n) { return ((n + NW - 1) / NW + 31) / 32 * 32; };
  const int per = part_of(share);
  const float u = fminf(fmaxf(un[0], 0.0f), 1.0f - 5.9604645e-8f);
  // The sum of the weights of the groups [from, to), a warp's.
  bool plain = false;  // the refused drafts leave nothing, so the row itself counts
  auto own = [&](int from, int to) {  // which of the refused tokens are this lane's of them
    w.mine = 0;
    if (plain || q) return;
    for (uint64_t left = refused; left; left &= left - 1) {
      const int i = __ffsll(left) - 1, g = int(token[i] + w.shift) / 4;
      if (g >= from && g < to && ((g - from) & 31) == lane) w.mine |= 1ull << i;
    }
  };
  auto sum_of = [&](int from, int to) {
    own(from, to);
    Pair sum;
    for (int g = from; g < to; g += 32 * 16) {  // 64 values a lane
      Pair part;
      w.each(g + lane, min(g + 32 * 16, to), 32, [&](int, float x, float err) {
        part.add(x, err);
        return true;
      });
      sum.add(part);
      sum.settle();
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) sum.add(sum.shuffled_xor(off));
    sum.settle();
    return sum;
  };
  Pair total;
  for (;;) {
    w.q = !plain && q && refused ? q + (r0 + __ffsll(refused) - 1) * a.q_stride : nullptr;
    w.aligned_q = w.q && int(reinterpret_cast<uintptr_t>(w.q) / sizeof(T) & 3) == w.shift;
    const int from = min(g1, g0 + warp * per);
    const Pair sum = sum_of(from, min(g1, from + per));
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    if (!plain) cluster.barrier_wait();
    if (warp == 0) {
      Pair x = lane < NW ? warp_sum[lane] : Pair{};
#pragma unroll
      for (int off = 16; off; off >>= 1) x.add(x.shuffled_xor(off));
      x = Pair{__shfl_sync(0xffffffffu, x.hi, 0), __shfl_sync(0xffffffffu, x.lo, 0)};  // one order of addition
      if (lane < C) *cluster.map_shared_rank(&totals[plain][rank], lane) = x;
    }
    cluster.sync();
    total = Pair{};
    for (int c = 0; c < C; ++c) total.add(totals[plain][c]);
    if (total.hi > 0.0f || !refused || plain) break;
    plain = true;
  }
  if (!(total.hi > 0.0f)) {
    if (rank == 0 && threadIdx.x == 0) a.next_tokens[s] = -1;
    return;
  }
  // Which of n parts the target falls into: the first that ends past it; the last with
  // anything, should rounding leave none. The target becomes that part's.
  Pair target = total.times(u);
  auto part_at = [&](const Pair *sums, int n) {
    Pair end, begin;
    int last = 0;
    for (int c = 0; c < n; ++c) {
      const Pair x = sums[c], at = end;
      end.add(x);
      if (!(x.hi > 0.0f)) continue;
      last = c, begin = at;
      if (end.above(target)) break;
    }
    target.sub(begin);
    return last;
  };
  if (rank != part_at(totals[plain], C)) return;
  // Again within the warp's part that it falls into, cut into parts for all warps; then a
  // warp goes over what is left, 128 elements at a time.
  const int from = min(g1, g0 + part_at(warp_sum, NW) * per), to = min(g1, from + per), sub = part_of(per);
  const int b0 = min(to, from + warp * sub), b1 = min(to, b0 + sub);
  const Pair sum = sum_of(b0, b1);
  if (lane == 0) part_sum[warp] = sum;
  __syncthreads();
  if (warp != part_at(part_sum, NW)) return;
  int at = -1;
  Pair run;
  for (int base = b0; base < b1; base += 32) {
    Pair mine;
    int last = -1;
    w.each(base + lane, min(base + 32, b1), 32, [&](int e, float x, float err) {
      mine.add(x, err);
      if (x > 0.0f) last = e;
      return true;
    });
    Pair incl = mine;  // of the lanes up to this one
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const Pair x = incl.shuffled_up(off);
      if (lane >= off) incl.add(x);
    }
    incl.add(run);
    const uint32_t some = __ballot_sync(0xffffffffu, last >= 0);
    const uint32_t past = __ballot_sync(0xffffffffu, last >= 0 && incl.above(target));
    if (past) {
      if (lane == __ffs(past) - 1) {
        Pair x = incl;
        x.sub(mine);
        w.each(base + lane, min(base + 32, b1), 32, [&](int e, float y, float err) {
          if (!(y > 0.0f)) return true;
          x.add(y, err);
          last = e;
          return !x.above(target);
        });
        a.next_tokens[s] = last;
      }
      return;
    }
    if (some) at = __shfl_sync(0xffffffffu, last, 31 - __clz(some));
    run = Pair{__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)};
    run.settle();
  }
  if (lane == 0) a.next_tokens[s] = at;  // (the last with anything, should rounding leave none)
}

// A sequence's kept rows to the places behind one another: thread = 16 bytes of a
// token's row, which it moves for all of the kept ones, first to last. A row never
// comes from before the place it goes to, and places are filled in order, so no
// source is overwritten before it is read. Eight of a thread's rows are under way at once.
// Measured: 256 sequences that keep 8 of 16 drafts, 8 heads of 128 in bf16 (15 MB), 9 us, the
// host call's; cold on the device 8 us, four reads one after the other.
__global__ void __launch_bounds__(128)
    compact_drafts_kernel(uint4 *k_cache, uint4 *v_cache, const int32_t *__restrict__ tables, int32_t max_blocks,
                          const int32_t *__restrict__ lens, const int32_t *__restrict__ q_offsets,
                          const int32_t *__restrict__ accepted, const int32_t *__restrict__ num_accepted,
                          int32_t *lens_out, int32_t num_rows, int32_t max_rows, int32_t block_size,
                          int32_t num_blocks, int32_t row_vecs) {
  constexpr int U = 8;
  const int s = blockIdx.y, side = blockIdx.z;
  const bool record = blockIdx.x == 0 && side == 0;
  __shared__ int from[PK_MAX_DRAFT], to[PK_MAX_DRAFT];  // slots
  __shared__ int sh_moves;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int r0 = __ldg(q_offsets + s), r1 = __ldg(q_offsets + s + 1);
    const int64_t n64 = int64_t(r1) - r0;
    const int ctx = __ldg(lens + s);
    int moves = 0, len = ctx;
    if (r0 < 0 || n64 < 0 || r1 > num_rows || n64 > max_rows) {
      if (record && lane == 0) record_error(&g_draft_ops_error, PK_DEVERR_OFFSETS, s);
    } else if (n64 > 0) {
      const int n = int(n64), last = __ldg(num_accepted + s);
      const bool fits = ctx >= n && ctx <= int64_t(max_blocks) * block_size;
      int kept[2];
      bool good = last >= 0 && last < n;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = lane + 32 * h;
        kept[h] = k < n ? __ldg(accepted + r0 + k) : 0;
        if (k < n && k <= last) {  // ascending, within the rows
          const int prev = k > 0 ? __ldg(accepted + r0 + k - 1) : -1;
          good = good && kept[h] > prev && kept[h] < n && kept[h] >= k;
        }
      }
      good = __all_sync(0xffffffffu, good);
      if (!good || !fits) {
        if (record && lane == 0) record_error(&g_draft_ops_error, fits ? PK_DEVERR_DRAFT : PK_DEVERR_CONTEXT, s);
      } else {
        const int base = ctx - n;
        len = base + last + 1;
        const int32_t *row = tables + size_t(s) * max_blocks;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = lane + 32 * h;
          bool move = k <= last && kept[h] != k;
          int f = 0, t = 0;
          if (move) {
            const int a = base + kept[h], b = base + k;
            const int pa = __ldg(row + a / block_size), pb = __ldg(row + b / block_size);
            if (pa < 0 || pa >= num_blocks || pb < 0 || pb >= num_blocks) {
              if (record) record_error(&g_draft_ops_error, PK_DEVERR_BLOCK_ID, s);
              move = false;
            } else {
              f = pa * block_size + a % block_size;
              t = pb * block_size + b % block_size;
            }
          }
          const uint32_t all = __ballot_sync(0xffffffffu, move);
          const int at = moves + __popc(all & ((1u << lane) - 1));
          if (move) from[at] = f, to[at] = t;
          moves += __popc(all);
        }
      }
    }
    if (lane == 0) {
      sh_moves = moves;
      if (record && lens_out) lens_out[s] = len;
    }
  }
  __syncthreads();
  const int moves = sh_moves, j = blockIdx.x * 128 + threadIdx.x;
  if (j >= row_vecs) return;
  uint4 *const pool = (side ? v_cache : k_cache) + j;
  for (int k0 = 0; k0 < moves; k0 += U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u < moves) x[u] = pool[size_t(from[k0 + u]) * row_vecs];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u < moves) pool[size_t(to[k0 + u]) * row_vecs] = x[u];
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
    return n;
  cudaGetLastError();
  return 152;
}

template <typename T>
pk_status launch_verify(const VerifyParams &a, int32_t num_seqs, cudaStream_t stream) {
  // CTAs a sequence: as many as all fit at once, two an SM (with a second round 64 trees over a
  // vocabulary of 128 000 took 40 us), of 2048 elements or more each.
  const int sms = sm_count();
  int C = 1;
  while (C < kMaxCluster && int64_t(num_seqs) * C <= sms && a.vocab / C >= 4096) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(num_seqs * C));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(C);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T>, a) == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // namespace

extern "C" {

pk_status pk_verify_drafts(int32_t *num_accepted, int32_t *accepted, int64_t *next_tokens,
                           const void *target_probs, int64_t target_stride, const void *draft_probs,
                           int64_t draft_stride, pk_dtype probs_dtype, const int64_t *tokens,
                           const float *uniforms, const int32_t *q_offsets, const int32_t *parents,
                           int32_t num_seqs, int32_t num_rows, int32_t max_rows, int32_t vocab, void *stream) {
  if (num_seqs < 0 || num_rows < 0 || max_rows < 0 || vocab <= 0) return PK_ERR_INVALID_ARG;
  if (probs_dtype != PK_F32 && probs_dtype != PK_BF16) return PK_ERR_UNSUPPORTED;
  if (max_rows > PK_MAX_DRAFT || vocab > (1 << 24)) return PK_ERR_UNSUPPORTED;
  if (draft_probs && parents) return PK_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PK_OK;
  if (num_seqs > (1 << 24)) return PK_ERR_UNSUPPORTED;
  if (!num_accepted || !next_tokens || !q_offsets) return PK_ERR_INVALID_ARG;
  if (num_rows > 0 && (!accepted || !target_probs || !tokens || !uniforms)) return PK_ERR_INVALID_ARG;
  if (target_stride < vocab || (draft_probs && draft_stride < vocab)) return PK_ERR_INVALID_ARG;
  const uintptr_t mask = probs_dtype == PK_F32 ? 3u : 1u;
  if (((reinterpret_cast<uintptr_t>(target_probs) | reinterpret_cast<uintptr_t>(draft_probs)) & mask) ||
      (reinterpret_cast<uintptr_t>(tokens) & 7u) || (reinterpret_cast<uintptr_t>(next_tokens) & 7u))
    return PK_ERR_INVALID_ARG;
  VerifyParams a{num_accepted, accepted, next_tokens, target_probs, draft_probs, target_stride, draft_stride,
                 tokens,       uniforms, q_offsets,   parents,      num_rows,    max_rows,      vocab};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return probs_dtype == PK_F32 ? launch_verify<float>(a, num_seqs, st)
                               : launch_verify<__nv_bfloat16>(a, num_seqs, st);
}

pk_status pk_compact_drafts(void *k_cache, void *v_cache, const int32_t *block_tables,
                            int32_t max_blocks_per_seq, const int32_t *context_lens, const int32_t *q_offsets,
                            const int32_t *accepted, const int32_t *num_accepted, int32_t *context_lens_out,
                            int32_t num_seqs, int32_t num_rows, int32_t max_rows, const pk_cache_desc *desc,
                            void *stream) {
  if (!desc || desc->num_blocks <= 0 || desc->block_size <= 0 || desc->num_kv_heads <= 0 || desc->head_dim <= 0 ||
      num_seqs < 0 || num_rows < 0 || max_rows < 0)
    return PK_ERR_INVALID_ARG;
  if (desc->dtype != PK_F32 && desc->dtype != PK_BF16) return PK_ERR_UNSUPPORTED;
  const int64_t bytes = int64_t(desc->num_kv_heads) * desc->head_dim * (desc->dtype == PK_F32 ? 4 : 2);
  if (bytes % 16 != 0) return PK_ERR_INVALID_ARG;
  if (max_rows > PK_MAX_DRAFT || num_seqs > 65535 || int64_t(desc->num_blocks) * desc->block_size > INT32_MAX ||
      bytes / 16 > 1 << 24)
    return PK_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PK_OK;
  if (!k_cache || !v_cache || !block_tables || max_blocks_per_seq <= 0 || !context_lens || !q_offsets ||
      !num_accepted || (num_rows > 0 && !accepted) || context_lens_out == context_lens)
    return PK_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PK_ERR_INVALID_ARG;
  const int32_t vecs = int32_t(bytes / 16);
  compact_drafts_kernel<<<dim3(unsigned((vecs + 127) / 128), unsigned(num_seqs), 2), 128, 0,
                          static_cast<cudaStream_t>(stream)>>>(
      static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), block_tables, max_blocks_per_seq, context_lens,
      q_offsets, accepted, num_accepted, context_lens_out, num_rows, max_rows, desc->block_size, desc->num_blocks,
      vecs);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // extern "C"

}  // namespace pk
