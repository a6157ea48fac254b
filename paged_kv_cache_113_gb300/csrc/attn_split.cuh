// Attention of rows of query over paged keys and values on mma.sync tensor cores,
// fp32 and bf16, for the calls that a view describes: which rows a CTA has, which
// tokens each sees, what becomes of a score, and where results go.
//
// A view (DraftView, ExtendView) provides
//   Params, Shared<R>     the kernel's parameters and R rows' entries in shared memory;
//   unit(p, R, record, u) this CTA's work; false: none;
//   rows(p, u, sh)        fills Shared (all threads; a barrier follows) and may narrow
//                         the tokens; false: nothing to do;
//   factor(p)             what a product is multiplied by before score();
//   score(p, sh, r, t, x) a score in the exponent's scale (base 2);
//   sees(u, sh, r, t)     whether row r sees token t of the CTA's;
//   all_from, all_to      the CTA's tokens that every row sees (after rows());
//   place(p, u, sh, r)    where row r's state goes; nonzero(u, sh, r) whether a sum of
//                         0 is NaN.
#pragma once

#include "attn_rows.cuh"

namespace pk {
namespace {

// A CTA's rows r0 .. r0 + rows - 1 of a (sequence, KV head), and its tokens.
struct SplitUnit {
  int s, part, kvh;
  SeqRows sr;
  int r0, rows;
  int start, end;
  bool void_rows;  // the rows are zero and nothing is read (an invalid length, recorded)
};
enum class Place { kNowhere, kOut, kWorkspace };

// ---------------------------------------------------------------------------
// fp32 pools, bf16 ones of other block sizes, and few rows of bf16 (attn_split_kernel).
//
// Products on the tensor cores (mma.sync m16n8k16 bf16): each fp32 factor is the
// sum of three bf16 parts, x = x0 + x1 + x2 to 2^-25, and of the nine partial
// products the six that matter are taken (the others are below 2^-24). Six
// products at the bf16 rate are four times what three in tf32 reach through
// mma.sync on this chip (measured: 1037 against 133 multiply-adds a clock and SM),
// and twice the fp32 FMAs. A bf16 pool's factors are one part; the weights that
// meet its values are a pair hi + lo, as above.
//
// A CTA is four warps with 8 NT rows of a (sequence, KV head) over one partition;
// warp w takes the 16 tokens 64 j + 16 w .. of every step on its own: it copies
// its K and V rows into shared memory (K of the next step under the softmax and
// the values, V under the next scores), S^T = K Q^T with tokens as M and rows as
// N, the weights cross to the other operand through shared memory, O^T += V^T P^T.
// No barrier before the warps' states are merged at the end.
// Which elements of d (or tokens) are a fragment's k (or M) is free as long as
// both factors agree: a lane takes four neighbours at a time, one vector load for
// two products.
//
// Measured (fp32, 64 sequences of some 1000 tokens, 32 = 4 x 8 heads of 128): 16
// drafts 431 us (404 with sums left to the tensor cores, whose error grew to 5 10^-5
// at 32 768 tokens; 652 with three tf32 products, 797 with fp32 FMAs), 4 drafts 151
// us (554 with FMAs), one draft 109 to 113 us: bounded by the splitting of K and V into
// parts and the products' issue, not by memory (half of its rate at 4 drafts).
// ---------------------------------------------------------------------------
template <typename T, int D, int NT>
struct SplitShape {
  static constexpr int R = 8 * NT;
  // Row pitches in bytes, such that the lanes' vector loads meet no bank twice.
  static constexpr int K_PITCH = D * int(sizeof(T)) + (sizeof(T) == 4 ? 64 : 32);
  static constexpr int V_PITCH = D * int(sizeof(T)) + 32;
  static constexpr int Q_PITCH = D * 2 + 32;   // of a part
  static constexpr int P_PITCH = 20 * 4;       // 16 tokens of a row
  static constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;    // of a key, a query, a value
  static constexpr int W_PARTS = sizeof(T) == 4 ? 3 : 2;  // of a weight
  static constexpr int WARP_KV = 16 * (K_PITCH + V_PITCH), WARP_P = R * P_PITCH;
  static constexpr int O_PITCH = D + 4;        // floats, of the merge
  static constexpr int WARP_MERGE = R * (O_PITCH + 2) * 4;
  static constexpr int KV_BYTES = 4 * (WARP_KV > WARP_MERGE ? WARP_KV : WARP_MERGE);
  static constexpr int SMEM_BYTES = KV_BYTES + PARTS * R * Q_PITCH + 4 * WARP_P;
};

// N bf16 parts of a pair of fp32 values, largest first. What is not finite becomes
// NaN if N > 1 (inf - inf); what is finite has finite parts: of three, the first is at
// most the largest bf16 (fp32's largest values would round to infinity, and their NaN
// would reach rows that do not see them).
template <int N>
__device__ __forceinline__ void bf16_parts(float x, float y, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = N == 3 && i == 0 ? pack_bf16x2_finite(x, y) : pack_bf16x2(x, y);
    if (i + 1 == N) break;
    x -= bf16_lo(w[i]);
    y -= bf16_hi(w[i]);
  }
}

// D += A B over the parts of both, smallest products first. The tensor cores cut
// their fp32 sums off instead of rounding them, always toward zero: over thousands of
// tokens 10^-5 would be missing. So fp32 products are summed from zero, and the sum
// is added to D with a rounding.
template <int NA, int NB>
__device__ __forceinline__ void mma_parts(float (&d)[4], const uint32_t (&a)[4][NA], const uint32_t (&b)[2][NB]) {
  constexpr int LAST = NA > NB ? NA : NB;
  constexpr bool APART = NA > 1;
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int order = LAST - 1; order >= 0; --order)
#pragma unroll
    for (int i = 0; i <= order; ++i)
      if (i < NA && order - i < NB)
        mma_bf16_16816(APART ? t : d, a[0][i], a[1][i], a[2][i], a[3][i], b[0][order - i], b[1][order - i]);
  if (APART)
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] += t[e];
}

template <typename T, int D, int NT, typename View>
__global__ void __launch_bounds__(128, 2) attn_split_kernel(typename View::Params p) {
  using S = SplitShape<T, D, NT>;
  constexpr int NP = S::PARTS, NW = S::W_PARTS;
  constexpr int R = S::R, MT = D / 16, CH = D * int(sizeof(T)) / 16;
  launch_dependents();  // the merge may be scheduled as this grid drains
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t *q_sm = smem + S::KV_BYTES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  SplitUnit u;
  if (!View::unit(p, R, blockIdx.x == 0 && threadIdx.x == 0, u)) return;
  const int s = u.s, kvh = u.kvh, r0 = u.r0, rows = u.rows, part = u.part, G = p.group;
  const SeqRows &sr = u.sr;
  auto q_row = [&](int r) {  // element offset of row r0 + r in q and out
    return (size_t(sr.q0 + (r0 + r) / G) * p.num_q_heads + kvh * G + (r0 + r) % G) * D;
  };
  __shared__ typename View::template Shared<R> sh;
  __shared__ int poisoned;
  if (threadIdx.x == 0) poisoned = 0;
  View view;
  if (!u.void_rows && !view.rows(p, u, sh)) return;
  if (u.void_rows) {
    for (int i = threadIdx.x; i < rows * D; i += 128)
      store_elem(static_cast<T *>(p.out) + q_row(i / D) + i % D, 0.0f);
    return;
  }
  const int start = u.start, end = u.end;

  // This warp's 16 tokens of a step: lanes 0 - 15 know a row each.
  uint8_t *kw = smem + warp * S::WARP_KV, *vw = kw + 16 * S::K_PITCH;
  float *pw = reinterpret_cast<float *>(q_sm + NP * R * S::Q_PITCH + warp * S::WARP_P);
  const int32_t *trow = p.tables + size_t(s) * p.max_blocks;
  auto slot_of = [&](int t0) {  // of token t0 + lane % 16, or -1 past the end
    const int t = t0 + (lane & 15);
    if (t >= end) return -1;
    int phys = __ldg(trow + t / p.block_size);
    if (phys < 0 || phys >= p.num_blocks) {
      record_error(&g_rows_error, PK_DEVERR_BLOCK_ID, s);
      phys = 0;  // stay in bounds; the result is flagged
    }
    return phys * p.block_size + t % p.block_size;
  };
  auto copy = [&](const void *pool, uint8_t *to, int pitch, int slot) {
#pragma unroll
    for (int i = 0; i < 16 * CH / 32; ++i) {
      const int row = (i * 32 + lane) / CH, ch = (i * 32 + lane) % CH;
      const int sl = __shfl_sync(0xffffffffu, slot, row);
      cp_async16(smem_addr(to + row * pitch + ch * 16),
                 static_cast<const uint8_t *>(pool) +
                     ((size_t(max(sl, 0)) * p.num_kv_heads + kvh) * D) * sizeof(T) + ch * 16,
                 sl < 0 ? 0 : 16);  // rows past the end are zeros
    }
    cp_async_commit();
  };
  int t0 = start + warp * 16;
  int slot = slot_of(t0), slot_next = slot_of(t0 + 64);
  copy(p.k_cache, kw, S::K_PITCH, slot);
  copy(p.v_cache, vw, S::V_PITCH, slot);
  for (int i = threadIdx.x; i < R * D / 2; i += 128) {
    const int r = i / (D / 2), c = i % (D / 2) * 2;
    const T *src = static_cast<const T *>(p.q) + q_row(min(r, rows - 1)) + c;
    const float f = r >= rows ? 0.0f : (NP > 1 ? View::factor(p) : 1.0f);  // bf16 queries stay as they are
    uint32_t w[NP];
    bf16_parts(r < rows ? load_elem(src) * f : 0.0f, r < rows ? load_elem(src + 1) * f : 0.0f, w);
#pragma unroll
    for (int k = 0; k < NP; ++k) *reinterpret_cast<uint32_t *>(q_sm + (k * R + r) * S::Q_PITCH + c * 2) = w[k];
  }
  __syncthreads();

  const int qd = lane & 3, rw = lane >> 2;
  float o[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.0f;
#pragma unroll
    for (int k = 0; k < MT; ++k) o[k][n][0] = o[k][n][1] = o[k][n][2] = o[k][n][3] = 0.0f;
  }
  for (; t0 < end; t0 += 64) {
    cp_async_wait_group<1>();  // K is here
    __syncwarp();
    // S^T = K Q^T: lanes hold tokens rw, rw + 8 and rows 2 qd, 2 qd + 1 of 8.
    float x[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.0f;
#pragma unroll 2  // all eight at once cost registers: 525 us for 431
    for (int c = 0; c < D / 16; ++c) {
      uint32_t a[4][NP];
      const float4 k0 = load4(reinterpret_cast<const T *>(kw + rw * S::K_PITCH) + 16 * c + 4 * qd);
      const float4 k1 = load4(reinterpret_cast<const T *>(kw + (rw + 8) * S::K_PITCH) + 16 * c + 4 * qd);
      bf16_parts(k0.x, k0.y, a[0]);
      bf16_parts(k1.x, k1.y, a[1]);
      bf16_parts(k0.z, k0.w, a[2]);
      bf16_parts(k1.z, k1.w, a[3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t b[2][NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const uint2 w = *reinterpret_cast<const uint2 *>(q_sm + (k * R + 8 * n + rw) * S::Q_PITCH +
                                                           32 * c + 8 * qd);
          b[0][k] = w.x, b[1][k] = w.y;
        }
        mma_parts(x[n], a, b);
      }
    }
    if (NP > 1) {
      // A key value that is not finite made its scores NaN, as its second part is
      // inf - inf: those are summed again without parts, as -inf is a score too.
      float odd = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) odd = fmaf(x[n][e], 0.0f, odd);
      if (__any_sync(0xffffffffu, odd != 0.0f)) {
        uint32_t which = 0;
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i)
          if (x[i / 4][i % 4] != x[i / 4][i % 4]) which |= 1u << i, x[i / 4][i % 4] = 0.0f;
#pragma unroll 1
        for (int j = 0; which && j < D; ++j)
#pragma unroll
          for (int i = 0; i < 4 * NT; ++i) {
            if (!((which >> i) & 1)) continue;
            float f = 0.0f;
#pragma unroll
            for (int k = NP - 1; k >= 0; --k)
              f += load_elem(reinterpret_cast<const __nv_bfloat16 *>(
                                 q_sm + (k * R + 8 * (i / 4) + 2 * qd + (i & 1)) * S::Q_PITCH) + j);
            x[i / 4][i % 4] =
                fmaf(load_elem(reinterpret_cast<const T *>(kw + (rw + 8 * (i % 4 / 2)) * S::K_PITCH) + j), f,
                     x[i / 4][i % 4]);
          }
      }
    }
    __syncwarp();
    const int slot_v = slot_next;
    slot = slot_next;
    copy(p.k_cache, kw, S::K_PITCH, slot);  // the next step's K
    slot_next = slot_of(t0 + 128);
    const bool careful = t0 < view.all_from || t0 + 16 > view.all_to;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (NP == 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] *= View::factor(p);
      if (View::SCORES)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[n][e] = View::score(p, sh, 8 * n + 2 * qd + (e & 1), t0 + rw + 8 * (e >> 1), x[n][e]);
      if (careful)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = t0 + rw + 8 * (e >> 1);
          if (!View::sees(u, sh, 8 * n + 2 * qd + (e & 1), t)) x[n][e] = -INFINITY;
        }
      float corr[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(x[n][h], x[n][2 + h]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m[n][h], mx);
        const float ref = mn == -INFINITY ? 0.0f : mn;  // nothing seen so far: every weight is 0
        corr[h] = exp2f(m[n][h] - ref);
        m[n][h] = mn;
        x[n][h] = exp2f(x[n][h] - ref);
        x[n][2 + h] = exp2f(x[n][2 + h] - ref);
        l[n][h] = fmaf(l[n][h], corr[h], x[n][h] + x[n][2 + h]);
      }
      if (__any_sync(0xffffffffu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
        for (int k = 0; k < MT; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][n][e] *= corr[e & 1];
      }
      float *pr = pw + (8 * n + 2 * qd) * (S::P_PITCH / 4) + rw;
      pr[0] = x[n][0];
      pr[S::P_PITCH / 4] = x[n][1];
      pr[8] = x[n][2];
      pr[S::P_PITCH / 4 + 8] = x[n][3];
    }
    cp_async_wait_group<1>();  // V is here
    __syncwarp();
    if (careful) {
      // What is not finite in values that some rows do not see becomes 0, or it would
      // reach those too (0 * NaN); the rows that do see it get it at the end.
      for (int i = lane; i < 16 * D; i += 32) {
        const int t = t0 + i / D;
        T *v = reinterpret_cast<T *>(vw + (i / D) * S::V_PITCH) + i % D;
        if ((t < view.all_from || t >= view.all_to) && t < end && !(fabsf(load_elem(v)) <= 3.402823466e38f)) {
          store_elem(v, 0.0f);
          poisoned = 1;
        }
      }
      __syncwarp();
    }
    // O^T += V^T P^T: k = 2 qd, 2 qd + 1, 2 qd + 8, 2 qd + 9 are tokens qd, qd + 4,
    // qd + 8, qd + 12; rows rw and rw + 8 of a column tile are 4 rw + 2 e and the next.
    uint32_t b[NT][2][NW];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float *w = pw + (8 * n + rw) * (S::P_PITCH / 4) + qd;
      bf16_parts(w[0], w[4], b[n][0]);
      bf16_parts(w[8], w[12], b[n][1]);
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      float v[4][4];  // [token][column]
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 y = load4(reinterpret_cast<const T *>(vw + (qd + 4 * k) * S::V_PITCH) + 32 * c + 4 * rw);
        v[k][0] = y.x, v[k][1] = y.y, v[k][2] = y.z, v[k][3] = y.w;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t a[4][NP];
        bf16_parts(v[0][2 * e], v[1][2 * e], a[0]);
        bf16_parts(v[0][2 * e + 1], v[1][2 * e + 1], a[1]);
        bf16_parts(v[2][2 * e], v[3][2 * e], a[2]);
        bf16_parts(v[2][2 * e + 1], v[3][2 * e + 1], a[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_parts(o[2 * c + e][n], a, b[n]);
      }
    }
    __syncwarp();
    copy(p.v_cache, vw, S::V_PITCH, slot_v);  // the next step's V
  }
  cp_async_wait();
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], off);
  // Merge the warps' states, over the K/V rows.
  __syncthreads();
  float *sm_o = reinterpret_cast<float *>(smem), *sm_m = sm_o + 4 * R * S::O_PITCH, *sm_l = sm_m + 4 * R;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = warp * R + 8 * n + 2 * qd;
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      // Tile k's rows rw and rw + 8 are columns 32 (k / 2) + 4 rw + 2 (k % 2) and the next.
      float *to = sm_o + r * S::O_PITCH + 32 * (k >> 1) + 4 * rw + 2 * (k & 1);
      *reinterpret_cast<float2 *>(to) = make_float2(o[k][n][0], o[k][n][2]);
      *reinterpret_cast<float2 *>(to + S::O_PITCH) = make_float2(o[k][n][1], o[k][n][3]);
    }
    if (rw == 0) {
      sm_m[r] = merge_max(m[n][0], l[n][0]), sm_m[r + 1] = merge_max(m[n][1], l[n][1]);
      sm_l[r] = l[n][0], sm_l[r + 1] = l[n][1];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * D; i += 128) {
    const int r = i / D, c = i % D;
    const Place place = View::place(p, u, sh, r);
    if (place == Place::kNowhere) continue;
    float M = -INFINITY, L = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sm_m[w * R + r]);
    const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = exp2f(sm_m[w * R + r] - ref);  // 0 for a warp that saw no token
      L = fmaf(sm_l[w * R + r], f, L);
      O = merge_add(O, sm_o[(w * R + r) * S::O_PITCH + c], f);
    }
    // A value that every row sees and that is not finite gave NaN, by the product with a
    // part of a weight that is 0 or negative: the sum of what is not finite in its place.
    if (!(fabsf(O) <= 3.402823466e38f) && fabsf(L) <= 3.402823466e38f) {
      float odd = 0.0f;
#pragma unroll 4
      for (int t = view.all_from; t < view.all_to; ++t) {
        const int phys = min(max(__ldg(trow + t / p.block_size), 0), p.num_blocks - 1);
        const float y = load_elem(static_cast<const T *>(p.v_cache) +
                                  ((size_t(phys) * p.block_size + t % p.block_size) * p.num_kv_heads + kvh) * D + c);
        odd += fabsf(y) <= 3.402823466e38f ? 0.0f : y;
      }
      if (odd != 0.0f) O = odd;
    }
    if (poisoned)  // what is not finite in the other values that the row sees
      for (int t = start; t < end; ++t) {
        if (t == view.all_from && t < view.all_to) t = view.all_to;
        if (t >= end || !View::sees(u, sh, r, t)) continue;
        const int phys = __ldg(trow + t / p.block_size);
        if (phys < 0 || phys >= p.num_blocks) continue;
        const float y = load_elem(static_cast<const T *>(p.v_cache) +
                                  ((size_t(phys) * p.block_size + t % p.block_size) * p.num_kv_heads + kvh) * D + c);
        if (!(fabsf(y) <= 3.402823466e38f)) O += y;
      }
    if (place == Place::kWorkspace) {
      const size_t to = q_row(r) / D * p.num_partitions + part;
      p.ws_acc[to * D + c] = O;
      if (c == 0) {
        p.ws_m[to] = merge_max(M, L);
        p.ws_l[to] = L;
      }
    } else {
      store_elem(static_cast<T *>(p.out) + q_row(r) + c, O / denominator(L, View::nonzero(u, sh, r)));
    }
  }
}

// The view of drafted tokens: rows see the tokens before the drafts, and those of their mask.
struct DraftView {
  using Params = RowsParams;
  static constexpr bool SCORES = false;
  template <int R>
  struct Shared {
    uint64_t masks[R];
  };
  int all_from, all_to;

  static __device__ __forceinline__ bool unit(const RowsParams &p, int R, bool record, SplitUnit &u) {
    u.kvh = blockIdx.x / p.row_tiles;
    if (!work_item(p, blockIdx.y, gridDim.z - 1 - blockIdx.z, record, u.s, u.part)) return false;
    u.sr = seq_rows(p, u.s, record && u.part == 0);
    u.r0 = blockIdx.x % p.row_tiles * R;
    u.rows = min(R, u.sr.n * p.group - u.r0);
    if (u.rows <= 0) return false;
    u.void_rows = u.sr.ctx == 0;
    if (u.void_rows) return u.part == 0;
    u.start = u.part * p.partition;
    u.end = min(u.sr.ctx, u.start + p.partition);
    return u.part < u.sr.np;
  }
  static __device__ __forceinline__ int base(const SplitUnit &u) { return u.sr.ctx - u.sr.n; }
  template <int R>
  __device__ __forceinline__ bool rows(const RowsParams &p, SplitUnit &u, Shared<R> &sh) {
    if (threadIdx.x < R)
      sh.masks[threadIdx.x] = int(threadIdx.x) < u.rows
                                  ? draft_mask(p, u.sr.q0, (u.r0 + int(threadIdx.x)) / p.group, u.sr.n)
                                  : 0;
    all_from = u.start, all_to = min(base(u), u.end);
    return true;
  }
  static __device__ __forceinline__ float factor(const RowsParams &p) { return p.scale_log2; }
  template <int R>
  static __device__ __forceinline__ float score(const RowsParams &, const Shared<R> &, int, int, float x) {
    return x;
  }
  template <int R>
  static __device__ __forceinline__ bool sees(const SplitUnit &u, const Shared<R> &sh, int r, int t) {
    return t < u.end && (t < base(u) || ((sh.masks[r] >> (t - base(u))) & 1));
  }
  template <int R>
  static __device__ __forceinline__ Place place(const RowsParams &, const SplitUnit &u, const Shared<R> &, int) {
    return u.sr.np > 1 ? Place::kWorkspace : Place::kOut;
  }
  template <int R>
  static __device__ __forceinline__ bool nonzero(const SplitUnit &u, const Shared<R> &sh, int r) {
    return base(u) > 0 || sh.masks[r] != 0;
  }
};

// Rows per CTA of attn_split_kernel: the fewest that hold a sequence's, at most 32.
int split_rows(int rows) { return rows <= 8 ? 8 : (rows <= 16 ? 16 : 32); }

template <typename T, int D, int NT, typename View>
pk_status launch_split(const typename View::Params &p, const dim3 &grid, cudaStream_t stream) {
  using S = SplitShape<T, D, NT>;
  auto kern = attn_split_kernel<T, D, NT, View>;
  static std::atomic<uint64_t> ready{0};
  if (!smem_ready(kern, S::SMEM_BYTES, ready)) return PK_ERR_CUDA;
  kern<<<grid, 128, S::SMEM_BYTES, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // namespace
}  // namespace pk
