// Up to eight rows of bf16 (attn_few_kernel): pk_paged_attention_extend for decoded tokens,
// one query head group each, or a few drafts of a small group.
//
// Per KV head it has 4 d operations a row and key for the 4 d bytes of key and value, so memory
// bounds it. A CTA has a unit: a producer warp streams the blocks' K and V rows into a ring of
// two stages of 64 tokens by TMA (three CTAs an SM: 192 KB under way), four warps take 16
// tokens of each: S^T = K Q^T and O^T += V^T P^T on mma.sync tensor cores, eight rows wide,
// softmax in registers, the weights a bf16 pair. The layout of pk_paged_attention_decode's
// kernel, and its rate: cap and bias are a few operations on four scores a lane, under the
// copies.
//
// Measured (heads of 128, blocks of 16): 8 sequences of 32 768 tokens, 64 / 8 heads, biased, 160 to
// 162 us, 6.6 TB/s (98% of a copy; 200 on attn_split_kernel); 64 of 1000 to 4000 tokens of which
// the last 1024 are seen, 32 / 32 heads, 163 to 168 us, 6.5 TB/s (180); 256 of some 500 tokens,
// 32 / 8 heads, capped, 84 to 88 us, 5.8 TB/s (106): there the launch's first loads and uneven ends.
#pragma once

#include "attn_extend.cuh"
#include "attn_tile.cuh"
#include "pk_tma_host.h"

namespace pk {
namespace {

constexpr int kFewRows = 8, kFewWarps = 4, kFewStages = 2;

template <int D, int BS>
struct FewShape {
  static constexpr int TPS = 16 * kFewWarps, BPS = TPS / BS;  // tokens and blocks of a stage
  static constexpr int SLABS = D / 64, SLAB = TPS * 128;      // 128-byte column slabs
  static constexpr int KV_BYTES = SLABS * SLAB, STAGE = 2 * KV_BYTES;
  static constexpr int PITCH = D + 4;                         // floats, of the merge
  static constexpr int MERGE = kFewWarps * kFewRows * (PITCH + 2) * 4;
  static constexpr int SMEM_BYTES = 1024 + (kFewStages * STAGE > MERGE ? kFewStages * STAGE : MERGE);
};

// tanh to 2^-20 of itself. (1 - 2 / (1 + e^2x) is off by 2^-21 whatever its size: with a cap of
// 10^6 that alone was 0.5 of a score of 1.)
__device__ __forceinline__ float tanh_rel(float x) {
  const float z = x * x;
  const float small = x * fmaf(fmaf(fmaf(fmaf(kTanh4, z, kTanh3), z, kTanh2), z, kTanh1), z, kTanh0);
  const float large = fmaf(-2.0f, reciprocal(1.0f + exp2_ftz(x * 2.88539008f)), 1.0f);
  return fabsf(x) <= kTanhSmall ? small : large;
}

template <int D, int BS>
__global__ void __launch_bounds__((kFewWarps + 1) * 32, 3)
    attn_few_kernel(ExtendParams p, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap) {
  using S = FewShape<D, BS>;
  constexpr int ST = kFewStages, KSTEPS = D / 16;
  launch_dependents();  // the merge may be scheduled as this grid drains
  extern __shared__ uint8_t smem_raw[];
  const uint32_t stages = (smem_addr(smem_raw) + 1023u) & ~1023u;
  __shared__ __align__(8) uint64_t bars[2 * ST];
  __shared__ ExtendView::Shared<kFewRows> sh;
  __shared__ int poisoned;
  auto full = [&](int i) { return smem_addr(bars + i % ST); };
  auto empty = [&](int i) { return smem_addr(bars + ST + i % ST); };
  auto phase = [](int i) { return uint32_t(i / ST) & 1u; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.group;
  SplitUnit u;
  if (!extend_unit(p, blockIdx.x, kFewRows, threadIdx.x == 0, u)) return;
  auto q_row = [&](int r) {  // element offset of row r0 + r in q and out
    return (size_t(u.sr.q0 + (u.r0 + r) / G) * p.num_q_heads + u.kvh * G + (u.r0 + r) % G) * D;
  };
  if (threadIdx.x == 0) {
    poisoned = 0;
    for (int i = 0; i < ST; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), kFewWarps);
    }
    fence_barrier_init();
  }
  ExtendView view;
  if (!u.void_rows && !view.rows(p, u, sh)) return;
  if (u.void_rows) {
    for (int i = threadIdx.x; i < u.rows * D; i += blockDim.x)
      static_cast<__nv_bfloat16 *>(p.out)[q_row(i / D) + i % D] = __float2bfloat16_rn(0.0f);
    return;
  }
  const int start = u.start, end = u.end, nst = (end - start + S::TPS - 1) / S::TPS;
  const int32_t *trow = p.tables + size_t(u.s) * p.max_blocks + start / BS;
  if (warp == kFewWarps) {
    // ---------------- producer ----------------
    if (lane == 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
    // Table entries are read ahead in chunks of 32 blocks, a lane each.
    const int nb = (end - start + BS - 1) / BS;
    auto entry = [&](int j) { return j < nb ? __ldg(trow + j) : 0; };
    int cur = entry(lane), nxt = entry(32 + lane), chunk = 0, issued = 0;
    for (int st = 0; st < nst; ++st) {
      const int b0 = st * S::BPS;
      if (b0 >= 32 * (chunk + 1)) {
        ++chunk;
        cur = nxt;
        nxt = entry(32 * (chunk + 1) + lane);
      }
      int phys = __shfl_sync(0xffffffffu, cur, (b0 & 31) + min(lane, S::BPS - 1));
      if (st >= ST && !mbar_wait(empty(st), phase(st - ST))) {
        if (lane == 0) record_error(&g_rows_error, PK_DEVERR_TIMEOUT, u.s);
        break;
      }
      const int nblk = min(S::BPS, nb - b0);
      if (lane == 0) mbar_arrive_expect_tx(full(st), uint32_t(nblk * S::SLABS * 2 * BS * 128));
      __syncwarp();
      if (lane < nblk) {
        if (phys < 0 || phys >= p.num_blocks) {
          record_error(&g_rows_error, PK_DEVERR_BLOCK_ID, u.s);
          phys = 0;  // stay in bounds and keep the byte count; the result is flagged
        }
        const uint32_t dst = stages + st % ST * S::STAGE + lane * BS * 128;
#pragma unroll
        for (int h = 0; h < S::SLABS; ++h) {
          tma_load_3d(dst + h * S::SLAB, &kmap, full(st), h * 64, u.kvh, phys * BS);
          tma_load_3d(dst + S::KV_BYTES + h * S::SLAB, &vmap, full(st), h * 64, u.kvh, phys * BS);
        }
      }
      issued = st + 1;
    }
    // Let every issued copy land before the warp leaves.
    for (int st = max(0, issued - ST); st < issued; ++st) mbar_wait(full(st), phase(st));
    return;
  }

  // ---------------- consumers ----------------
  const int qd = lane & 3, rw = lane >> 2;  // rows 2 qd, 2 qd + 1; tokens rw, rw + 8
  uint32_t qb[KSTEPS][2];                   // Q^T as the B operand
  {
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) + q_row(min(rw, u.rows - 1));
#pragma unroll
    for (int ks = 0; ks < KSTEPS; ++ks) {
      const uint32_t a = *reinterpret_cast<const uint32_t *>(src + ks * 16 + 2 * qd);
      const uint32_t b = *reinterpret_cast<const uint32_t *>(src + ks * 16 + 8 + 2 * qd);
      qb[ks][0] = rw < u.rows ? a : 0u;
      qb[ks][1] = rw < u.rows ? b : 0u;
    }
  }
  float o[KSTEPS][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int mt = 0; mt < KSTEPS; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.0f;
  const float slope[2] = {sh.slope[2 * qd], sh.slope[2 * qd + 1]};
  const int pos[2] = {sh.pos[2 * qd], sh.pos[2 * qd + 1]};
  const int row0 = warp * 16;
  for (int st = 0; st < nst; ++st) {
    if (!mbar_wait(full(st), phase(st))) {
      if (lane == 0) record_error(&g_rows_error, PK_DEVERR_TIMEOUT, u.s);
      break;
    }
    __syncwarp();
    const uint32_t kbase = stages + st % ST * S::STAGE, vbase = kbase + S::KV_BYTES;
    const int t0 = start + st * S::TPS + row0, nvalid = end - t0;
    if (nvalid > 0) {
      const bool careful = t0 < view.all_from || t0 + 16 > view.all_to;
      if (careful) {
        // Values past the end are zeroed, and so is what is not finite in values that some rows
        // do not see, which would reach those too (0 * NaN); the rows that do get it at the end.
        bool wrote = false;
        for (int i = lane; i < 16 * S::SLABS * 8; i += 32) {
          const int r = i / (S::SLABS * 8), c = i % (S::SLABS * 8), t = t0 + r;
          if (t >= view.all_from && t < view.all_to) continue;
          const uint32_t a = vbase + (c >> 3) * S::SLAB + (row0 + r) * 128 + (c & 7) * 16;
          uint32_t w[4];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(a));
          bool odd = r >= nvalid;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (r >= nvalid || (w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u, odd = true;
            if (r >= nvalid || (w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu, odd = true;
          }
          if (!odd) continue;
          wrote = true;
          if (r < nvalid) poisoned = 1;
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                       "r"(w[3])
                       : "memory");
        }
        // A later tile's copies go to the same bytes by the other proxy.
        if (__any_sync(0xffffffffu, wrote)) fence_proxy_async_shared();
        __syncwarp();
      }
      float sacc[2][4];
      tile_scores<KSTEPS>(kbase, S::SLAB, row0, qb, sacc, lane);
      float x[4];  // token rw + 8 (e / 2), row 2 qd + e % 2
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = (sacc[0][e] + sacc[1][e]) * p.factor;
        if (p.cap_log2 != 0.0f) x[e] = p.cap_log2 * tanh_rel(x[e]);
        if (p.slopes) x[e] = fmaf(-slope[e & 1], float(abs(pos[e & 1] - (t0 + rw + 8 * (e >> 1)))), x[e]);
        if (careful && !ExtendView::sees(u, sh, 2 * qd + (e & 1), t0 + rw + 8 * (e >> 1))) x[e] = -INFINITY;
      }
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(x[h], x[2 + h]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m[h], mx);
        const float ref = mn == -INFINITY ? 0.0f : mn;  // nothing seen so far: every weight is 0
        f[h] = exp2f(m[h] - ref);
        m[h] = mn;
        x[h] = exp2f(x[h] - ref);
        x[2 + h] = exp2f(x[2 + h] - ref);
        l[h] = fmaf(l[h], f[h], x[h] + x[2 + h]);
      }
      // The weights enter the product as a bf16 pair: one bf16 would put 2^-9 on every output.
      const uint32_t w01 = pack_bf16x2(x[0], x[1]), w23 = pack_bf16x2(x[2], x[3]);
      const uint32_t r01 = pack_bf16x2(x[0] - bf16_lo(w01), x[1] - bf16_hi(w01));
      const uint32_t r23 = pack_bf16x2(x[2] - bf16_lo(w23), x[3] - bf16_hi(w23));
#pragma unroll
      for (int mt = 0; mt < KSTEPS; ++mt) {
        o[mt][0] *= f[0];
        o[mt][1] *= f[1];
        o[mt][2] *= f[0];
        o[mt][3] *= f[1];
      }
      tile_values<KSTEPS>(vbase, S::SLAB, row0, w01, w23, r01, r23, o, lane);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty(st));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);

  // Merge the warps' states in shared memory (the ring is free: every copy has landed and has
  // been used).
  named_barrier(1, kFewWarps * 32);
  float *sm_o = reinterpret_cast<float *>(smem_raw + (stages - smem_addr(smem_raw)));
  float *sm_m = sm_o + kFewWarps * kFewRows * S::PITCH, *sm_l = sm_m + kFewWarps * kFewRows;
#pragma unroll
  for (int mt = 0; mt < KSTEPS; ++mt) {
    float *to = sm_o + (warp * kFewRows + 2 * qd) * S::PITCH + mt * 16 + rw;
    to[0] = o[mt][0];
    to[S::PITCH] = o[mt][1];
    to[8] = o[mt][2];
    to[S::PITCH + 8] = o[mt][3];
  }
  if (rw < 2) {
    sm_m[warp * kFewRows + 2 * qd + rw] = merge_max(rw ? m[1] : m[0], rw ? l[1] : l[0]);
    sm_l[warp * kFewRows + 2 * qd + rw] = rw ? l[1] : l[0];
  }
  named_barrier(1, kFewWarps * 32);
  for (int idx = threadIdx.x; idx < u.rows * (D / 2); idx += kFewWarps * 32) {
    const int r = idx / (D / 2), i = (idx % (D / 2)) * 2;
    const Place place = row_place(p, sh.lo[r], sh.hi[r], u.part);
    if (place == Place::kNowhere) continue;
    float M = -INFINITY, L = 0.0f, O[2] = {0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, sm_m[w * kFewRows + r]);
    const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float f = exp2f(sm_m[w * kFewRows + r] - ref);  // 0 for a warp that saw no token
      const float *row = sm_o + (w * kFewRows + r) * S::PITCH + i;
      L = fmaf(sm_l[w * kFewRows + r], f, L);
      O[0] = merge_add(O[0], row[0], f);
      O[1] = merge_add(O[1], row[1], f);
    }
    if (poisoned)  // what is not finite in values that the row sees and others do not
      for (int t = max(start, sh.lo[r]); t < min(end, sh.hi[r]); ++t) {
        if (t >= view.all_from && t < view.all_to) continue;
        const int phys = __ldg(trow + (t - start) / BS);
        if (phys < 0 || phys >= p.num_blocks) continue;
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v_cache) +
                                 ((size_t(phys) * BS + t % BS) * p.num_kv_heads + u.kvh) * D + i;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y = __bfloat162float(v[e]);
          if (!(fabsf(y) <= 3.402823466e38f)) O[e] += y;
        }
      }
    const size_t at = q_row(r);
    if (place == Place::kOut) {
      const float inv = 1.0f / denominator(L, false);
      *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.out) + at + i) =
          __floats2bfloat162_rn(O[0] * inv, O[1] * inv);
    } else {
      const size_t slot = at / D * p.num_partitions + u.part;
      *reinterpret_cast<float2 *>(p.ws_acc + slot * D + i) = make_float2(O[0], O[1]);
      if (i == 0) {
        p.ws_m[slot] = merge_max(M, L);
        p.ws_l[slot] = L;
      }
    }
  }
}

template <int D, int BS>
pk_status launch_few_as(const ExtendParams &p, const pk_cache_desc &d, unsigned units, cudaStream_t stream) {
  CUtensorMap kmap, vmap;
  if (!encode_bf16_pool(&kmap, p.k_cache, d) || !encode_bf16_pool(&vmap, p.v_cache, d)) return PK_ERR_CUDA;
  auto kern = attn_few_kernel<D, BS>;
  static std::atomic<uint64_t> ready{0};
  if (!smem_ready(kern, FewShape<D, BS>::SMEM_BYTES, ready)) return PK_ERR_CUDA;
  kern<<<units, (kFewWarps + 1) * 32, FewShape<D, BS>::SMEM_BYTES, stream>>>(p, kmap, vmap);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

template <int D>
pk_status launch_few(const ExtendParams &p, const pk_cache_desc &d, unsigned units, cudaStream_t stream) {
  return d.block_size == 8    ? launch_few_as<D, 8>(p, d, units, stream)
         : d.block_size == 16 ? launch_few_as<D, 16>(p, d, units, stream)
                              : launch_few_as<D, 32>(p, d, units, stream);
}

}  // namespace
}  // namespace pk
