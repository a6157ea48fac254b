// Attention of each sequence's drafted tokens over its cached context
// (pk_paged_attention_tree), for verifying a tree or a chain of drafts in one
// pass: the n drafted tokens are the last n of the context, their K/V already
// in the cache, and a 64-bit mask per token says which drafts it sees.
//
// Per KV head a sequence is n G rows of query against ctx keys: 4 d operations
// per row and key for 4 d bytes (bf16), so that up to some 283 rows of work per
// byte read the memory bounds it, beyond that the tensor cores.
//
// bf16 (attn_tree_kernel): tcgen05 products with tensor-memory accumulators. A
// CTA holds 128 rows, one lane of tensor memory each, and goes over its keys in
// tiles of 64 tokens:
//   producer warp   TMA loads of each block's K and V into two rings;
//   product warp    one thread issues S_j = Q K_j^T (128 x 64) and, once the
//                   weights are there, O += P_j V_j, P_j read from tensor
//                   memory; S_{j+1} is issued before P_j V_j, so that it runs
//                   under the softmax of tile j;
//   softmax warps   a thread owns a row: reads its 64 scores, masks them,
//                   keeps the running maximum and sum, and writes the weights
//                   over the scores.
// O stays in tensor memory. A row's reference of the exponent moves only when
// the maximum has outgrown it by 2^8: until then weights up to 2^8 are added as
// they are (fp32 accumulators, fp32 sums), and O is rescaled a few times per
// row instead of once per tile.
// The weights enter the product as a bf16 pair hi + lo (one bf16 would put
// 2^-9 on every output).
// 256 columns of tensor memory (two 64-column score tiles, 128 for O) and 97 KB
// of shared memory let two CTAs share an SM: one's softmax overlaps the
// other's products.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_rows.cuh"
#include "pagedkv.h"
#include "pk_tcgen05.cuh"
#include "pk_tma_host.h"

namespace pk {

extern "C" int pkx_take_tree_attention_error(cudaStream_t stream) {
  return take_error_word(g_rows_error, stream);
}

namespace {

constexpr int kRows = 128;          // query rows of a CTA
constexpr int kTile = 64;           // tokens of a tile
constexpr int kThreads = 192;       // 4 softmax warps, the producer, the product warp
constexpr uint32_t kTmemCols = 256;
constexpr float kSlack = 8.0f;      // log2 of how far a maximum may outgrow the reference

template <int D, int BS>
struct TreeShape {
  static constexpr int SLABS = D / 64;               // 128-byte column slabs
  static constexpr int Q_SLAB = kRows * 128, KV_SLAB = kTile * 128;
  static constexpr int Q_BYTES = SLABS * Q_SLAB, KV_BYTES = SLABS * KV_SLAB;
  static constexpr int STAGES = 2;                   // of the K ring and of the V ring
  static constexpr int BPT = kTile / BS;             // blocks per tile
  static constexpr int SMEM_BYTES = 1024 + Q_BYTES + 2 * STAGES * KV_BYTES;
};

template <int D, int BS>
__global__ void __launch_bounds__(kThreads, 2)
    attn_tree_kernel(RowsParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using S = TreeShape<D, BS>;
  constexpr int STAGES = S::STAGES;
  launch_dependents();  // the merge may be scheduled as this grid drains
  extern __shared__ uint8_t smem_raw[];
  const uint32_t q_sm = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t k_sm = q_sm + S::Q_BYTES, v_sm = k_sm + STAGES * S::KV_BYTES;
  __shared__ __align__(8) uint64_t bars[7 + 4 * STAGES];
  __shared__ uint32_t tmem_slot;
  __shared__ int poisoned;
  auto bar = [&](int i) { return smem_addr(bars + i); };
  // Every wait names a phase of which the one before has ended for certain and
  // the one after cannot: a wait by parity tells neighbouring phases apart, not
  // more. So the products' ends alternate between two barriers: when tile j's
  // scores are there, product j - 2 has ended, but j - 1 may not have.
  const uint32_t q_ready = bar(0);
  auto s_full = [&](int i) { return bar(1 + i); };
  auto p_full = [&](int i) { return bar(3 + i); };
  auto o_done = [&](int i) { return bar(5 + i); };  // product i, i + 2, ... has ended
  auto k_full = [&](int i) { return bar(7 + i); };
  auto k_empty = [&](int i) { return bar(7 + STAGES + i); };
  auto v_full = [&](int i) { return bar(7 + 2 * STAGES + i); };
  auto v_empty = [&](int i) { return bar(7 + 3 * STAGES + i); };

  const int kvh = blockIdx.x / p.row_tiles, tile = blockIdx.x % p.row_tiles;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool record = blockIdx.x == 0 && threadIdx.x == 0;
  int s, part;
  if (!work_item(p, blockIdx.y, gridDim.z - 1 - blockIdx.z, record, s, part)) return;
  const SeqRows sr = seq_rows(p, s, record && part == 0);
  const int G = p.group, r0 = tile * kRows, rows = min(kRows, sr.n * G - r0);
  if (rows <= 0) return;
  auto q_row = [&](int r) {  // element offset of row r0 + r in q and out
    return (size_t(sr.q0 + (r0 + r) / G) * p.num_q_heads + kvh * G + (r0 + r) % G) * D;
  };
  if (sr.ctx == 0) {  // invalid length (recorded): zero rows
    if (part == 0)
      for (int i = threadIdx.x; i < rows * (D / 8); i += kThreads)
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + q_row(i / (D / 8)) +
                                   (i % (D / 8)) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  if (part >= sr.np) return;
  const int start = part * p.partition, end = min(sr.ctx, start + p.partition);
  const int base = sr.ctx - sr.n;
  const int nt = (end - start + kTile - 1) / kTile;
  const int active = (rows + 31) / 32;  // softmax warps with rows

  if (threadIdx.x == 0) {
    mbar_init(q_ready, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(o_done(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), active);
    }
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(k_full(i), 1);
      mbar_init(k_empty(i), 1);
      mbar_init(v_full(i), 1);
      mbar_init(v_empty(i), 1);
    }
    poisoned = 0;
    fence_barrier_init();
  }
  if (warp == 5) tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t t_o = tmem + 128;                       // O: columns 128 .. 128 + D
  auto t_s = [&](int i) { return tmem + 64u * i; };      // S_i, then P_i: hi 32 columns, lo 32
  auto timeout = [&] { record_error(&g_rows_error, PK_DEVERR_TIMEOUT, s); };

  if (warp == 4) {
    // ---------------- producer ----------------
    if (lane == 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
    const int32_t *trow = p.tables + size_t(s) * p.max_blocks + start / BS;
    const int nb = (end - start + BS - 1) / BS;
    const int mine = min(lane, S::BPT - 1);
    auto entry = [&](int j) { return j * S::BPT + mine < nb ? __ldg(trow + j * S::BPT + mine) : 0; };
    // One tile's K (or V) blocks into its ring's slot.
    auto load = [&](const CUtensorMap *map, uint32_t ring, uint32_t full, int j, int phys) {
      const int nblk = min(S::BPT, nb - j * S::BPT);
      if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(nblk * S::SLABS * BS * 128));
      __syncwarp();
      if (lane < nblk) {
        if (phys < 0 || phys >= p.num_blocks) {
          record_error(&g_rows_error, PK_DEVERR_BLOCK_ID, s);
          phys = 0;  // stay in bounds and keep the byte count; the result is flagged
        }
        const uint32_t dst = ring + (j % STAGES) * S::KV_BYTES + lane * BS * 128;
#pragma unroll
        for (int h = 0; h < S::SLABS; ++h)
          tma_load_3d(dst + h * S::KV_SLAB, map, full, h * 64, kvh, phys * BS);
      }
    };
    // K runs one tile ahead of V: its slots come free earlier.
    int cur = entry(0), nxt = entry(1);
    int kdone = 0, vdone = 0;
    load(&kmap, k_sm, k_full(0), 0, cur);
    kdone = 1;
    for (int j = 0; j < nt; ++j) {
      const int after = entry(j + 2);
      if (j + 1 < nt) {
        const int i = j + 1;
        if (i >= STAGES && !mbar_wait(k_empty(i % STAGES), ((i / STAGES) - 1) & 1)) {
          if (lane == 0) timeout();
          break;
        }
        load(&kmap, k_sm, k_full(i % STAGES), i, nxt);
        kdone = i + 1;
      }
      if (j >= STAGES && !mbar_wait(v_empty(j % STAGES), ((j / STAGES) - 1) & 1)) {
        if (lane == 0) timeout();
        break;
      }
      load(&vmap, v_sm, v_full(j % STAGES), j, cur);
      vdone = j + 1;
      cur = nxt;
      nxt = after;
    }
    // Let every issued copy land before the warp leaves.
    for (int j = max(0, kdone - STAGES); j < kdone; ++j) mbar_wait(k_full(j % STAGES), (j / STAGES) & 1);
    for (int j = max(0, vdone - STAGES); j < vdone; ++j) mbar_wait(v_full(j % STAGES), (j / STAGES) & 1);
  } else if (warp == 5) {
    // ---------------- products ----------------
    if (lane == 0) {
      constexpr uint32_t S_DESC = mma_desc(kRows, kTile, false), O_DESC = mma_desc(kRows, D, true);
      bool ok = mbar_wait(q_ready, 0);
      int issued = 0;  // P V products
      auto pv = [&](int j) {
        const int slot = j % STAGES;
        ok = ok && mbar_wait(p_full(j & 1), (j >> 1) & 1) && mbar_wait(v_full(slot), (j / STAGES) & 1);
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            tc_mma_ts(t_o, t_s(j & 1) + 32 * part + 8 * ks,
                      smem_desc(v_sm + slot * S::KV_BYTES + ks * 2048, S::KV_SLAB, 1024), O_DESC,
                      j > 0 || part > 0 || ks > 0);
        tc_commit(v_empty(slot));
        tc_commit(o_done(j & 1));
        issued = j + 1;
      };
      for (int j = 0; j < nt && ok; ++j) {
        const int slot = j % STAGES;
        // The score tile holds the weights of tile j - 2 until their product ends.
        ok = mbar_wait(k_full(slot), (j / STAGES) & 1) && (j < 2 || mbar_wait(o_done(j & 1), ((j >> 1) - 1) & 1));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_ss(t_s(j & 1), smem_desc(q_sm + (ks / 4) * S::Q_SLAB + (ks % 4) * 32, 16, 1024),
                    smem_desc(k_sm + slot * S::KV_BYTES + (ks / 4) * S::KV_SLAB + (ks % 4) * 32, 16, 1024),
                    S_DESC, ks > 0);
        tc_commit(k_empty(slot));
        tc_commit(s_full(j & 1));
        if (j > 0) pv(j - 1);
      }
      if (ok) pv(nt - 1);
      if (!ok) timeout();
      // Nothing of the tensor cores' is under way when tensor memory is freed.
      for (int j = max(0, issued - 2); j < issued; ++j) mbar_wait(o_done(j & 1), (j >> 1) & 1);
    }
    __syncwarp();
  } else {
    // ---------------- softmax: a thread is a row ----------------
    const int r = threadIdx.x;
    // A negative scale turns the queries' signs, so that scores order as the
    // products do.
    const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;
    for (int i = r; i < kRows * (D / 8); i += 128) {
      const int row = i / (D / 8), c = i % (D / 8);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (row < rows)
        x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + q_row(row) + c * 8));
      x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
      const uint32_t a = q_sm + (c >> 3) * S::Q_SLAB + row * 128 + (((c & 7) ^ (row & 7)) << 4);
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                   : "memory");
    }
    fence_proxy_async();
    mbar_arrive(q_ready);
    if (warp < active) {
      const uint32_t lane_base = uint32_t(warp * 32) << 16;
      const uint64_t mask = r < rows ? draft_mask(p, sr.q0, (r0 + r) / G, sr.n) : 0;
      const float sl = fabsf(p.scale_log2);
      float ref = -INFINITY, l = 0.0f;  // the exponent's reference (scaled scores), the sum
      bool ok = true;
      // A wait of the whole warp (which converges on it): tensor memory is
      // accessed by whole warps.
      auto wait = [&](uint32_t b, uint32_t parity) {
        const bool done = __all_sync(0xffffffffu, mbar_wait(b, parity));
        if (!done && lane == 0) timeout();
        return done;
      };
      const int lim = min(base, end);  // tokens before it are seen by every row
      for (int j = 0; j < nt; ++j) {
        const int t0 = start + j * kTile;
        const bool careful = t0 + kTile > lim;
        if (!(ok = wait(s_full(j & 1), (j >> 1) & 1))) break;
        tc_fence_after();
        uint32_t x[2][32];
        tmem_load32(t_s(j & 1) + lane_base, x[0]);
        tmem_load32(t_s(j & 1) + lane_base + 32, x[1]);
        if (careful) {
          // Drafts, or the partition's end: what a row does not see is masked, the
          // values past the end are zeroed, and so is what is not finite in the
          // drafts' values, which would reach rows that do not see it (0 * NaN);
          // the rows that do see it get it at the end.
          if (!(ok = wait(v_full(j % STAGES), (j / STAGES) & 1))) break;
          const uint32_t vb = v_sm + (j % STAGES) * S::KV_BYTES;
          const int first = max(0, lim - t0), valid = min(kTile, end - t0);
          for (int i = first * (D / 8) + int(threadIdx.x); i < kTile * (D / 8); i += active * 32) {
            const int row = i / (D / 8), c = i % (D / 8);
            const uint32_t a = vb + (c >> 3) * S::KV_SLAB + row * 128 + (c & 7) * 16;
            uint32_t w[4] = {0, 0, 0, 0};
            bool dirty = row >= valid;
            if (!dirty) {
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                           : "r"(a));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u, dirty = true;
                if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu, dirty = true;
              }
              if (dirty) poisoned = 1;
            }
            if (dirty)
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                           "r"(w[3])
                           : "memory");
          }
          fence_proxy_async();
        }
        tmem_wait_load(x[0]);
        tmem_wait_load(x[1]);
        if (careful) {
          const uint64_t see = see64(mask, base, t0);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w = uint32_t(see >> (32 * h));
            const int live = end - t0 - 32 * h;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((w >> i) & 1) || i >= live) x[h][i] = 0xff800000u;  // -inf
          }
        }
        float mx = -INFINITY;
        {
          float part[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; ++i)
            part[i & 3] = max3(part[i & 3], __uint_as_float(x[i >> 4][2 * (i & 15)]),
                               __uint_as_float(x[i >> 4][2 * (i & 15) + 1]));
          mx = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])) * sl;
        }
        const bool move = mx > ref + kSlack;
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? exp2_ftz(ref - mx) : 1.0f;
          if (move) ref = mx;
          const uint64_t f2 = pack2(f, f);
          l *= f;
          if (j > 0) {
            if (!(ok = wait(o_done((j - 1) & 1), ((j - 1) >> 1) & 1))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_load32(t_o + lane_base + 32 * c, o);
              tmem_wait_load(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float a, b;
                unpack2(mul2(pack2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), f2), a, b);
                o[2 * i] = __float_as_uint(a);
                o[2 * i + 1] = __float_as_uint(b);
              }
              tmem_store32(t_o + lane_base + 32 * c, o);
            }
          }
        }
        const float m = ref == -INFINITY ? 0.0f : ref;  // nothing seen so far: every weight is 0
        const uint64_t sl2 = pack2(sl, sl), m2 = pack2(-m, -m), minus = pack2(-1.0f, -1.0f);
        uint64_t sum2 = 0;
        uint32_t hi[32], lo[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float a, b;
          unpack2(fma2(pack2(__uint_as_float(x[i >> 4][2 * (i & 15)]), __uint_as_float(x[i >> 4][2 * (i & 15) + 1])),
                       sl2, m2),
                  a, b);
          a = exp2_ftz(a);
          b = exp2_ftz(b);
          const uint64_t ab = pack2(a, b);
          sum2 = add2(sum2, ab);
          hi[i] = pack_bf16x2(a, b);
          unpack2(fma2(pack2(bf16_lo(hi[i]), bf16_hi(hi[i])), minus, ab), a, b);
          lo[i] = pack_bf16x2(a, b);
        }
        {
          float a, b;
          unpack2(sum2, a, b);
          l += a + b;
        }
        tmem_store32(t_s(j & 1) + lane_base, hi);
        tmem_store32(t_s(j & 1) + lane_base + 32, lo);
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(j & 1));
      }
      ok = ok && wait(o_done((nt - 1) & 1), ((nt - 1) >> 1) & 1);
      tc_fence_after();
      named_barrier(1, active * 32);  // every warp's part of `poisoned` is in
      if (ok) {
        const bool split = sr.np > 1;
        const float inv = split ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
        const size_t at = r < rows ? q_row(r) : 0;
        const size_t slot = at / D * p.num_partitions + part;
        const bool fix = poisoned;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_load32(t_o + lane_base + 32 * c, o);
          tmem_wait_load(o);
          if (fix && r < rows) {
            for (int t = max(base, start); t < end; ++t) {
              if (!((mask >> (t - base)) & 1)) continue;
              const int phys = __ldg(p.tables + size_t(s) * p.max_blocks + t / BS);
              if (phys < 0 || phys >= p.num_blocks) continue;
              const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v_cache) +
                                       ((size_t(phys) * BS + t % BS) * p.num_kv_heads + kvh) * D + 32 * c;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = __bfloat162float(v[i]);
                if (!(fabsf(y) <= 3.402823466e38f)) o[i] = __float_as_uint(__uint_as_float(o[i]) + y);
              }
            }
          }
          if (split && r < rows) {
            float4 *dst = reinterpret_cast<float4 *>(p.ws_acc + slot * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                   __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          } else if (r < rows) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at + 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * e]) * inv, __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
              dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
        }
        if (split && r < rows) {
          p.ws_m[slot] = ref;
          p.ws_l[slot] = l;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_free(tmem, kTmemCols);
  }
}

template <int D, int BS>
pk_status launch_tree(RowsParams p, const pk_cache_desc &d, cudaStream_t stream) {
  using S = TreeShape<D, BS>;
  CUtensorMap kmap, vmap;
  if (!encode_bf16_pool(&kmap, p.k_cache, d) || !encode_bf16_pool(&vmap, p.v_cache, d)) return PK_ERR_CUDA;
  auto kern = attn_tree_kernel<D, BS>;
  static std::atomic<uint64_t> ready{0};
  if (!smem_ready(kern, S::SMEM_BYTES, ready)) return PK_ERR_CUDA;
  p.row_tiles = (p.max_draft * p.group + kRows - 1) / kRows;
  kern<<<rows_grid(p), kThreads, S::SMEM_BYTES, stream>>>(p, kmap, vmap);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

template <int D>
pk_status launch_tree_d(const RowsParams &p, const pk_cache_desc &d, cudaStream_t stream) {
  return d.block_size == 8    ? launch_tree<D, 8>(p, d, stream)
         : d.block_size == 16 ? launch_tree<D, 16>(p, d, stream)
                              : launch_tree<D, 32>(p, d, stream);
}

// fp32 pools, and bf16 ones of other block sizes, on CUDA cores.
template <typename T, int D>
pk_status run(const RowsParams &p, const pk_cache_desc &d, cudaStream_t stream) {
  pk_status st;
  if (sizeof(T) == 2 && (d.block_size == 8 || d.block_size == 16 || d.block_size == 32))
    st = launch_tree_d<D>(p, d, stream);
  else
    st = p.max_draft * p.group <= 8 ? launch_rows<T, T, D, 1>(p, stream)
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
    return desc->head_dim == 128 ? run<float, 128>(p, *desc, s) : run<float, 64>(p, *desc, s);
  return desc->head_dim == 128 ? run<__nv_bfloat16, 128>(p, *desc, s)
                               : run<__nv_bfloat16, 64>(p, *desc, s);
}

}  // extern "C"

}  // namespace pk
