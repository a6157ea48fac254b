// Prompts and chunks of bf16 on tcgen05 (attn_prompt_kernel): pk_paged_attention_extend
// for sequences of more than eight rows.
//
// n new tokens are n G rows of query a KV head, and a row has 4 d operations for each token
// that it sees: from some 300 rows on the tensor cores bound it. A CTA has 256 rows, two
// halves of 128, one lane of tensor memory each, and goes over its keys in tiles of 128:
//   producer warp    TMA loads of the blocks' K and V tiles, in turn, into a ring of 128 KB;
//   a half's warp    O += P V, then the next tile's S = Q K^T, all in tensor memory (S 128
//                    columns, P over it, O 128: 512 for both halves, so a CTA an SM);
//   softmax warps    four a half, a thread a row: cap, bias and mask, the running maximum and
//                    sum, weights as bf16 over the scores. A row's reference of the exponent
//                    moves only when the maximum has outgrown it by 2^8, so O is rescaled a few
//                    times a row;
//   units' warp      units (256 rows of a sequence and KV head over a partition) by launch
//                    control, the next one before this one's last tiles;
//   four warps       queries of the next unit, and hidden values that are not finite cleared.
// Only tiles that some row does not see as a whole are masked.
//
// Measured (32 / 8 heads of 128): one prompt of 16 384 tokens 1.42 ms, 1.55 PFLOP/s of the
// formula's work (scores capped 1.70 ms, biased 1.91; heads of 64 1.05); eight of 2000 261 us;
// the last 512 tokens of two contexts of 32 768, 64 / 8 heads, capped, 953 us, 1.14 PFLOP/s.
// What bounds it now: long, a tile's chain in a half (1370 cycles of softmax, 1140 of products,
// 680 of waits between them) with two halves to overlap it: a tile takes 3200 cycles, 2050 of
// them products; capped, the softmax's operations; short, a unit's beginning and end, some
// four microseconds in which the tensor cores idle.
#pragma once

#include <cuda.h>

#include "attn_extend.cuh"
#include "pk_tcgen05.cuh"
#include "pk_tma_host.h"

namespace pk {
namespace {

constexpr int kPromptRows = 256;     // of a unit: two halves of 128, one lane of tensor memory each
constexpr int kPromptTile = 128;     // tokens
// Two warpgroups of softmax; the producer, a half's products, units, the other half's
// products; four warps that bring queries and look after values.
constexpr int kPromptThreads = 512;
constexpr int kPromptUnits = 4;      // units known at a time
// 512 threads of 128 registers at launch: 2 x 200 + 2 x 56 = 4 x 128.
constexpr int kPromptSoftmaxRegs = 200, kPromptOtherRegs = 56;
// Scores (of which the reference) up to which they are scaled in one operation with the subtraction.
constexpr float kPromptExact = 1048576.0f;
constexpr float kPromptSlack = 8.0f;  // log2 of how far a maximum may outgrow the reference

template <int D>
struct PromptShape {
  static constexpr int SLABS = D / 64;                   // 128-byte column slabs
  static constexpr int SLAB = 128 * 128;                 // of 128 rows
  static constexpr int Q_HALF = SLABS * SLAB, TILE = SLABS * SLAB;
  static constexpr int STAGES = D == 128 ? 4 : 8;        // tiles of K and V in flight
  static constexpr int OUT_BYTES = 4096;                 // per softmax warp: 128 bytes of each of its rows
  static constexpr int SMEM_BYTES = 1024 + 2 * Q_HALF + STAGES * TILE + 8 * OUT_BYTES;
};

// tanh of two values times `k` / (2 log2(e)): 1 - 2 / (1 + 2^(k x)). The error is absolute, 2^-21
// or so, whatever the value.
__device__ __forceinline__ uint64_t tanh2(uint64_t x, uint64_t k) {
  float a, b;
  unpack2(mul2(x, k), a, b);
  a = reciprocal(1.0f + exp2_ftz(a));
  b = reciprocal(1.0f + exp2_ftz(b));
  return fma2(pack2(a, b), pack2(-2.0f, -2.0f), pack2(1.0f, 1.0f));
}
// tanh of two values to 2^-20 of itself: by the polynomial up to kTanhSmall, and as above beyond.
__device__ __forceinline__ uint64_t tanh2_relative(uint64_t y) {
  const uint64_t z = mul2(y, y), t = tanh2(y, pack2(2.0f * 1.44269504f, 2.0f * 1.44269504f));
  uint64_t r = fma2(z, pack2(kTanh4, kTanh4), pack2(kTanh3, kTanh3));
  r = fma2(r, z, pack2(kTanh2, kTanh2));
  r = fma2(r, z, pack2(kTanh1, kTanh1));
  r = mul2(fma2(r, z, pack2(kTanh0, kTanh0)), y);
  float ya, yb, ta, tb, ra, rb;
  unpack2(y, ya, yb);
  unpack2(t, ta, tb);
  unpack2(r, ra, rb);
  return pack2(fabsf(ya) <= kTanhSmall ? ra : ta, fabsf(yb) <= kTanhSmall ? rb : tb);
}
// For |y| <= kTanhTiny tanh(y) = y (t0 + t1 y^2 + t2 y^4) to 2^-17.3 of itself. This polynomial and
// the longer one need no exponential and no reciprocal, whose unit the softmax's own exponentials
// keep busy.
constexpr float kTanhTiny = 0.4f;
constexpr float kTiny0 = 0.9999939203262329f, kTiny1 = -0.3326335847377777f, kTiny2 = 0.12132595479488373f;
// How scores are capped. kNear: the polynomials are of products as they come, their coefficients
// holding up to the eighth power of scale / cap, which has to be a normal number; scores of which
// some reach the cap go through tanh2, whose 2^-21 of the cap is 2^-14 of the exponent at most.
// kWide, any cap: products are scaled first, and such scores go through tanh2_relative, as 2^-21
// of a large cap would be more than the scores far below it (0.7 at 10^6). A prompt of 16 384 tokens
// (32 / 8 heads of 128): 1700 us near and 1800 wide, and where scores reach the cap 2740 and 3570.
enum class Cap { kNone, kNear, kWide };
constexpr float kNearFrom = 6.103515625e-5f, kNearTo = 16384.0f;  // scale / cap
constexpr float kNearCap = 128.0f;                                // cap log2(e)

// A unit of work: up to 256 rows of one (sequence, KV head) over one partition.
struct PromptUnit {
  int s, kvh, part;
  SeqRows sr;
  int r0, rows;
  int start, end, nt;         // its tokens and tiles; s < 0: no more units
  int all_from, all_to;       // the tokens that every row sees
  // Whether some row does not see some token of tile j.
  __device__ __forceinline__ bool careful(int j) const {
    const int t0 = start + j * kPromptTile;
    return t0 < all_from || t0 + kPromptTile > all_to;
  }
  __device__ __forceinline__ int halves() const { return rows > 128 ? 2 : 1; }
};

template <int D, Cap CAP, bool SLOPES>
__global__ void __launch_bounds__(kPromptThreads, 1)
    attn_prompt_kernel(ExtendParams p, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using S = PromptShape<D>;
  constexpr int ST = S::STAGES;
  constexpr bool CAPPED = CAP != Cap::kNone;
  constexpr bool EXACT = CAP != Cap::kNear && !SLOPES;  // scores may be too large for the shorter way
  launch_dependents();  // the merge may be scheduled as this grid drains
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.group;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t q_sm = (smem_addr(smem_raw) + 1023u) & ~1023u, kv_sm = q_sm + 2 * S::Q_HALF;
  constexpr int NB = 3 * ST + 2 * kPromptUnits;
  __shared__ __align__(8) uint64_t bars[NB + 16];
  __shared__ uint4 answer;
  __shared__ PromptUnit units[kPromptUnits];
  __shared__ uint32_t tmem_slot;
  // The unit, plus one, whose values were not all finite where some rows do not see them.
  // Nothing is cleared: a unit's mark is written before its products and read before its
  // softmax warps give its entry back, which comes before the next unit of the same word.
  __shared__ int poisoned[kPromptUnits];
  // Units i, tiles of K and V k, tiles and units of a half are counted over the life of the
  // CTA; a barrier's phase is the count of what uses it. Every wait names a phase of which the
  // one before has ended for certain and the one after cannot have: a wait by parity tells
  // neighbouring phases apart, not more.
  auto bar = [&](int i) { return smem_addr(bars + i); };
  auto kv_full = [&](int k) { return bar(k % ST); };           // the copy has landed
  auto v_ready = [&](int k) { return bar(ST + k % ST); };      // and its values are fit for the product
  auto kv_empty = [&](int k) { return bar(2 * ST + k % ST); };
  auto kv_phase = [](int k) { return uint32_t(k / ST) & 1u; };
  auto u_full = [&](int i) { return bar(3 * ST + i % kPromptUnits); };
  auto u_empty = [&](int i) { return bar(3 * ST + kPromptUnits + i % kPromptUnits); };
  auto u_phase = [](int i) { return uint32_t(i / kPromptUnits) & 1u; };
  auto q_full = [&](int h) { return bar(NB + h); };       // of a half, by unit
  auto q_empty = [&](int h) { return bar(NB + 2 + h); };
  auto o_done = [&](int h) { return bar(NB + 4 + h); };
  auto s_full = [&](int h) { return bar(NB + 6 + h); };   // of a half, by tile
  auto p_full = [&](int h) { return bar(NB + 8 + h); };
  auto turn = [&](int h) { return bar(NB + 10 + h); };    // the other half's products are issued
  auto drained = [&](int h) { return bar(NB + 12 + h); };
  const uint32_t u_want = bar(NB + 14), u_answer = bar(NB + 15);
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(kv_full(i), 1);
      mbar_init(v_ready(i), 4);
      mbar_init(kv_empty(i), 2);
    }
    for (int i = 0; i < kPromptUnits; ++i) {
      mbar_init(u_full(i), 1);
      mbar_init(u_empty(i), 15);  // every warp but the one that fills them
      poisoned[i] = 0;
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(q_full(h), 128);
      mbar_init(q_empty(h), 1);
      mbar_init(o_done(h), 1);
      mbar_init(s_full(h), 1);
      mbar_init(p_full(h), 4);
      mbar_init(turn(h), 1);
      mbar_init(drained(h), 1);
    }
    mbar_init(u_want, 1);
    mbar_init(u_answer, 1);
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(smem_addr(&tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  auto t_s = [&](int h) { return tmem + 128u * h; };                // scores, then weights (64 columns)
  auto t_o = [&](int h) { return tmem + 256u + uint32_t(D) * h; };  // O
  // A wait of the whole warp, which converges on it; once one has failed, so do all.
  auto warp_wait = [](uint32_t b, uint32_t parity, bool &ok) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(b, parity));
    return ok;
  };
  auto release = [&](int i) {  // this warp is done with the unit's entry
    __syncwarp();
    if (lane == 0) mbar_arrive(u_empty(i));
  };
  auto timeout = [&] { record_error(&g_rows_error, PK_DEVERR_TIMEOUT, blockIdx.x); };
  auto q_row = [&](const SeqRows &sr, int kvh, int row) {  // element offset of a row of q and out
    return (size_t(sr.q0 + row / G) * p.num_q_heads + kvh * G + row % G) * D;
  };

  if (warp >= 8) {
    setmaxnreg_dec<kPromptOtherRegs>();
    if (warp == 8) {
      // ---------------- producer: K and V tiles in turn ----------------
      if (lane == 0) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
      }
      const int BS = p.block_size, per = kPromptTile / BS;
      bool ok = true;
      int k = 0;  // tiles of K and V
      for (int i = 0; warp_wait(u_full(i), u_phase(i), ok); ++i) {
        const PromptUnit &c = units[i % kPromptUnits];
        const int s = c.s, kvh = c.kvh, nt = c.nt, nb = (c.end - c.start + BS - 1) / BS;
        const int32_t *row = p.tables + size_t(max(s, 0)) * p.max_blocks + c.start / BS;
        release(i);
        if (s < 0) break;
        auto entry = [&](int j) {  // the lane's block of tile j
          const int b = j * per + lane;
          int phys = lane < per && b < nb ? __ldg(row + b) : 0;
          if (phys < 0 || phys >= p.num_blocks) {
            record_error(&g_rows_error, PK_DEVERR_BLOCK_ID, s);
            phys = 0;  // stay in bounds and keep the byte count; the result is flagged
          }
          return phys;
        };
        int next = entry(0);
        for (int j = 0; ok && j < nt; ++j) {
          // The unit after this one is asked for three tiles before the end: early enough
          // to be here in time, late enough to go to the CTA that is free first.
          if (j == max(0, nt - 3) && lane == 0) mbar_arrive(u_want);
          const int phys = next, nblk = min(per, nb - j * per);
          next = entry(j + 1);
          for (int side = 0; side < 2; ++side, ++k) {
            if (k >= ST && !warp_wait(kv_empty(k), kv_phase(k - ST), ok)) break;
            if (lane == 0) mbar_arrive_expect_tx(kv_full(k), uint32_t(nblk * S::SLABS * BS * 128));
            __syncwarp();
            if (lane < nblk) {
              const uint32_t dst = kv_sm + k % ST * S::TILE + lane * BS * 128;
#pragma unroll
              for (int x = 0; x < S::SLABS; ++x)
                tma_load_3d(dst + x * S::SLAB, side ? &vmap : &kmap, kv_full(k), x * 64, kvh, phys * BS);
            }
          }
        }
      }
      if (!ok && lane == 0) timeout();
      // Let every issued copy land before the warp leaves.
      for (int x = max(0, k - ST); x < k; ++x) mbar_wait(kv_full(x), kv_phase(x));
    } else if (warp == 9 || warp == 11) {
      // ---------------- products of a half ----------------
      // S of the first tile, then in turn O += P V and the next tile's S: while one half's
      // softmax runs, the tensor cores have the other's products. A warp for each, as a wait
      // costs some 200 cycles even where its phase has ended, and in one warp the waits and
      // issues of both took longer than the products (3550 cycles a tile). The two take turns:
      // products of both that are issued together end together, and then both halves are in
      // their softmax at once and the tensor cores idle (3400 cycles; now 3200). Heads of 64 have
      // half the products, and turns only hold them up (1140 us for 1030).
      constexpr bool TURNS = D == 128;
      constexpr uint32_t O_DESC = mma_desc(128, D, true);
      const uint32_t s_desc = mma_desc(128, kPromptTile, false) | (p.factor < 0.0f ? 1u << 13 : 0u);  // -Q
      const int h = (warp - 9) / 2;
      const uint64_t q_d = smem_desc(q_sm + h * S::Q_HALF, 16, 1024);
      bool ok = true;
      int k0 = 0, n = 0, done = 0, m = 0;  // tiles of K and V before the unit, tiles of the half, its units, turns
      for (int i = 0; warp_wait(u_full(i), u_phase(i), ok); ++i) {
        const PromptUnit &unit = units[i % kPromptUnits];
        const int s = unit.s, nt = unit.nt, halves = unit.halves();
        release(i);
        if (s < 0) break;
        if (h >= halves) {  // the other half has it alone
          k0 += 2 * nt;
          continue;
        }
        auto my_turn = [&] { return !TURNS || halves == 1 || (h == 0 && m == 0) || warp_wait(turn(h), (m - (h == 0)) & 1, ok); };
        // O += P V of tile j and S of the next (j < 0: only that).
        auto products = [&](int j) {
          if (elect_one()) {
            if (j >= 0) {
              const int k = k0 + 2 * j + 1;
              const uint64_t b = smem_desc(kv_sm + k % ST * S::TILE, S::SLAB, 1024);
#pragma unroll
              for (int ks = 0; ks < kPromptTile / 16; ++ks)  // a descriptor's address counts 16 bytes
                tc_mma_ts(t_o(h), t_s(h) + 8 * ks, b + ks * 128, O_DESC, j > 0 || ks > 0);
              tc_commit(kv_empty(k));
              if (halves == 1) tc_commit(kv_empty(k));  // for the other half
              if (j + 1 == nt) tc_commit(o_done(h));
            }
            if (j + 1 < nt) {
              const int k = k0 + 2 * j + 2;
              const uint64_t b = smem_desc(kv_sm + k % ST * S::TILE, 16, 1024);
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)
                tc_mma_ss(t_s(h), q_d + (ks / 4) * (S::SLAB / 16) + (ks % 4) * 2,
                          b + (ks / 4) * (S::SLAB / 16) + (ks % 4) * 2, s_desc, ks > 0);
              tc_commit(s_full(h));
              tc_commit(kv_empty(k));
              if (halves == 1) tc_commit(kv_empty(k));
              if (j + 2 == nt) tc_commit(q_empty(h));
            }
            if (TURNS && halves == 2) mbar_arrive(turn(1 - h));
          }
          __syncwarp();
          m += halves == 2;
        };
        if (!warp_wait(q_full(h), done++ & 1, ok) || !warp_wait(kv_full(k0), kv_phase(k0), ok) || !my_turn()) break;
        tc_fence_after();
        products(-1);
        for (int j = 0; j < nt; ++j, ++n) {
          const int iv = k0 + 2 * j + 1, ik = iv + 1;
          if (!warp_wait(v_ready(iv), kv_phase(iv), ok) || (j + 1 < nt && !warp_wait(kv_full(ik), kv_phase(ik), ok)) ||
              !my_turn() || !warp_wait(p_full(h), n & 1, ok))
            break;
          tc_fence_after();
          products(j);
        }
        if (!ok) break;
        k0 += 2 * nt;
      }
      if (!ok && lane == 0) timeout();
      // Nothing of this warp's products is under way when tensor memory is freed.
      if (elect_one()) tc_commit(drained(h));
      __syncwarp();
      mbar_wait(drained(h), 0);
      __syncwarp();
    } else if (warp == 10) {
      // ---------------- units ----------------
      // The grid has a CTA per unit; those that find no room are taken over, one at a time,
      // by whichever CTA needs work next (the list is longest first).
      bool ok = true;
      int published = 0;
      auto publish = [&](const PromptUnit &c) {
        const int i = published;
        if (i >= kPromptUnits && !warp_wait(u_empty(i), u_phase(i - kPromptUnits), ok)) return;
        if (lane == 0) {
          units[i % kPromptUnits] = c;
          mbar_arrive(u_full(i));
        }
        ++published;
      };
      for (int cta = blockIdx.x, asked = 0; cta >= 0;) {
        SplitUnit u;
        bool work = extend_unit(p, cta, kPromptRows, lane == 0, u), zero = work && u.void_rows;
        PromptUnit c;
        if (work && !zero) {
          // What the unit's rows see between them, and what all see.
          int from = INT32_MAX, to = 0, af = 0, at = INT32_MAX;
          for (int r = lane; r < u.rows; r += 32) {
            const RowSpan x = row_span(p, u.sr, u.s, (u.r0 + r) / G);
            const bool some = x.lo < x.hi;
            if (some) from = min(from, x.lo), to = max(to, x.hi);
            af = max(af, some ? x.lo : INT32_MAX), at = min(at, some ? x.hi : 0);
          }
          from = __reduce_min_sync(0xffffffffu, from), to = __reduce_max_sync(0xffffffffu, to);
          af = __reduce_max_sync(0xffffffffu, af), at = __reduce_min_sync(0xffffffffu, at);
          if (!extend_tokens(p, u, from, to)) work = false, zero = p.num_partitions == 1;
          c.all_from = af, c.all_to = min(at, u.end);
        }
        if (zero) {
          for (int k = lane; k < u.rows * (D / 8); k += 32)
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + q_row(u.sr, u.kvh, u.r0 + k / (D / 8)) +
                                       k % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
        } else if (work) {
          c.s = u.s, c.kvh = u.kvh, c.part = u.part, c.sr = u.sr, c.r0 = u.r0, c.rows = u.rows;
          c.start = u.start, c.end = u.end, c.nt = (u.end - u.start + kPromptTile - 1) / kPromptTile;
          publish(c);
          if (!ok || !warp_wait(u_want, (published - 1) & 1, ok)) break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(u_answer, 16);
          try_cancel(smem_addr(&answer), u_answer);
        }
        if (!warp_wait(u_answer, asked & 1, ok)) break;
        ++asked;
        cta = cancelled_cta(smem_addr(&answer));
        fence_answer_read();
        __syncwarp();
      }
      PromptUnit end{};
      end.s = -1;
      if (ok) publish(end);
      if (!ok && lane == 0) timeout();
    } else {
      // ---------------- queries and values ----------------
      // These warps bring a half's queries once the scores of the unit before are done with the
      // last ones, and look at each tile of values that has landed: rows past the end are
      // zeroed, and so is what is not finite in values that some rows do not see, which would
      // reach those too (0 * NaN); the rows that do see it get it at the end. A half's queries
      // are there when all four warps are past the unit before, so that no wait for values
      // can be a phase early.
      const int w = warp - 12;
      constexpr int CH = D / 8;  // chunks of a row
      const uint32_t inv_g = (65536 + G - 1) / G;  // x / G = x inv_g >> 16 for x < 512
      bool ok = true;
      int k0 = 0, done[2] = {0, 0};
      for (int i = 0; warp_wait(u_full(i), u_phase(i), ok); ++i) {
        const PromptUnit &c = units[i % kPromptUnits];
        if (c.s < 0) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= c.halves() || (done[h] > 0 && !warp_wait(q_empty(h), (done[h] - 1) & 1, ok))) break;
          ++done[h];
          // Rows past the last keep what is there: no row's result depends on another's query.
          constexpr int STEP = 128 / CH;  // rows at once
          const int t = tid & 127, ch = t % CH, tok0 = c.r0 / G, rows = min(128, c.rows - 128 * h);
          const uint32_t x0 = c.r0 % G + 128 * h;
          const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) +
                                     (size_t(c.sr.q0 + tok0) * p.num_q_heads + c.kvh * G) * D + ch * 8;
          const uint32_t dst = q_sm + h * S::Q_HALF + (ch >> 3) * S::SLAB;
#pragma unroll 4
          for (int row = t / CH; row < rows; row += STEP) {
            const uint32_t x = x0 + row, tok = x * inv_g >> 16;
            cp_async16(dst + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                       src + (size_t(tok) * (p.num_q_heads - G) + x) * D, 16);
          }
          cp_async_wait();
          fence_proxy_async_shared();
          mbar_arrive(q_full(h));
        }
        const int nt = c.nt;
        for (int j = 0; ok && j < nt; ++j) {
          const int iv = k0 + 2 * j + 1;
          if (!warp_wait(kv_full(iv), kv_phase(iv), ok)) break;
          if (c.careful(j)) {
            const int t0 = c.start + j * kPromptTile, valid = min(kPromptTile, c.end - t0);
            const int all_from = c.all_from - t0, all_to = c.all_to - t0;
            const int ch = lane % CH;
            const uint32_t at = kv_sm + iv % ST * S::TILE + (ch >> 3) * S::SLAB + (ch & 7) * 16;
            bool wrote = false;
            constexpr int STEP = 32 / CH;  // rows at once
            const int first = 32 * w + lane / CH, last = 32 * w + 32;
            for (int k = first; k < last; k += STEP)
              if (k >= valid) {
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + k * 128), "r"(0) : "memory");
                wrote = true;
              }
            if (32 * w < all_from || 32 * w + 32 > all_to) {  // some of the warp's rows are hidden from some
              // Four rows' chunks at once; they are looked at one by one only if a carry into a
              // half's sign shows an exponent of all ones.
#pragma unroll 1
              for (int k0 = first; k0 < min(last, valid); k0 += 4 * STEP) {
                uint32_t v[4][4], odd = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const int k = k0 + u * STEP;
                  v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0;
                  if (k < valid && (k < all_from || k >= all_to))
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[u][0]), "=r"(v[u][1]), "=r"(v[u][2]), "=r"(v[u][3])
                                 : "r"(at + k * 128));
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                  for (int e = 0; e < 4; ++e) odd |= (v[u][e] & 0x7f807f80u) + 0x00800080u;
                if (!(odd & 0x80008000u)) continue;
                poisoned[i % kPromptUnits] = i + 1;
                wrote = true;
#pragma unroll 1
                for (int u = 0; u < 4; ++u) {
                  const int k = k0 + u * STEP;
                  if (k >= valid || (k >= all_from && k < all_to)) continue;
#pragma unroll 1
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t a = at + k * 128 + 4 * e;
                    uint32_t x;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(a));
                    if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
                    if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
                  }
                }
              }
            }
            if (__any_sync(0xffffffffu, wrote)) fence_proxy_async_shared();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(v_ready(iv));
        }
        if (!ok) break;
        k0 += 2 * nt;
        release(i);
      }
      if (!ok && lane == 0) timeout();
    }
  } else {
    // ---------------- softmax: a thread is a row ----------------
    setmaxnreg_inc<kPromptSoftmaxRegs>();
    const int h = warp >> 2;
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    // In the exponent's scale. At least the smallest normal number: a scale of 0 must not
    // turn the -inf of what is masked into NaN.
    const float fac0 = fmaxf(fabsf(p.factor), 1.17549435e-38f), fac = CAP == Cap::kWide ? 1.0f : fac0;
    const float sl = SLOPES ? 1.0f : (CAPPED ? p.cap_log2 : fac);
    // The polynomial of a product, in the exponent's scale.
    const float f1 = p.cap_log2 * fac, ff = fac * fac;
    const float tc[5] = {kTanh0 * f1, kTanh1 * f1 * ff, kTanh2 * f1 * ff * ff, kTanh3 * f1 * ff * ff * ff,
                         kTanh4 * f1 * ff * ff * ff * ff};
    const float tt[3] = {kTiny0 * f1, kTiny1 * f1 * ff, kTiny2 * f1 * ff * ff};
    bool ok = true;
    int n = 0, done = 0;  // the half's tiles and units
    for (int i = 0; warp_wait(u_full(i), u_phase(i), ok); ++i) {
      const PromptUnit &unit = units[i % kPromptUnits];
      if (unit.s < 0) break;
      const int nt = unit.nt, start = unit.start, end = unit.end, halves = unit.halves(), rows = unit.rows;
      if (h >= halves) {  // the other half has it alone
        release(i);
        continue;
      }
      const bool busy = warp * 32 < rows;  // this warp has rows
      RowSpan x{0, 0, 0};
      float slope = 0.0f;
      if (tid < rows) {
        x = row_span(p, unit.sr, unit.s, (unit.r0 + tid) / G);
        if (SLOPES) slope = __ldg(p.slopes + unit.kvh * G + (unit.r0 + tid) % G) * 1.44269504f;
      }
      float ref = -INFINITY, l = 0.0f;  // the exponent's reference (scaled scores), the sum
      bool exact = false;               // a reference of the warp's is above kPromptExact
      for (int j = 0; j < nt; ++j, ++n) {
        const int t0 = start + j * kPromptTile;
        const bool careful = unit.careful(j);
        uint32_t s[4][32];
        if (!warp_wait(s_full(h), n & 1, ok)) break;
        tc_fence_after();
        if (busy) {
#pragma unroll
          for (int e = 0; e < 4; ++e) tmem_load32(t_s(h) + lane_base + 32 * e, s[e]);
#pragma unroll
          for (int e = 0; e < 4; ++e) tmem_wait_load(s[e]);
          auto pair = [&](int i) {
            return pack2(__uint_as_float(s[i / 16][2 * (i % 16)]), __uint_as_float(s[i / 16][2 * (i % 16) + 1]));
          };
          auto set_pair = [&](int i, uint64_t v) {
            float a, b;
            unpack2(v, a, b);
            s[i / 16][2 * (i % 16)] = __float_as_uint(a), s[i / 16][2 * (i % 16) + 1] = __float_as_uint(b);
          };
          auto largest = [&](auto of) {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 64; ++i)
              top[i & 3] = max3(top[i & 3], of(__uint_as_float(s[i / 16][2 * (i % 16)])),
                                of(__uint_as_float(s[i / 16][2 * (i % 16) + 1])));
            return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          };
          auto hide = [&](uint32_t with) {  // the scores of tokens that the row does not see
            const int lo = max(0, x.lo - t0), hi = min(x.hi, end) - t0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int a = min(max(lo - 32 * e, 0), 32), b = min(max(hi - 32 * e, 0), 32);  // columns a .. b - 1 seen
              const uint32_t see = (b == 32 ? ~0u : (1u << b) - 1) & (a == 32 ? 0u : ~0u << a);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(see & (1u << k))) s[e][k] = with;
            }
          };
          // Small scores are capped by a polynomial, together with the subtraction of the
          // reference where no bias comes between; others by exponentials, in place.
          float most = 0.0f;  // the largest magnitude
          bool poly = false, tiny = false;
          if (CAPPED) {
            // Of what is seen, by rows that there are: the others hold what units before have left,
            // which differs from call to call, and must not choose the way of a result.
            if (CAP == Cap::kWide)
#pragma unroll
              for (int i = 0; i < 64; ++i) set_pair(i, mul2(pair(i), pack2(fac0, fac0)));
            if (careful) hide(0);
            most = tid < rows ? largest([](float v) { return fabsf(v); }) : 0.0f;
            poly = __all_sync(0xffffffffu, most * fac <= kTanhSmall && (CAP == Cap::kNear || most * f1 <= kPromptExact));
            tiny = !SLOPES && __all_sync(0xffffffffu, most * fac <= kTanhTiny) && poly;
            if (!poly) {
              const uint64_t k2 = pack2(2.0f * 1.44269504f * fac, 2.0f * 1.44269504f * fac);
#pragma unroll
              for (int i = 0; i < 64; ++i) set_pair(i, CAP == Cap::kNear ? tanh2(pair(i), k2) : tanh2_relative(pair(i)));
            }
          }
          // The polynomials' sums without the last factor.
          auto capped = [&](int i) {
            const uint64_t x = pair(i), z = mul2(x, x);
            uint64_t r = fma2(z, pack2(tc[4], tc[4]), pack2(tc[3], tc[3]));
            r = fma2(r, z, pack2(tc[2], tc[2]));
            r = fma2(r, z, pack2(tc[1], tc[1]));
            return fma2(r, z, pack2(tc[0], tc[0]));
          };
          auto capped_tiny = [&](int i) {
            const uint64_t x = pair(i), z = mul2(x, x);
            return fma2(fma2(z, pack2(tt[2], tt[2]), pack2(tt[1], tt[1])), z, pack2(tt[0], tt[0]));
          };
          if (SLOPES) {
            const float d0 = float(t0 - x.pos), f = CAPPED ? p.cap_log2 : fac;
            const uint64_t f2 = pack2(f, f), m2 = pack2(-slope, -slope);
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              const uint64_t away =
                  add2(pack2(d0, d0), pack2(float(2 * i), float(2 * i + 1))) & 0x7fffffff7fffffffull;
              set_pair(i, fma2(away, m2, CAPPED && poly ? mul2(capped(i), pair(i)) : mul2(pair(i), f2)));
            }
          }
          float sl_now = sl;
          if (CAPPED && !SLOPES && poly && careful) {  // ahead of the mask, whose -inf is no factor of a polynomial
#pragma unroll
            for (int i = 0; i < 64; ++i) set_pair(i, mul2(capped(i), pair(i)));
            sl_now = 1.0f;
            poly = tiny = false;
          }
          if (careful) hide(0xff800000u);  // -inf
          float mx;
          if (CAPPED && !SLOPES && poly && __all_sync(0xffffffffu, most * f1 <= 30.0f)) {
            // Every score is seen and between -30 and 30 in the exponent, so the largest magnitude
            // serves as a reference: no weight that counts is below 2^-60, and a search for
            // the maximum is saved.
            mx = most * f1;
          } else {
            mx = largest([](float v) { return v; });
            if (CAPPED && !SLOPES && poly) {
              const float z = mx * mx;
              mx = mx == -INFINITY ? mx : mx * fmaf(fmaf(fmaf(fmaf(tc[4], z, tc[3]), z, tc[2]), z, tc[1]), z, tc[0]);
            } else {
              mx = mx == -INFINITY ? mx : mx * sl_now;
            }
          }
          const bool move = mx > ref + kPromptSlack;
          if (__any_sync(0xffffffffu, move || (EXACT && exact))) {
            const float f = move ? exp2_ftz(ref - mx) : 1.0f;
            if (move) ref = mx;
            l *= f;
            if (EXACT) exact = exact || __any_sync(0xffffffffu, tid < rows && move && fabsf(mx) > kPromptExact);
            if (EXACT && exact && !poly) {
              // The weights' multiply-add takes the reference, a rounded product, from exact ones: of scores
              // of 2^31 the difference of a score from itself would be some 2^7 and its weight infinite.
#pragma unroll
              for (int i = 0; i < 64; ++i) set_pair(i, mul2(pair(i), pack2(sl_now, sl_now)));
              sl_now = 1.0f;
            }
            if (j > 0) {  // these scores came after the products of the tile before
              const uint64_t f2 = pack2(f, f);
#pragma unroll 1
              for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t o[32];
                tmem_load32(t_o(h) + lane_base + 32 * ch, o);
                tmem_wait_load(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  float a, b;
                  unpack2(mul2(pack2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), f2), a, b);
                  o[2 * k] = __float_as_uint(a);
                  o[2 * k + 1] = __float_as_uint(b);
                }
                tmem_store32(t_o(h) + lane_base + 32 * ch, o);
              }
            }
          }
          const float m = ref == -INFINITY ? 0.0f : ref;  // nothing seen so far: every weight is 0
          const uint64_t sl2 = pack2(sl_now, sl_now), m2 = pack2(-m, -m);
          uint64_t sum2[2] = {0, 0};
          auto weights = [&](auto of) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float a, b;
                unpack2(of(16 * e + k), a, b);
                // The weights enter the product as one bf16 each: an average of values, each weight
                // off by 2^-8 at most. A second half of each would cost half as many products
                // again; to sum them as they enter, two more operations a weight (1494 us for 1413).
                a = exp2_ftz(a), b = exp2_ftz(b);
                w[k] = pack_bf16x2(a, b);
                sum2[k & 1] = add2(sum2[k & 1], pack2(a, b));
              }
              tmem_store16(t_s(h) + lane_base + 16 * e, w);
            }
          };
          if (CAPPED && !SLOPES && tiny)
            weights([&](int i) { return fma2(capped_tiny(i), pair(i), m2); });
          else if (CAPPED && !SLOPES && poly)
            weights([&](int i) { return fma2(capped(i), pair(i), m2); });
          else
            weights([&](int i) { return fma2(pair(i), sl2, m2); });
          {
            float a, b;
            unpack2(add2(sum2[0], sum2[1]), a, b);
            l += a + b;
          }
          tmem_wait_store();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(h));
      }
      // (The products came after the values were looked at, so the marks are in.)
      if (!ok || !warp_wait(o_done(h), done++ & 1, ok)) break;
      if (!busy) {
        release(i);
        continue;
      }
      tc_fence_after();
      const bool mine = tid < rows;
      const Place place = mine ? row_place(p, x.lo, x.hi, unit.part) : Place::kNowhere;
      const float inv = 1.0f / denominator(l, false);
      const size_t at = mine ? q_row(unit.sr, unit.kvh, unit.r0 + tid) : 0, slot = at / D * p.num_partitions + unit.part;
      // A lane has a row, but rows are 128 bytes or more apart in memory: 128 bytes of each go
      // through shared memory, so that eight lanes write a row's together (written by its own
      // lane, 32 bytes at a time, a unit's rows took 4600 cycles).
      const uint32_t stage = kv_sm + ST * S::TILE + warp * S::OUT_BYTES;
      auto put = [&](const uint32_t (&w)[32], char *row) {  // row: where the lane's goes, or null
#pragma unroll
        for (int e = 0; e < 8; ++e)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((e ^ (lane & 7)) << 4)),
                       "r"(w[4 * e]), "r"(w[4 * e + 1]), "r"(w[4 * e + 2]), "r"(w[4 * e + 3])
                       : "memory");
        __syncwarp();
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = 4 * e + lane / 8;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[e].x), "=r"(v[e].y), "=r"(v[e].z), "=r"(v[e].w)
                       : "r"(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4)));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          char *dst = reinterpret_cast<char *>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), 4 * e + lane / 8));
          if (dst) *reinterpret_cast<uint4 *>(dst + (lane & 7) * 16) = v[e];
        }
        __syncwarp();
      };
      char *const res = place == Place::kOut ? static_cast<char *>(p.out) + at * 2 : nullptr;
      char *const acc = place == Place::kWorkspace ? reinterpret_cast<char *>(p.ws_acc + slot * D) : nullptr;
      const bool some_out = __any_sync(0xffffffffu, res != nullptr), some_acc = __any_sync(0xffffffffu, acc != nullptr);
#pragma unroll 1
      for (int ch = 0; ch < D / 64; ++ch) {
        uint32_t o[2][32];
        tmem_load32(t_o(h) + lane_base + 64 * ch, o[0]);
        tmem_load32(t_o(h) + lane_base + 64 * ch + 32, o[1]);
        tmem_wait_load(o[0]);
        tmem_wait_load(o[1]);
        if (some_out) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            w[e] = pack_bf16x2(__uint_as_float(o[e / 16][2 * (e % 16)]) * inv,
                               __uint_as_float(o[e / 16][2 * (e % 16) + 1]) * inv);
          put(w, res ? res + 128 * ch : nullptr);
        }
        if (some_acc) {
          put(o[0], acc ? acc + 256 * ch : nullptr);
          put(o[1], acc ? acc + 256 * ch + 128 : nullptr);
        }
      }
      if (acc) {
        p.ws_m[slot] = merge_max(ref, l);
        p.ws_l[slot] = l;
      }
      if (poisoned[i % kPromptUnits] == i + 1 && place != Place::kNowhere) {
        // What is not finite in the values that the row sees, of the tiles that were cleared.
        for (int j = 0; j < nt; ++j) {
          if (!unit.careful(j)) continue;
          const int t0 = start + j * kPromptTile;
          for (int t = max(x.lo, t0); t < min(min(x.hi, end), t0 + kPromptTile); ++t) {
            if (t >= unit.all_from && t < unit.all_to) continue;
            const int phys = __ldg(p.tables + size_t(unit.s) * p.max_blocks + t / p.block_size);
            if (phys < 0 || phys >= p.num_blocks) continue;
            const __nv_bfloat16 *v =
                static_cast<const __nv_bfloat16 *>(p.v_cache) +
                ((size_t(phys) * p.block_size + t % p.block_size) * p.num_kv_heads + unit.kvh) * D;
            for (int e = 0; e < D; ++e) {
              const float y = __bfloat162float(v[e]);
              if (fabsf(y) <= 3.402823466e38f) continue;
              if (acc) {
                reinterpret_cast<float *>(acc)[e] += y;
              } else {
                __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(res) + e;
                *dst = __float2bfloat16_rn(__bfloat162float(*dst) + y);
              }
            }
          }
        }
      }
      release(i);
      tc_fence_before();  // O may be overwritten once the next unit's weights are there
    }
    if (!ok && lane == 0) timeout();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

template <int D, Cap CAP, bool SLOPES>
pk_status launch_prompt_as(const ExtendParams &p, const pk_cache_desc &d, unsigned units, cudaStream_t stream) {
  CUtensorMap kmap, vmap;
  if (!encode_bf16_pool(&kmap, p.k_cache, d) || !encode_bf16_pool(&vmap, p.v_cache, d)) return PK_ERR_CUDA;
  auto kern = attn_prompt_kernel<D, CAP, SLOPES>;
  static std::atomic<uint64_t> ready{0};
  if (!smem_ready(kern, PromptShape<D>::SMEM_BYTES, ready)) return PK_ERR_CUDA;
  kern<<<units, kPromptThreads, PromptShape<D>::SMEM_BYTES, stream>>>(p, kmap, vmap);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

template <int D, Cap CAP>
pk_status launch_prompt_as(const ExtendParams &p, const pk_cache_desc &d, unsigned units, cudaStream_t stream) {
  return p.slopes ? launch_prompt_as<D, CAP, true>(p, d, units, stream)
                  : launch_prompt_as<D, CAP, false>(p, d, units, stream);
}

template <int D>
pk_status launch_prompt(const ExtendParams &p, const pk_cache_desc &d, unsigned units, cudaStream_t stream) {
  if (p.cap_log2 == 0.0f) return launch_prompt_as<D, Cap::kNone>(p, d, units, stream);
  const float f = fabsf(p.factor);
  return f >= kNearFrom && f <= kNearTo && p.cap_log2 <= kNearCap
             ? launch_prompt_as<D, Cap::kNear>(p, d, units, stream)
             : launch_prompt_as<D, Cap::kWide>(p, d, units, stream);
}

}  // namespace
}  // namespace pk
