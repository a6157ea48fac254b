// Attention of each sequence's drafted tokens over its cached context
// (pk_paged_attention_tree), for verifying a tree or a chain of drafts in one
// pass: the n drafted tokens are the last n of the context, their K/V already
// in the cache, and a 64-bit mask per token says which drafts it sees.
//
// Per KV head a sequence is n G rows of query against ctx keys: 4 d operations
// per row and key for 4 d bytes of key and value (bf16), so up to some 283 rows
// the memory bounds it, beyond that the tensor cores.
//
// bf16 (attn_tree_kernel): tcgen05 products with tensor-memory accumulators. A
// CTA holds 128 rows, one lane of tensor memory each, and goes over its keys in
// pairs of 64-token tiles:
//   producer warp   TMA loads of each block's K (a pair at a time) and V (a tile
//                   at a time);
//   score warp      S = Q K^T of a pair (128 x 128) as soon as the last pair's
//                   products have ended; a 128 x 64 product costs as much time;
//   value warp      O += P V per tile, P read from tensor memory, under the
//                   softmax of the next tile;
//   softmax warps   a thread owns a row: reads its 64 scores, masks them, keeps
//                   the running maximum and sum, and writes the weights over the
//                   scores;
//   units' warp     asks launch control for the next unit.
// O stays in tensor memory. A row's reference of the exponent moves only when
// the maximum has outgrown it by 2^8: until then weights up to 2^8 are added as
// they are (fp32 accumulators, fp32 sums), and O is rescaled a few times per
// row instead of once per tile.
// The weights enter the product as a bf16 pair hi + lo (one bf16 would put
// 2^-9 on every output).
// 256 columns of tensor memory (128 of scores, 128 of O) and 105 KB of shared
// memory let two CTAs share an SM: one's softmax overlaps the other's products.
// The CTAs stay: a unit is 128 rows of a (sequence, KV head) over a partition,
// and when one is almost done its CTA takes over the unit of one that has not
// started, so that short contexts keep memory busy too and uneven ones even out.
//
// Measured (heads of 128, blocks of 16): 8 sequences of 32 768 tokens with 32
// drafts, 64 = 8 x 8 heads (256 rows a KV head) 340 us, 805 TFLOP/s of the
// formula's work, 1.2 PFLOP/s with the second half of the weights; with 1 to 16
// drafts (one unit of 128 rows reads all) 173 to 193 us, 5.6 to 6.2 TB/s. 256
// sequences of some 500 (64 to 4608) tokens with 16 drafts, 32 = 4 x 8 heads, 98 to
// 105 us, 5.1 to 5.3 TB/s (75 to 78% of a copy). There units dealt out at launch took 149 us
// against 115 by launch control; then 100 by shortening what a unit's end costs its
// softmax warps (a timeline: 2700 cycles to ask for the next unit's queries, 1700 to
// look for values that are not finite, and fences that waited for the last unit's
// stores). One product warp in place of two: equal. Scores of 64 tokens at a time:
// 343 us against 334 (the long case). What bounds it now: long, the chain of a pair,
// 5200 cycles of which each softmax is 1330 and each wait for scores 970, with two
// CTAs to overlap (tensor pipe 44% busy); short, beginnings and ends of units.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <new>
#include <vector>

#include "attn_rows.cuh"
#include "pagedkv.h"
#include "pk_tcgen05.cuh"
#include "pk_tma_host.h"

namespace pk {

extern "C" int *pkx_tree_attention_error_word() { return error_word(g_rows_error); }

namespace {

constexpr int kRows = 128;          // query rows of a CTA
constexpr int kTile = 64;           // tokens of a tile
constexpr int kPair = 2 * kTile;    // tokens whose scores are computed at once
constexpr int kThreads = 256;       // 4 softmax warps, the producer, two product warps, the units'
// Registers: 256 threads of 128 at launch, of which the softmax warps' four take
// 176 each and the other four leave themselves 80 (176 + 80 = 2 x 128).
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
constexpr uint32_t kTmemCols = 256;
// Units known at a time: the softmax may be one behind the producer, which asks
// for one more.
constexpr int kUnits = 4;
constexpr uint32_t kNegateA = 1u << 13;  // of an instruction descriptor
constexpr float kSlack = 8.0f;      // log2 of how far a maximum may outgrow the reference

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0)
    return n;
  cudaGetLastError();  // clear a failed query on a machine without a GPU
  return 152;
}

template <int D, int BS>
struct TreeShape {
  static constexpr int SLABS = D / 64;               // 128-byte column slabs
  static constexpr int Q_SLAB = kRows * 128, K_SLAB = kPair * 128, V_SLAB = kTile * 128;
  static constexpr int Q_BYTES = SLABS * Q_SLAB, K_BYTES = SLABS * K_SLAB, V_BYTES = SLABS * V_SLAB;
  static constexpr int BPT = kTile / BS, BPP = kPair / BS;  // blocks per tile, per pair
  static constexpr int STAGE_BYTES = 2048;  // per softmax warp: 64 bytes of each of its rows, on their way out
  static constexpr int SMEM_BYTES = 1024 + Q_BYTES + K_BYTES + 2 * V_BYTES + 4 * STAGE_BYTES;
};

// A unit of work: 128 rows of one (sequence, KV head) over one partition.
struct Unit {
  int s, kvh, part;
  int q0, n, ctx, np;  // as SeqRows
  int r0, rows;        // its rows
  int start, end, nt;  // its tokens and tiles (the last pair may be half); s < 0: no more units
};

template <int D, int BS>
__global__ void __launch_bounds__(kThreads, 2)
    attn_tree_kernel(RowsParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using S = TreeShape<D, BS>;
  launch_dependents();  // the merge may be scheduled as this grid drains
  extern __shared__ uint8_t smem_raw[];
  const uint32_t q_sm = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t k_sm = q_sm + S::Q_BYTES, v_sm = k_sm + S::K_BYTES;
  __shared__ __align__(8) uint64_t bars[14 + 2 * kUnits];
  __shared__ uint4 answer;
  __shared__ Unit units[kUnits];
  __shared__ uint32_t tmem_slot;
  // The last unit, plus one, of either parity whose drafts' values were not all finite.
  // Nothing is cleared: a unit's mark is written by its own softmax warps and read once
  // all four are past its tiles (u_done), and the next unit but one, which writes the
  // same word, is begun only after all four have read it.
  __shared__ int poisoned[2];
  auto bar = [&](int i) { return smem_addr(bars + i); };
  // Units i, pairs g and, as the last pair of a unit may be half, second halves f
  // are counted over the whole life of the CTA; a barrier's phase is the count of
  // what uses it. Every wait names a phase of which the one before has ended for
  // certain and the one after cannot have: a wait by parity tells neighbouring
  // phases apart, not more.
  const uint32_t q_ready = bar(0), u_done = bar(1);
  const uint32_t k_full = bar(2), k_empty = bar(3), s_full = bar(4);  // by pair
  auto p_full = [&](int h) { return bar(5 + h); };                     // by half
  auto o_done = [&](int h) { return bar(7 + h); };
  auto v_full = [&](int h) { return bar(9 + h); };
  const uint32_t u_want = bar(11), u_answer = bar(12);
  auto u_full = [&](int i) { return bar(14 + i % kUnits); };
  auto u_empty = [&](int i) { return bar(14 + kUnits + i % kUnits); };
  auto u_phase = [](int i) { return uint32_t(i / kUnits) & 1u; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  if (threadIdx.x == 0) {
    mbar_init(q_ready, 128);
    mbar_init(u_done, 4);
    mbar_init(u_want, 1);
    mbar_init(u_answer, 1);
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    mbar_init(s_full, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(p_full(h), 4);
      mbar_init(o_done(h), 1);
      mbar_init(v_full(h), 1);
      poisoned[h] = 0;
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(u_full(i), 1);
      mbar_init(u_empty(i), 7);  // every warp but the one that fills them
    }
    fence_barrier_init();
  }
  if (warp == 5) tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t t_o = tmem + 128;                             // O: columns 128 .. 128 + D
  auto t_s = [&](int h) { return tmem + 64u * h; };  // a half's scores, then its weights: hi 32 columns, lo 32
  // A wait of the whole warp, which converges on it (tensor memory is accessed
  // by whole warps); once one has failed, so do all.
  auto warp_wait = [](uint32_t b, uint32_t parity, bool &ok) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(b, parity));
    return ok;
  };
  auto q_row = [&](int q0, int row, int kvh) {  // element offset of a row of q and out
    return (size_t(q0 + row / G) * p.num_q_heads + kvh * G + row % G) * D;
  };
  auto timeout = [&] { record_error(&g_rows_error, PK_DEVERR_TIMEOUT, blockIdx.x); };

  // Registers change hands by whole warpgroups: all four warps of one have to execute
  // the same instruction, so it stands before the roles of the second one part.
  if (warp >= 4) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == 4) {
      // ---------------- producer ----------------
      if (lane == 0) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
      }
      // A pair of tiles to load: the lane's block of it, read from the table ahead
      // of time.
      struct Pair {
        int phys, nblk, kvh, s;  // nblk 0: no more
      };
      const Unit *at = nullptr;  // the unit that `next` is in, its pairs so far, its number
      int at_g = 0, at_n = 0, at_i = -1;
      bool ok = true;
      auto next = [&] {
        Pair x{0, 0, 0, 0};
        if (at && ++at_g == at_n) at = nullptr;
        if (!at) {
          ++at_i;
          if (!warp_wait(u_full(at_i), u_phase(at_i), ok)) return x;
          const Unit *c = units + at_i % kUnits;
          if (c->s < 0) return x;
          at = c, at_g = 0, at_n = (c->nt + 1) / 2;
        }
        // The unit after this one is asked for two pairs before the end: early enough
        // to be here in time, late enough to go to the CTA that is free first.
        if (at_g == max(0, at_n - 2) && lane == 0) mbar_arrive(u_want);
        const int nb = (at->end - at->start + BS - 1) / BS;
        x.nblk = min(S::BPP, nb - at_g * S::BPP);
        x.kvh = at->kvh;
        x.s = at->s;
        if (lane < x.nblk)
          x.phys = __ldg(p.tables + size_t(at->s) * p.max_blocks + at->start / BS + at_g * S::BPP + lane);
        if (x.phys < 0 || x.phys >= p.num_blocks) {
          record_error(&g_rows_error, PK_DEVERR_BLOCK_ID, at->s);
          x.phys = 0;  // stay in bounds and keep the byte count; the result is flagged
        }
        if (at_g == at_n - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(u_empty(at_i));  // done with the unit's entry
        }
        return x;
      };
      // The blocks [b0, b0 + n) of a pair into dst, their rows' slabs `slab` apart.
      auto load = [&](const CUtensorMap *map, uint32_t dst, int slab, uint32_t full, const Pair &x, int b0, int n) {
        if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(n * S::SLABS * BS * 128));
        __syncwarp();
        if (lane >= b0 && lane < b0 + n) {
#pragma unroll
          for (int h = 0; h < S::SLABS; ++h)
            tma_load_3d(dst + h * slab + (lane - b0) * BS * 128, map, full, h * 64, x.kvh, x.phys * BS);
        }
      };
      // A pair's K goes when the scores of the one before are done, its V tiles when
      // the products before have ended; the block table is read ahead of both.
      int g = 0, f = 0;  // pairs whose V, and second halves whose V, are loaded
      Pair a{0, 0, 0, 0}, b = next();
      while (ok && (a.nblk || b.nblk)) {
        if (a.nblk) {
          // o_done(0) of pair g - 1 is its phase g - 1.
          if (!(ok = g < 1 || mbar_wait(o_done(0), (g - 1) & 1))) break;
          load(&vmap, v_sm, S::V_SLAB, v_full(0), a, 0, min(a.nblk, S::BPT));
          if (a.nblk > S::BPT) {
            if (!(ok = f < 1 || mbar_wait(o_done(1), (f - 1) & 1))) break;
            load(&vmap, v_sm + S::V_BYTES, S::V_SLAB, v_full(1), a, S::BPT, a.nblk - S::BPT);
            ++f;
          }
          ++g;
        }
        if (b.nblk) {
          // Pair g's K: the scores of pair g - 1 are done.
          if (!(ok = g < 1 || mbar_wait(k_empty, (g - 1) & 1))) break;
          load(&kmap, k_sm, S::K_SLAB, k_full, b, 0, b.nblk);
        }
        a = b;
        b = a.nblk ? next() : Pair{0, 0, 0, 0};
      }
      if (!ok && lane == 0) timeout();
      // Let every issued copy land before the warp leaves.
      if (g > 0) mbar_wait(k_full, (g - 1) & 1), mbar_wait(v_full(0), (g - 1) & 1);
      if (f > 0) mbar_wait(v_full(1), (f - 1) & 1);
    } else if (warp == 5) {
      // ---------------- scores ----------------
      // The whole warp goes over the tiles, so that descriptors and addresses are
      // uniform values, and one elected lane issues. Scores and values have a warp
      // each: a wait on a barrier costs some 200 cycles even when its phase has
      // ended, and in one warp the waits and issues of both took longer than the
      // products. Every order between the two is by barrier.
      // A negative scale negates the queries, so that scores order as their
      // exponents do.
      const uint32_t s_desc = mma_desc(kRows, kPair, false) | (p.scale_log2 < 0.0f ? kNegateA : 0u);
      const uint64_t q_d = smem_desc(q_sm, 16, 1024), k_d = smem_desc(k_sm, 16, 1024);
      bool ok = true;
      int g = 0, f = 0;
      bool whole = false;  // the pair before had a second half
      for (int i = 0; warp_wait(u_full(i), u_phase(i), ok); ++i) {
        const int nt = units[i % kUnits].nt;
        const bool last = units[i % kUnits].s < 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(u_empty(i));
        if (last || !warp_wait(q_ready, i & 1, ok)) break;
        for (int j = 0; j < nt; j += 2, ++g) {
          // The score columns hold the weights of the pair before until its last
          // product ends (products end in order).
          if (!warp_wait(k_full, g & 1, ok)) break;
          if (g > 0 && !(whole ? warp_wait(o_done(1), (f - 1) & 1, ok) : warp_wait(o_done(0), (g - 1) & 1, ok))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)  // a descriptor's address counts 16 bytes
              tc_mma_ss(tmem, q_d + (ks / 4) * (S::Q_SLAB / 16) + (ks % 4) * 2,
                        k_d + (ks / 4) * (S::K_SLAB / 16) + (ks % 4) * 2, s_desc, ks > 0);
            tc_commit(k_empty);
            tc_commit(s_full);
          }
          whole = j + 1 < nt;
          f += whole;
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) timeout();
      // Nothing of this warp's products is under way when tensor memory is freed.
      if (g > 0) mbar_wait(s_full, (g - 1) & 1);
      __syncwarp();
    } else if (warp == 6) {
      // ---------------- weights times values ----------------
      constexpr uint32_t O_DESC = mma_desc(kRows, D, true);
      const uint64_t v_d = smem_desc(v_sm, S::V_SLAB, 1024);
      bool ok = true;
      int g = 0, f = 0;
      for (int i = 0; warp_wait(u_full(i), u_phase(i), ok); ++i) {
        const int nt = units[i % kUnits].nt;
        const bool last = units[i % kUnits].s < 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(u_empty(i));
        if (last) break;
        for (int j = 0; j < nt; ++j) {
          const int h = j & 1;
          const uint32_t phase = uint32_t(h ? f : g) & 1u;
          if (!warp_wait(v_full(h), phase, ok) || !warp_wait(p_full(h), phase, ok)) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t d = v_d + (h ? S::V_BYTES / 16 : 0);
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int ks = 0; ks < kTile / 16; ++ks)
                tc_mma_ts(t_o, t_s(h) + 32 * half + 8 * ks, d + ks * 128, O_DESC, j > 0 || half > 0 || ks > 0);
            tc_commit(o_done(h));  // and the V tile is free
          }
          f += h;
          g += h || j + 1 == nt;
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) timeout();
      if (g > 0) mbar_wait(o_done(0), (g - 1) & 1);
      if (f > 0) mbar_wait(o_done(1), (f - 1) & 1);
      __syncwarp();
    } else {
      // ---------------- units ----------------
      // The grid has a CTA per unit, longest first; those that find no room are
      // taken over, one at a time, by whichever CTA needs work next.
      const int X = p.num_kv_heads * p.row_tiles, Y = p.items ? p.num_items : p.num_seqs;
      bool ok = true;
      int published = 0;
      auto publish = [&](const Unit &c) {
        const int i = published;
        if (i >= kUnits && !warp_wait(u_empty(i), u_phase(i - kUnits), ok)) return;
        if (lane == 0) {
          units[i % kUnits] = c;
          mbar_arrive(u_full(i));
        }
        ++published;
      };
      for (int u = blockIdx.x, asked = 0; u >= 0;) {
        const int x = u % X, y = (u / X) % Y, z = u / X / Y;
        Unit c;
        if (work_item(p, y, p.num_partitions - 1 - z, x == 0 && lane == 0, c.s, c.part)) {
          const SeqRows sr = seq_rows(p, c.s, x == 0 && lane == 0 && c.part == 0);
          c.kvh = x / p.row_tiles;
          c.r0 = x % p.row_tiles * kRows;
          c.rows = min(kRows, sr.n * G - c.r0);
          if (c.rows > 0 && sr.ctx == 0) {  // invalid length (recorded): zero rows
            for (int k = lane; c.part == 0 && k < c.rows * (D / 8); k += 32)
              *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                         q_row(sr.q0, c.r0 + k / (D / 8), c.kvh) + k % (D / 8) * 8) =
                  make_uint4(0, 0, 0, 0);
          } else if (c.rows > 0 && c.part < sr.np) {
            c.q0 = sr.q0, c.n = sr.n, c.ctx = sr.ctx, c.np = sr.np;
            c.start = c.part * p.partition;
            c.end = min(sr.ctx, c.start + p.partition);
            c.nt = (c.end - c.start + kTile - 1) / kTile;
            publish(c);
            if (!ok || !warp_wait(u_want, (published - 1) & 1, ok)) break;
          }
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(u_answer, 16);
          try_cancel(smem_addr(&answer), u_answer);
        }
        if (!warp_wait(u_answer, asked & 1, ok)) break;
        ++asked;
        u = cancelled_cta(smem_addr(&answer));
        fence_answer_read();
        __syncwarp();
      }
      Unit end;
      end.s = -1;
      if (ok) publish(end);
      if (!ok && lane == 0) timeout();
    }
  } else {
    // ---------------- softmax: a thread is a row ----------------
    setmaxnreg_inc<kSoftmaxRegs>();
    const int r = threadIdx.x;
    const uint32_t lane_base = uint32_t(warp * 32) << 16;
    // At least the smallest normal number: a scale of 0 must not turn the -inf of
    // what is masked into NaN.
    const float sl = fmaxf(fabsf(p.scale_log2), 1.17549435e-38f);
    bool ok = true;
    auto wait = [&](uint32_t b, uint32_t parity) { return warp_wait(b, parity, ok); };
    // A unit's queries into shared memory. Rows past its last keep what was there:
    // no row's result depends on another's query.
    const uint32_t inv_g = (65536 + G - 1) / G;  // x / G = x inv_g >> 16 for x < 512
    auto load_q = [&](const Unit &c) {
      constexpr int CH = D / 8, STEP = 128 / CH;  // chunks of a row, rows at once
      const int ch = r % CH;
      const __nv_bfloat16 *src =
          static_cast<const __nv_bfloat16 *>(p.q) + (size_t(c.q0) * p.num_q_heads + c.kvh * G) * D + ch * 8;
      const uint32_t dst = q_sm + (ch >> 3) * S::Q_SLAB;
#pragma unroll 4
      for (int row = r / CH; row < c.rows; row += STEP) {
        const uint32_t x = c.r0 + row, tok = x * inv_g >> 16;
        cp_async16(dst + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                   src + size_t(tok * (p.num_q_heads - G) + x) * D, 16);
      }
    };
    auto q_landed = [&] {
      cp_async_wait();
      fence_proxy_async_shared();
      mbar_arrive(q_ready);
    };
    bool loaded = false;  // the unit's queries were loaded under the one before
    for (int i = 0, g = 0, f = 0; wait(u_full(i), u_phase(i)); ++i) {
      const Unit &c = units[i % kUnits];  // read where it is needed: registers are short
      auto release = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(u_empty(i));
      };
      if (c.s < 0) break;
      if (!loaded) {
        load_q(c);
        q_landed();
      }
      loaded = false;
      const bool busy = warp * 32 < c.rows;  // this warp has rows
      const int unit = i;
      const int nt = c.nt, start = c.start;
      const int lim = min(c.ctx - c.n, c.end);  // tokens before it are seen by every row
      // The drafts that this thread's row sees, loaded ahead of the tiles that need it.
      const uint64_t mask = r < c.rows ? draft_mask(p, c.q0, (c.r0 + r) / G, c.n) : 0;
      float ref = -INFINITY, l = 0.0f;  // the exponent's reference (scaled scores), the sum
      for (int j = 0; j < nt; ++j) {
        const int t0 = start + j * kTile, h = j & 1;
        const uint32_t phase = uint32_t(h ? f : g) & 1u;
        const bool careful = t0 + kTile > lim;
        if (h == 0 && !wait(s_full, g & 1)) break;
        tc_fence_after();
        uint32_t x[2][32];
        if (busy) {
          tmem_load32(t_s(h) + lane_base, x[0]);
          tmem_load32(t_s(h) + lane_base + 32, x[1]);
        }
        if (careful) {
          // Drafts, or the partition's end: what a row does not see is masked, the
          // values past the end are zeroed, and so is what is not finite in the
          // drafts' values, which would reach rows that do not see it (0 * NaN);
          // the rows that do see it get it at the end.
          if (!wait(v_full(h), phase)) break;
          const uint32_t vb = v_sm + (h ? S::V_BYTES : 0);
          const int first = max(0, lim - t0), valid = min(kTile, c.end - t0);
          // Four rows' chunks of 16 bytes at once; they are looked at word by word only
          // if a carry into a half's sign shows an exponent of all ones.
          constexpr int STEP = 128 / (D / 8);  // rows that the threads cover at once
          const uint32_t a = vb + (r % (D / 8) >> 3) * S::V_SLAB + r / (D / 8) * 128 + (r & 7) * 16;
          bool wrote = valid < kTile;
#pragma unroll 1
          for (int k0 = first / (4 * STEP) * (4 * STEP); k0 < kTile; k0 += 4 * STEP) {
            uint32_t w[4][4], odd = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = k0 + i * STEP + r / (D / 8);
              w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0;
              if (row >= first && row < valid)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                             : "r"(a + (k0 + i * STEP) * 128));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (k0 + i * STEP + r / (D / 8) >= valid)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a + (k0 + i * STEP) * 128), "r"(0)
                             : "memory");
#pragma unroll
              for (int e = 0; e < 4; ++e) odd |= (w[i][e] & 0x7f807f80u) + 0x00800080u;
            }
            if (odd & 0x80008000u) {
              poisoned[unit & 1] = unit + 1;
              wrote = true;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((w[i][e] & 0x7f80u) == 0x7f80u) w[i][e] &= 0xffff0000u;
                  if ((w[i][e] & 0x7f800000u) == 0x7f800000u) w[i][e] &= 0xffffu;
                }
                const int row = k0 + i * STEP + r / (D / 8);
                if (row >= first && row < valid)
                  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a + (k0 + i * STEP) * 128),
                               "r"(w[i][0]), "r"(w[i][1]), "r"(w[i][2]), "r"(w[i][3])
                               : "memory");
              }
            }
          }
          if (__any_sync(0xffffffffu, wrote)) fence_proxy_async_shared();
          __syncwarp();
        }
        if (j == nt - 1) {
          // The unit's last scores are there, so its queries are done with: the
          // next unit's, if it is known already, come in under this tile's softmax
          // (after the fence above, which would wait for them).
          loaded = __all_sync(0xffffffffu, mbar_test(u_full(i + 1), u_phase(i + 1))) &&
                   units[(i + 1) % kUnits].s >= 0;
          if (loaded) load_q(units[(i + 1) % kUnits]);
        }
        if (busy) {
          tmem_wait_load(x[0]);
          tmem_wait_load(x[1]);
          if (careful) {
            const int live = c.end - t0;  // more than 0
            const uint64_t see = see64(mask, c.ctx - c.n, t0) & (live < 64 ? (1ull << live) - 1 : ~0ull);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t w = uint32_t(see >> (32 * e));
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(w & (1u << k))) x[e][k] = 0xff800000u;  // -inf
            }
          }
          float mx;
          {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 32; ++k)
              top[k & 3] = max3(top[k & 3], __uint_as_float(x[k >> 4][2 * (k & 15)]),
                                __uint_as_float(x[k >> 4][2 * (k & 15) + 1]));
            mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            mx = mx == -INFINITY ? mx : mx * sl;
          }
          const bool move = mx > ref + kSlack;
          if (__any_sync(0xffffffffu, move)) {
            const float f = move ? exp2_ftz(ref - mx) : 1.0f;
            if (move) ref = mx;
            l *= f;
            if (j > 0) {
              // The scores of a pair come after the products of the one before.
              if (h == 1 && !wait(o_done(0), g & 1)) break;
              tc_fence_after();
              const uint64_t f2 = pack2(f, f);
#pragma unroll 1
              for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t o[32];
                tmem_load32(t_o + lane_base + 32 * ch, o);
                tmem_wait_load(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  float a, b;
                  unpack2(mul2(pack2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), f2), a, b);
                  o[2 * k] = __float_as_uint(a);
                  o[2 * k + 1] = __float_as_uint(b);
                }
                tmem_store32(t_o + lane_base + 32 * ch, o);
              }
            }
          }
          const float m = ref == -INFINITY ? 0.0f : ref;  // nothing seen so far: every weight is 0
          const uint64_t sl2 = pack2(sl, sl), m2 = pack2(-m, -m), minus = pack2(-1.0f, -1.0f);
          uint64_t sum2 = 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float a, b;
              unpack2(fma2(pack2(__uint_as_float(x[e][2 * k]), __uint_as_float(x[e][2 * k + 1])), sl2, m2), a, b);
              a = exp2_ftz(a);
              b = exp2_ftz(b);
              const uint64_t ab = pack2(a, b);
              sum2 = add2(sum2, ab);
              hi[k] = pack_bf16x2(a, b);
              unpack2(fma2(pack2(bf16_lo(hi[k]), bf16_hi(hi[k])), minus, ab), a, b);
              lo[k] = pack_bf16x2(a, b);
            }
            tmem_store16(t_s(h) + lane_base + 16 * e, hi);
            tmem_store16(t_s(h) + lane_base + 32 + 16 * e, lo);
          }
          {
            float a, b;
            unpack2(sum2, a, b);
            l += a + b;
          }
          tmem_wait_store();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(h));
        f += h;
        g += h || j + 1 == nt;
      }
      if (!ok) break;
      if (loaded) q_landed();
      // Every warp is past the tiles: their marks are in.
      if (lane == 0) mbar_arrive(u_done);
      if (!wait(u_done, i & 1)) break;
      const bool fix = poisoned[i & 1] == i + 1;
      if (!busy) {
        release();
        continue;
      }
      if (!(nt & 1 ? wait(o_done(0), (g - 1) & 1) : wait(o_done(1), (f - 1) & 1))) break;
      tc_fence_after();
      const bool mine = r < c.rows;
      const size_t at = mine ? q_row(c.q0, c.r0 + r, c.kvh) : 0;
      const bool split = c.np > 1;
      const float inv = split ? 1.0f : 1.0f / denominator(l, c.ctx > c.n || mask != 0);
      const size_t slot = at / D * p.num_partitions + c.part;
      // A lane has a row, but rows are 64 bytes or more apart in memory: 64 bytes of
      // each go through shared memory, so that four lanes write a row's together.
      const uint32_t stage = v_sm + 2 * S::V_BYTES + warp * S::STAGE_BYTES;
      const size_t to = split ? slot * D * 4 : at * 2;  // byte offset of the row
      size_t dst[4];  // where the lane's quarters of rows go
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[e] = __shfl_sync(0xffffffffu, to, 8 * e + lane / 4) + (lane & 3) * 16;
      char *const base = split ? reinterpret_cast<char *>(p.ws_acc) : static_cast<char *>(p.out);
      auto put = [&](const uint32_t (&w)[16], int byte) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 64 +
                                                                       ((e ^ ((lane >> 1) & 3)) << 4)),
                       "r"(w[4 * e]), "r"(w[4 * e + 1]), "r"(w[4 * e + 2]), "r"(w[4 * e + 3])
                       : "memory");
        __syncwarp();
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 8 * e + lane / 4;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[e].x), "=r"(v[e].y), "=r"(v[e].z), "=r"(v[e].w)
                       : "r"(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4)));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (warp * 32 + 8 * e + lane / 4 < c.rows) *reinterpret_cast<uint4 *>(base + dst[e] + byte) = v[e];
        __syncwarp();
      };
      float odd = 0.0f;  // NaN once an element is not finite
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        tmem_load32(t_o + lane_base + 32 * ch, o);
        tmem_wait_load(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) odd = fmaf(__uint_as_float(o[e]), 0.0f, odd);
        uint32_t w[16];
        if (split) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = o[16 * h + e];
            put(w, 128 * ch + 64 * h);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          put(w, 64 * ch);
        }
      }
      if (mine && split) {
        p.ws_m[slot] = merge_max(ref, l);
        p.ws_l[slot] = l;
      }
      __syncwarp();
      if (odd != 0.0f && mine && fabsf(l) <= 3.402823466e38f) {
        // A context value that is not finite gave NaN, by the product with a weight's
        // lower half: the sum of what is not finite in its place. Eight columns at a
        // time.
#pragma unroll 1
        for (int ch = 0; ch < D / 8; ++ch) {
          float *const acc = p.ws_acc + slot * D + ch * 8;
          __nv_bfloat16 *const res = static_cast<__nv_bfloat16 *>(p.out) + at + ch * 8;
          bool bad = false;
          for (int e = 0; e < 8; ++e)
            bad = bad || !(fabsf(split ? acc[e] : __bfloat162float(res[e])) <= 3.402823466e38f);
          if (!bad) continue;
          float sum[8] = {};
#pragma unroll 4
          for (int k = c.start; k < lim; ++k) {
            const int phys = min(max(__ldg(p.tables + size_t(c.s) * p.max_blocks + k / BS), 0), p.num_blocks - 1);
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(
                static_cast<const __nv_bfloat16 *>(p.v_cache) +
                ((size_t(phys) * BS + k % BS) * p.num_kv_heads + c.kvh) * D + ch * 8));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float y = e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
              sum[e] += fabsf(y) <= 3.402823466e38f ? 0.0f : y;
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (sum[e] == 0.0f) continue;
            if (split)
              acc[e] = sum[e];
            else
              res[e] = __float2bfloat16_rn(sum[e]);
          }
        }
      }
      if (fix && mine) {  // what is not finite in the values of the drafts that the row sees
        const int base = c.ctx - c.n;
        for (int k = max(base, c.start); k < c.end; ++k) {
          const int phys = __ldg(p.tables + size_t(c.s) * p.max_blocks + k / BS);
          if (!((mask >> (k - base)) & 1) || phys < 0 || phys >= p.num_blocks) continue;
          const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v_cache) +
                                   ((size_t(phys) * BS + k % BS) * p.num_kv_heads + c.kvh) * D;
          for (int e = 0; e < D; ++e) {
            const float y = __bfloat162float(v[e]);
            if (fabsf(y) <= 3.402823466e38f) continue;
            if (split) {
              p.ws_acc[slot * D + e] += y;
            } else {
              __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + at + e;
              *dst = __float2bfloat16_rn(__bfloat162float(*dst) + y);
            }
          }
        }
      }
      release();
      tc_fence_before();  // O may be overwritten once the next unit's weights are there
    }
    if (!ok && lane == 0) timeout();
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
  const dim3 g = rows_grid(p);
  const int64_t units = int64_t(g.x) * g.y * g.z;
  if (units > INT32_MAX) return PK_ERR_UNSUPPORTED;
  kern<<<unsigned(units), kThreads, S::SMEM_BYTES, stream>>>(p, kmap, vmap);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

template <int D>
pk_status launch_tree_d(const RowsParams &p, const pk_cache_desc &d, cudaStream_t stream) {
  return d.block_size == 8    ? launch_tree<D, 8>(p, d, stream)
         : d.block_size == 16 ? launch_tree<D, 16>(p, d, stream)
                              : launch_tree<D, 32>(p, d, stream);
}

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

template <typename T, int D, int NT>
__global__ void __launch_bounds__(128, 2) attn_split_kernel(RowsParams p) {
  using S = SplitShape<T, D, NT>;
  constexpr int NP = S::PARTS, NW = S::W_PARTS;
  constexpr int R = S::R, MT = D / 16, CH = D * int(sizeof(T)) / 16;
  launch_dependents();  // the merge may be scheduled as this grid drains
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t *q_sm = smem + S::KV_BYTES;
  const int kvh = blockIdx.x / p.row_tiles, tile = blockIdx.x % p.row_tiles;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool record = blockIdx.x == 0 && threadIdx.x == 0;
  int s, part;
  if (!work_item(p, blockIdx.y, gridDim.z - 1 - blockIdx.z, record, s, part)) return;
  const SeqRows sr = seq_rows(p, s, record && part == 0);
  const int G = p.group, r0 = tile * R, rows = min(R, sr.n * G - r0);
  if (rows <= 0) return;
  auto q_row = [&](int r) {  // element offset of row r0 + r in q and out
    return (size_t(sr.q0 + (r0 + r) / G) * p.num_q_heads + kvh * G + (r0 + r) % G) * D;
  };
  if (sr.ctx == 0) {  // invalid length (recorded): zero rows
    if (part == 0)
      for (int i = threadIdx.x; i < rows * D; i += 128)
        store_elem(static_cast<T *>(p.out) + q_row(i / D) + i % D, 0.0f);
    return;
  }
  if (part >= sr.np) return;
  const int start = part * p.partition, end = min(sr.ctx, start + p.partition), base = sr.ctx - sr.n;
  const int lim = min(base, end);  // tokens before it are seen by every row
  __shared__ uint64_t masks[R];
  __shared__ int poisoned;
  if (threadIdx.x == 0) poisoned = 0;
  if (threadIdx.x < R)
    masks[threadIdx.x] = int(threadIdx.x) < rows ? draft_mask(p, sr.q0, (r0 + int(threadIdx.x)) / G, sr.n) : 0;

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
    const float f = r >= rows ? 0.0f : (NP > 1 ? p.scale_log2 : 1.0f);  // bf16 queries stay as they are
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
    const bool careful = t0 + 16 > lim;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (NP == 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] *= p.scale_log2;
      if (careful)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = t0 + rw + 8 * (e >> 1);
          if (t >= end || (t >= base && !((masks[8 * n + 2 * qd + (e & 1)] >> (t - base)) & 1))) x[n][e] = -INFINITY;
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
    if (t0 + 16 > lim && lim < end) {
      // Drafts: what is not finite in their values becomes 0, or it would reach rows
      // that do not see it (0 * NaN); the rows that do see it get it at the end.
      for (int i = lane; i < 16 * D; i += 32) {
        const int t = t0 + i / D;
        T *v = reinterpret_cast<T *>(vw + (i / D) * S::V_PITCH) + i % D;
        if (t >= base && t < end && !(fabsf(load_elem(v)) <= 3.402823466e38f)) {
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
  const bool split = sr.np > 1;
  for (int i = threadIdx.x; i < rows * D; i += 128) {
    const int r = i / D, c = i % D;
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
    // A context value that is not finite gave NaN, by the product with a part of a
    // weight that is 0 or negative: the sum of what is not finite in its place.
    if (!(fabsf(O) <= 3.402823466e38f) && fabsf(L) <= 3.402823466e38f) {
      float odd = 0.0f;
#pragma unroll 4
      for (int t = start; t < lim; ++t) {
        const int phys = min(max(__ldg(trow + t / p.block_size), 0), p.num_blocks - 1);
        const float y = load_elem(static_cast<const T *>(p.v_cache) +
                                  ((size_t(phys) * p.block_size + t % p.block_size) * p.num_kv_heads + kvh) * D + c);
        odd += fabsf(y) <= 3.402823466e38f ? 0.0f : y;
      }
      if (odd != 0.0f) O = odd;
    }
    if (poisoned)  // what is not finite in the values of the drafts that the row sees
      for (int t = max(base, start); t < end; ++t) {
        const int phys = __ldg(trow + t / p.block_size);
        if (!((masks[r] >> (t - base)) & 1) || phys < 0 || phys >= p.num_blocks) continue;
        const float y = load_elem(static_cast<const T *>(p.v_cache) +
                                  ((size_t(phys) * p.block_size + t % p.block_size) * p.num_kv_heads + kvh) * D + c);
        if (!(fabsf(y) <= 3.402823466e38f)) O += y;
      }
    if (split) {
      const size_t to = q_row(r) / D * p.num_partitions + part;
      p.ws_acc[to * D + c] = O;
      if (c == 0) {
        p.ws_m[to] = merge_max(M, L);
        p.ws_l[to] = L;
      }
    } else {
      store_elem(static_cast<T *>(p.out) + q_row(r) + c, O / denominator(L, base > 0 || masks[r] != 0));
    }
  }
}

template <typename T, int D, int NT>
pk_status launch_split(RowsParams p, cudaStream_t stream) {
  using S = SplitShape<T, D, NT>;
  auto kern = attn_split_kernel<T, D, NT>;
  static std::atomic<uint64_t> ready{0};
  if (!smem_ready(kern, S::SMEM_BYTES, ready)) return PK_ERR_CUDA;
  p.row_tiles = (p.max_draft * p.group + S::R - 1) / S::R;
  kern<<<rows_grid(p), 128, S::SMEM_BYTES, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

// Whether `rows` rows of a (sequence, KV head) go to attn_tree_kernel. Up to eight
// rows of 64 values are too little for its 128 lanes and its chain of a pair, and
// attn_split_kernel, with more CTAs an SM, reads faster (us, tcgen05 and split):
// 256 x 500 tokens, 4 x 8 heads, one draft 76 and 62, two 76 and 66, four (16 rows)
// 76 and 91; 8 x 32 768 tokens 118 and 103, 118 and 105, 119 and 115. Between, with a
// query head per KV head: 256 x 510 tokens of very uneven lengths, 8 rows 80 and 84, 9
// to 16 rows 81 and 93 to 96; 8 x 32 768 tokens, 8 rows 125 and 103, 9 to 16 rows 125
// and 116 to 119. With rows of 128 values it does not: 99 and 117, 172 and 234 with one
// draft.
bool tcgen05_path(const pk_cache_desc &d, int64_t rows) {
  return d.dtype == PK_BF16 && (d.block_size == 8 || d.block_size == 16 || d.block_size == 32) &&
         (d.head_dim == 128 || rows > 8);
}
// Rows per CTA of attn_split_kernel: the fewest that hold a sequence's, at most 32.
int split_rows(int rows) { return rows <= 8 ? 8 : (rows <= 16 ? 16 : 32); }

template <typename T, int D>
pk_status run(const RowsParams &p, const pk_cache_desc &d, cudaStream_t stream) {
  pk_status st = PK_ERR_UNSUPPORTED;
  if (sizeof(T) == 2 && tcgen05_path(d, p.max_draft * p.group)) {
    st = launch_tree_d<D>(p, d, stream);
  } else {
    switch (split_rows(p.max_draft * p.group)) {
      case 8: st = launch_split<T, D, 1>(p, stream); break;
      case 16: st = launch_split<T, D, 2>(p, stream); break;
      default: st = launch_split<T, D, 4>(p, stream);
    }
  }
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

// The partition size that the planner chooses (0: none). The units (the rows of a
// sequence and KV head that a CTA holds, over one partition) go longest first to the CTA that is
// free first, so a launch lasts about as long as its longest unit or as the mean
// share of a CTA, whichever is more, plus what the last round leaves idle (of the
// shortest units' length). Each partition of a context that is split adds a
// partial row of d + 2 floats per query row, written and read once: 6 TB/s,
// against 22 ns for a token of a CTA where two share an SM's bandwidth; a unit
// costs about 128 tokens more than its own.
int32_t tree_partition(const int32_t *context_lens, int32_t num_seqs, int32_t longest,
                       int32_t max_draft_len, int32_t num_q_heads, const pk_cache_desc &d) {
  if (longest <= 1024) return 0;
  const int64_t rows = int64_t(max_draft_len) * (num_q_heads / d.num_kv_heads);
  const int unit_rows = tcgen05_path(d, rows) ? kRows : split_rows(int(rows));
  const int64_t per_item = d.num_kv_heads * ((rows + unit_rows - 1) / unit_rows);
  const int64_t slots = 2 * sm_count();
  const double merge = double(max_draft_len) * num_q_heads * (d.head_dim + 2) * 8 / 6e12 / 22e-9;
  std::vector<int32_t> count;  // items by tiles
  int32_t best = 0;
  double least = 0;
  for (int c = 1; c <= 32; ++c) {
    int64_t n = (int64_t(longest) + c - 1) / c;
    n = (n + kTile - 1) / kTile * kTile;
    n = (n + d.block_size - 1) / d.block_size * d.block_size;
    if (c > 1 && n < 512) break;
    count.assign(size_t(n / kTile + 2), 0);
    double partials = 0;
    for (int32_t s = 0; s < num_seqs; ++s) {
      const int64_t len = std::max(context_lens[s], 1), whole = len / n;
      count[size_t((n + kTile - 1) / kTile)] += int32_t(whole);
      if (len % n) ++count[size_t((len % n + kTile - 1) / kTile)];
      if (len > n) partials += double(whole + (len % n != 0));
    }
    int64_t units = 0, tail = 0;
    double work = 0;
    size_t top = 0;
    for (size_t tiles = 0; tiles < count.size(); ++tiles) {
      if (!count[tiles]) continue;
      if (units < slots) tail = int64_t(tiles) * kTile;  // the length that the last `slots` units reach
      units += count[tiles] * per_item;
      work += double(count[tiles] * per_item) * (double(tiles) * kTile + 128);
      top = tiles;
    }
    const double idle = double((slots - units % slots) % slots) / double(slots) * double(tail);
    const double cost = merge * partials + std::max(double(top * kTile), work / double(slots) + idle);
    if (c == 1 || cost < 0.97 * least) {
      least = cost;
      best = c == 1 ? 0 : int32_t(n);
    }
  }
  return best;
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
  for (int32_t s = 0; s < num_seqs; ++s) longest = std::max(longest, context_lens[s]);
  const pk_status st = check_tree(desc, num_q_heads, longest, std::max(partition_size, 0));
  if (st != PK_OK) return st;
  int32_t part = partition_size > 0 && partition_size < longest ? partition_size : 0;
  if (partition_size == -1) {
    try {
      part = tree_partition(context_lens, num_seqs, longest, max_draft_len, num_q_heads, *desc);
    } catch (const std::bad_alloc &) {
      return PK_ERR_NOMEM;
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
