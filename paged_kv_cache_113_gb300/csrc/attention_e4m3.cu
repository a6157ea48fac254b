// Decode attention over the 8-bit cache (pk_paged_attention_decode_e4m3).
//
// With K_t = 2^ek_t kc_t and V_t = 2^ev_t vc_t (e4m3 codes kc, vc), x in log2:
//     x_t = scale log2(e) 2^ek_t <q, kc_t>
//     out = sum_t 2^(x_t + ev_t) vc_t / sum_t 2^x_t
// Bound by memory: a token and KV head cost 2 (d + 1) bytes, half of bf16, for
// 4 G d operations.
//
// A unit of work is a (KV head, sequence, partition) or work item. Four consumer
// warps and a producer warp make a CTA; three CTAs share an SM, and each stays:
// when a unit's stages are almost all asked for, the producer asks launch control
// for a CTA that has not started and takes its unit over, so the next unit's codes
// are under way while the consumers finish this one. The producer streams each
// block's codes with TMA tensor loads into a ring of three 16 KB stages (64 tokens
// of d = 128, 128 of d = 64), their exponents with 16-byte asynchronous copies (a
// block and head's K and V exponents are contiguous) and a unit's queries with one
// bulk copy. Consumers widen codes to fp16, where e4m3 is exact, in registers and
// multiply on the tensor cores (m16n8k16, tokens as M, the group's heads as N); V's
// codes are transposed on their way out of shared memory (ldmatrix .b8.trans),
// which fixes the order of a tile's tokens. The exponents never touch the codes.
// K's scale the finished scores. V's join the softmax's exponent: the weight of a
// token is 2^(x_t + ev_t - m) with m the largest x_t + ev_t so far, less 10, moved
// only when a weight would pass 2^15: fp16 weights keep their 11 bits down to 2^-24
// of the largest, and most tiles need neither the warp's maximum nor a rescaling.
// The denominator's terms 2^(x_t - m) stay fp32: at most 2^115, as ev >= -100, so that
// their sum overflows only past 2^13 tokens of which no value reaches 2^-90.
//
// mma.sync carries it: with 8 rows of query for 2 (d + 1) bytes the tensor cores
// are 19 to 22% busy, and the widening to fp16 has to pass registers in any case, where
// tcgen05 would want it back in shared memory.
//
// Measured (bf16 queries, 64 = 8 x 8 heads of 128 unless said): 8 sequences of
// 32 768 tokens in 91 to 92 us, 5.9 TB/s (87% of a copy); 256 of some 500 (33 to
// 4608) tokens, 32 = 4 x 8 heads, in 50 to 54, 4.7 to 5.1 TB/s (69 to 75%): there the
// first stage is full 4.8 us after the launch (items, lengths and tables, then
// codes, each from cold memory), and the last CTAs end 7 us apart. A stage costs
// the producer 620 cycles of issue for its eight tensor loads, of 2100 to 2400;
// before the next unit was looked up without a wait it cost 590 more, 53 to 57 us.
// One CTA per unit took 58.0 us with 4 stages, 56.0 with 3 stages and 4 CTAs;
// exponents by bulk copies 68 against 63.5 at blocks of 8; stages of 64 tokens at
// d = 64 50.8 against 42.6.
//
// Precision: a query head is scaled by the power of two that brings its largest
// value into [2^14, 2^15), so bf16 queries are exact in fp16 (down to 2^-32 of
// the largest). fp32 queries, and all weights, are fp16 pairs, hi + lo, good to
// 2^-22, at twice the tensor work. For bf16 results weights of one fp16 (2^-11, not
// what the denominator sums) and sums left to the tensor cores took 69.3 us against
// 70.1 (256 x 577 tokens), 90.3 against 91.7 (8 x 32 768), 43.6 against 45.4 (heads of
// 64), and made them 8 10^-4 away from rounded fp32 ones.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_rows.cuh"
#include "pagedkv.h"
#include "pk_tma_host.h"

namespace pk {

extern "C" int *pkx_attention_e4m3_error_word() { return error_word(g_rows_error); }

namespace {

constexpr int kWarps = 4;             // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;  // and the producer
constexpr int kUnits = 4;             // units known at a time
constexpr int kAhead = 5;             // stages of a unit left when the next is asked for
// log2 of the largest fp16 weight when the reference is set, and at most.
constexpr float kHeadroom = 10.0f, kSlack = 15.0f;

template <typename IO, int D, int BS>
struct Shape {
  static constexpr int STAGES = 3;
  static constexpr int TILES = 128 / D;         // 16-token tiles of a warp in a stage: 16 KB of codes
  static constexpr int TPS = 16 * kWarps * TILES;  // tokens per stage
  static constexpr int BPS = TPS / BS;          // blocks per stage
  static constexpr int KV_BYTES = TPS * D;      // the stage's K, and its V
  static constexpr int STAGE_BYTES = 2 * KV_BYTES;
  static constexpr int EXP_BYTES = TPS * 2;
  static constexpr int EXP_LANES = TPS / 8;     // lanes that copy 16 bytes of exponents each
  static constexpr int KC = D / 32;             // 32-byte steps of a row
  static constexpr int Q_ROW = D * int(sizeof(IO)) + 16;  // padded against bank conflicts
  static constexpr int Q_BYTES = 8 * Q_ROW;     // a group's queries
  static constexpr int OUT_STRIDE = D + 4;      // padded row of the warps' merge
  static constexpr int MERGE_BYTES = kWarps * 8 * (OUT_STRIDE + 2) * 4;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * (STAGE_BYTES + EXP_BYTES) + 2 * Q_BYTES + MERGE_BYTES;
  static_assert(32 % BPS == 0, "a stage's blocks lie in one chunk of 32 table entries");
};

// A unit of work: a sequence and KV head's queries over one partition.
struct Unit {
  int s, kvh, part, np;
  int start, end, nst;  // its tokens and stages; s < 0: no more units
};

// Byte offset of 16-byte chunk c of row r in a TMA tile of D-byte rows (128- or
// 64-byte swizzle).
template <int D>
__device__ __forceinline__ int swizzled(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Whether the codes of row r of a tile are all zeros.
template <int D>
__device__ __forceinline__ bool zero_row(uint32_t base, int r) {
  uint32_t any = 0;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    uint32_t x, y, z, w;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
                 : "r"(base + r * D + c * 16));
    any |= x | y | z | w;
  }
  return (any & 0x7f7f7f7fu) == 0;
}

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

template <typename IO, int D, int BS>
__global__ void __launch_bounds__(kThreads, 3)
    attn_e4m3_kernel(RowsParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<IO, D, BS>;
  constexpr int STAGES = S::STAGES, KC = S::KC;
  constexpr int QW = sizeof(IO) == 4 ? 2 : 1;   // fp16 parts of a query
  launch_dependents();  // the merge may be scheduled as this grid drains
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t stages = (raw + 1023u) & ~1023u;
  const uint32_t exps = stages + STAGES * S::STAGE_BYTES;
  const uint32_t q_sm = exps + STAGES * S::EXP_BYTES;
  __shared__ __align__(8) uint64_t bars[2 * STAGES + 7 + 2 * kUnits];
  __shared__ uint4 answer;
  __shared__ Unit units[kUnits];
  auto bar = [&](int i) { return smem_addr(bars + i); };
  // Units i and stages t are counted over the whole life of the CTA.
  auto full_bar = [&](int t) { return bar(t % STAGES); };
  auto empty_bar = [&](int t) { return bar(STAGES + t % STAGES); };
  auto q_full = [&](int i) { return bar(2 * STAGES + (i & 1)); };
  auto q_empty = [&](int i) { return bar(2 * STAGES + 2 + (i & 1)); };
  const uint32_t m_full = bar(2 * STAGES + 4), m_empty = bar(2 * STAGES + 5);  // the warps' merge
  const uint32_t u_answer = bar(2 * STAGES + 6);
  auto u_full = [&](int i) { return bar(2 * STAGES + 7 + i % kUnits); };
  auto u_empty = [&](int i) { return bar(2 * STAGES + 7 + kUnits + i % kUnits); };
  auto t_phase = [](int t) { return uint32_t(t / STAGES) & 1u; };
  auto u_phase = [](int i) { return uint32_t(i / kUnits) & 1u; };
  // A wait of the whole warp, which converges on it; once one has failed, so do all.
  auto warp_wait = [](uint32_t b, uint32_t parity, bool &ok) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(b, parity));
    return ok;
  };
  auto timeout = [&] { record_error(&g_rows_error, PK_DEVERR_TIMEOUT, blockIdx.x); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full_bar(i), 1 + S::EXP_LANES);
      mbar_init(empty_bar(i), kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), kWarps);
    }
    mbar_init(m_full, kWarps);
    mbar_init(m_empty, kWarps);
    mbar_init(u_answer, 1);
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(u_full(i), 1);
      mbar_init(u_empty(i), kWarps);
    }
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    // ---------------- producer ----------------
    // The grid has a CTA per unit, longest first; those that find no room are
    // taken over, one at a time, by whichever CTA needs work next. The next unit is
    // asked for kAhead stages before the end of this one: early enough to be here in
    // time, late enough to go to the CTA that is free first (4, 5, 6 and 8 stages:
    // 52, 50, 50.3 and 53 us for 256 sequences of some 500 tokens; of lengths more
    // uneven, of heads of 64, of blocks of 8 and for 8 x 32 768 tokens all within 1%).
    if (lane == 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
    const int X = p.num_kv_heads, Y = p.items ? p.num_items : p.num_seqs;
    bool ok = true, open = false;  // open: an answer is under way
    int asked = 0;
    auto ask = [&] {
      open = true;
      if (lane == 0) {
        mbar_arrive_expect_tx(u_answer, 16);
        try_cancel(smem_addr(&answer), u_answer);
      }
    };
    auto answered = [&] {  // the unit's number, or -1: none is left
      ++asked;
      open = false;
      const int u = cancelled_cta(smem_addr(&answer));
      fence_answer_read();
      __syncwarp();
      return u;
    };
    // Whether a barrier's phase has ended; with `wait`, after a wait for it.
    auto ended = [&](uint32_t b, uint32_t parity, bool wait) {
      return wait ? warp_wait(b, parity, ok) : bool(__all_sync(0xffffffffu, mbar_test(b, parity)));
    };
    // The next unit u becomes known, and its queries come, in five steps, a stage or
    // more apart; a step whose barrier is not there yet is left to the next stage.
    // What a step needs from memory is loaded after the one before it, by every
    // stage alike (from somewhere harmless when nothing is needed), so that no
    // branch has a load of its own to wait for.
    int step = 1, u = blockIdx.x;
    const int32_t *at0 = p.ctx_lens, *at1 = p.ctx_lens;
    int got0 = 0, got1 = 0;
    Unit next;
    int first = 0;                 // its first 32 table entries, a lane's one
    bool have = false;             // it is known and has work
    int loaded = 0;                // units whose queries are under way
    int x = 0, y = 0, z = 0;       // u's place: KV head, work, partition of the grid
    auto advance = [&](bool wait) {
      const bool record = x == 0 && lane == 0;
      switch (step++) {
        case 0:
          ask();
          break;
        case 1:
          if (open) {  // else the first unit, the CTA's own
            if (!ended(u_answer, asked & 1, wait)) {
              --step;
              break;
            }
            u = answered();
          }
          x = u % X, y = u / X % Y, z = u / X / Y;
          if (u >= 0 && p.items) at0 = p.items + 2 * y + (lane & 1);
          break;
        case 2: {
          next.s = p.items ? __shfl_sync(0xffffffffu, got0, 0) : y;
          next.part = p.items ? __shfl_sync(0xffffffffu, got0, 1) : p.num_partitions - 1 - z;
          have = u >= 0 && checked_item(p, y, next.s, next.part, record);
          if (!have) break;
          next.start = next.part * p.partition;
          at0 = p.tables + size_t(next.s) * p.max_blocks + min(next.start / BS + lane, p.max_blocks - 1);
          at1 = p.ctx_lens + next.s;
          break;
        }
        case 3: {
          if (!have) break;
          const int ctx = checked_context(p, next.s, 1, got1, record && next.part == 0);
          if (ctx == 0)  // invalid (recorded): a zero row
            for (int k = lane; next.part == 0 && k < G * D; k += 32)
              store_elem(static_cast<IO *>(p.out) + (size_t(next.s) * p.num_q_heads + x * G) * D + k, 0.0f);
          next.kvh = x;
          next.np = partitions_of(p, ctx);
          have = next.part < next.np;
          if (!have) break;
          next.end = min(ctx, next.start + p.partition);
          next.nst = (next.end - next.start + S::TPS - 1) / S::TPS;
          first = got0;
          break;
        }
        case 4: {
          if (!have) break;
          const int k = loaded;
          if (k >= 2 && !ended(q_empty(k), uint32_t((k >> 1) - 1) & 1u, wait)) {
            --step;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(q_full(k), uint32_t(G * D * sizeof(IO)));
          __syncwarp();
          if (lane < G)
            bulk_load(q_sm + (k & 1) * S::Q_BYTES + lane * S::Q_ROW,
                      static_cast<const IO *>(p.q) + (size_t(next.s) * p.num_q_heads + x * G + lane) * D,
                      D * sizeof(IO), q_full(k));
          ++loaded;
        }
      }
    };
    auto fetch = [&] {
      got0 = __ldg(at0);
      got1 = __ldg(at1);
    };
    int t = 0, i = 0;
    for (; ok; ++i) {
      while (ok && (step < 5 || (!have && u >= 0))) {
        if (step == 5) step = 0;  // a unit without work
        advance(true);
        fetch();
      }
      if (!ok || (i >= kUnits && !warp_wait(u_empty(i), u_phase(i - kUnits), ok))) break;
      if (lane == 0) {
        if (have)
          units[i % kUnits] = next;
        else
          units[i % kUnits].s = -1;
        mbar_arrive(u_full(i));
      }
      if (!have) break;
      const Unit c = next;
      // Table entries are read ahead in chunks of 32, one per lane, one chunk in
      // reserve, so that no stage waits on a dependent load.
      const int32_t *trow = p.tables + size_t(c.s) * p.max_blocks + c.start / BS;
      const int nb = (c.end - c.start + BS - 1) / BS;
      int cur = first, nxt = 32 + lane < nb ? __ldg(trow + 32 + lane) : 0;
      int chunk = 0;
      step = 0;
      have = false;
      for (int st = 0; st < c.nst; ++st, ++t) {
        if (c.nst - st <= kAhead && step < 5) advance(false);
        fetch();
        const int b0 = st * S::BPS;
        if (b0 >= 32 * (chunk + 1)) {
          ++chunk;
          cur = nxt;
          const int j = 32 * (chunk + 1) + lane;
          nxt = j < nb ? __ldg(trow + j) : 0;
        }
        int phys = __shfl_sync(0xffffffffu, cur, (b0 & 31) + min(lane, S::BPS - 1));
        if (t >= STAGES && !warp_wait(empty_bar(t), t_phase(t - STAGES), ok)) break;
        const int nblk = min(S::BPS, nb - b0);
        if (lane == 0) mbar_arrive_expect_tx(full_bar(t), uint32_t(nblk * BS * 2 * D));
        if (lane < nblk && (phys < 0 || phys >= p.num_blocks)) {
          record_error(&g_rows_error, PK_DEVERR_BLOCK_ID, c.s);
          phys = 0;  // stay in bounds and keep the byte count; the result is flagged
        }
        // The exponents, eight tokens' 16 bytes a lane: through the load unit, as
        // small blocks already give TMA a request per kilobyte.
        const int eb = __shfl_sync(0xffffffffu, phys, lane * 8 / BS % 32);
        if (lane < S::EXP_LANES) {
          if (lane * 8 / BS < nblk)
            cp_async16(exps + (t % STAGES) * S::EXP_BYTES + lane * 16,
                       p.kv_exp + ((size_t(eb) * p.num_kv_heads + c.kvh) * BS + lane * 8 % BS) * 2, 16);
          cp_async_arrive(full_bar(t));
        }
        if (lane < nblk) {
          const uint32_t dst = stages + (t % STAGES) * S::STAGE_BYTES + lane * BS * D;
          tma_load_3d(dst, &kmap, full_bar(t), 0, c.kvh, phys * BS);
          tma_load_3d(dst + S::KV_BYTES, &vmap, full_bar(t), 0, c.kvh, phys * BS);
        }
      }
    }
    if (!ok && lane == 0) timeout();
    // Let every issued copy, and an answer, land before the warp leaves.
    if (open) mbar_wait(u_answer, asked & 1);
    for (int k = max(0, t - STAGES); k < t; ++k) mbar_wait(full_bar(k), t_phase(k));
    for (int k = max(0, loaded - 2); k < loaded; ++k) mbar_wait(q_full(k), uint32_t(k >> 1) & 1u);
    return;
  }

  // ---------------- consumer warps ----------------
  // C fragments: a lane holds rows rw and rw + 8, heads 2 qd and 2 qd + 1. Rows of
  // the scores are tokens in the order in which a lane gets four consecutive
  // tokens of a value column: rows 2 q, 2 q + 1, 8 + 2 q, 9 + 2 q are tokens 4 q
  // to 4 q + 3. A key row's 32-byte step comes as four bytes 4 qd .. 4 qd + 3 per
  // lane and 16-byte chunk; the product's k index follows that order, and so
  // does the query operand.
  const int qd = lane & 3, rw = lane >> 2;
  const int mi = lane >> 3, r8 = lane & 7;
  auto token_of = [](int row) { return 4 * ((row & 7) >> 1) + 2 * (row >> 3) + (row & 1); };
  const int tok0 = token_of(rw);  // of row rw; that of row rw + 8 is two later
  float *sm_o = reinterpret_cast<float *>(smem_raw + (q_sm + 2 * S::Q_BYTES - raw));
  float *sm_m = sm_o + kWarps * 8 * S::OUT_STRIDE, *sm_l = sm_m + kWarps * 8;
  bool ok = true;
  for (int i = 0, t = 0; warp_wait(u_full(i), u_phase(i), ok); ++i) {
    const Unit c = units[i % kUnits];
    __syncwarp();
    if (lane == 0) mbar_arrive(u_empty(i));
    if (c.s < 0 || !warp_wait(q_full(i), uint32_t(i >> 1) & 1u, ok)) break;
    uint32_t qb[QW][KC][4];
    float sl0, sl1;  // scale log2(e) and the query scaling undone, heads 2 qd and 2 qd + 1
    {
      float qv[KC][8];
      uint32_t top = 0;
      const IO *qrow = reinterpret_cast<const IO *>(smem_raw + (q_sm - raw) + (i & 1) * S::Q_BYTES +
                                                    min(rw, G - 1) * S::Q_ROW);
#pragma unroll
      for (int k = 0; k < KC; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 x = load4(qrow + 32 * k + 16 * h + 4 * qd);
          qv[k][4 * h] = x.x, qv[k][4 * h + 1] = x.y, qv[k][4 * h + 2] = x.z, qv[k][4 * h + 3] = x.w;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b = __float_as_uint(qv[k][4 * h + e]) & 0x7fffffffu;
            top = max(top, b < 0x7f800000u ? b : 0u);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(i));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int up = min(126, 14 - (int(top >> 23) - 127));  // >= -113
      const float f = pow2(up);
      const float sl = p.scale_log2 * pow2(-up);
      sl0 = __shfl_sync(0xffffffffu, sl, 8 * qd);
      sl1 = __shfl_sync(0xffffffffu, sl, 8 * qd + 4);
#pragma unroll
      for (int k = 0; k < KC; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = rw < G ? qv[k][2 * e] * f : 0.0f, b = rw < G ? qv[k][2 * e + 1] * f : 0.0f;
          qb[0][k][e] = pack_f16x2(a, b);
          if (QW == 2) {
            const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&qb[0][k][e]));
            qb[QW - 1][k][e] = pack_f16x2(a - hi.x, b - hi.y);
          }
        }
    }
    float o[KC][2][4];  // [32-column step][16-column half]
#pragma unroll
    for (int k = 0; k < KC; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) o[k][h][0] = o[k][h][1] = o[k][h][2] = o[k][h][3] = 0.0f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    for (int st = 0; st < c.nst; ++st, ++t) {
      const int slot = t % STAGES;
      if (!warp_wait(full_bar(t), t_phase(t), ok)) break;
      const uint32_t kbase = stages + slot * S::STAGE_BYTES, vbase = kbase + S::KV_BYTES;
#pragma unroll 1
      for (int tile = 0; tile < S::TILES; ++tile) {
        const int t0 = (tile * kWarps + warp) * 16;
        const int nvalid = c.end - (c.start + st * S::TPS + t0);
        if (nvalid <= 0) break;
        if (nvalid < 16) {
          // Rows past the end may hold anything: zero values, so that a zero
          // weight never meets a NaN.
          for (int i = lane; i < (16 - nvalid) * (D / 16); i += 32) {
            const uint32_t a = vbase + (t0 + nvalid + i / (D / 16)) * D + (i % (D / 16)) * 16;
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
          }
          fence_proxy_async_shared();  // a later unit's copies go to the same rows
          __syncwarp();
        }
        uint32_t e0, e1;  // exponents of the lane's tokens: K in the low byte, V above
        {
          const uint32_t a = exps + slot * S::EXP_BYTES + (t0 + tok0) * 2;
          asm volatile("ld.shared.u16 %0, [%1];" : "=r"(e0) : "r"(a));
          asm volatile("ld.shared.u16 %0, [%1];" : "=r"(e1) : "r"(a + 4));
        }
        // S^T = K_tile Q^T; low 16 bits and high 16 bits of a lane's four bytes
        // are the two k halves of one product.
        float sa[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          uint32_t r[4];
          ldmatrix_x4(kbase + swizzled<D>(t0 + token_of((mi & 1) * 8 + r8), 2 * k + (mi >> 1)), r[0],
                      r[1], r[2], r[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(r[2 * h], a0, a2);
            e4m3x4_to_f16x4(r[2 * h + 1], a1, a3);
#pragma unroll
            for (int w = 0; w < QW; ++w)
              mma_f16_16816(sa[h], a0, a1, a2, a3, qb[w][k][2 * h], qb[w][k][2 * h + 1]);
          }
        }
        const float k0 = __uint_as_float((e0 & 0xffu) << 23), k1 = __uint_as_float((e1 & 0xffu) << 23);
        // A row of zeros is written with exponent 0, which says nothing of its
        // neighbours: it counts as the smallest, or it would push the weights of
        // far smaller values out of fp16's range.
        int ev0 = int(e0 >> 8) - 127, ev1 = int(e1 >> 8) - 127;
        if (__any_sync(0xffffffffu, ev0 == 0 || ev1 == 0)) {
          if (zero_row<D>(vbase, t0 + tok0)) ev0 = -100;
          if (zero_row<D>(vbase, t0 + tok0 + 2)) ev1 = -100;
        }
        const float v0 = float(ev0), v1 = float(ev1);
        float x0 = (sa[0][0] + sa[1][0]) * sl0 * k0, x1 = (sa[0][1] + sa[1][1]) * sl1 * k0;
        float x2 = (sa[0][2] + sa[1][2]) * sl0 * k1, x3 = (sa[0][3] + sa[1][3]) * sl1 * k1;
        if (tok0 >= nvalid) x0 = x1 = -INFINITY;
        if (tok0 + 2 >= nvalid) x2 = x3 = -INFINITY;
        float z0 = fmaxf(x0 + v0, x2 + v1), z1 = fmaxf(x1 + v0, x3 + v1);
        // The reference moves only when a weight would pass fp16's range.
        if (__any_sync(0xffffffffu, z0 > m0 + kSlack || z1 > m1 + kSlack)) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            z0 = fmaxf(z0, __shfl_xor_sync(0xffffffffu, z0, off));
            z1 = fmaxf(z1, __shfl_xor_sync(0xffffffffu, z1, off));
          }
          const float n0 = fmaxf(m0, z0 - kHeadroom), n1 = fmaxf(m1, z1 - kHeadroom);
          const float c0 = exp2_ftz(m0 - n0), c1 = exp2_ftz(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= c0;
          l1 *= c1;
#pragma unroll
          for (int k = 0; k < KC; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              o[k][h][0] *= c0;
              o[k][h][1] *= c1;
              o[k][h][2] *= c0;
              o[k][h][3] *= c1;
            }
        }
        const float y0 = x0 - m0, y1 = x1 - m1, y2 = x2 - m0, y3 = x3 - m1;
        l0 += exp2_ftz(y0) + exp2_ftz(y2);
        l1 += exp2_ftz(y1) + exp2_ftz(y3);
        const float p0 = exp2_ftz(y0 + v0), p1 = exp2_ftz(y1 + v0);
        const float p2 = exp2_ftz(y2 + v1), p3 = exp2_ftz(y3 + v1);
        uint32_t b[2][2];  // P^T as the B operand, high and low parts: the C fragments transposed
        {
          const uint32_t w0 = pack_f16x2(p0, p1), w1 = pack_f16x2(p2, p3);
          b[0][0] = movmatrix_trans(w0);
          b[0][1] = movmatrix_trans(w1);
          const float2 h0 = __half22float2(*reinterpret_cast<const __half2 *>(&w0));
          const float2 h1 = __half22float2(*reinterpret_cast<const __half2 *>(&w1));
          b[1][0] = movmatrix_trans(pack_f16x2(p0 - h0.x, p1 - h0.y));
          b[1][1] = movmatrix_trans(pack_f16x2(p2 - h1.x, p3 - h1.y));
        }
        // O^T += V^T P^T: a transposed load gives a lane four tokens of a column, the
        // ones that its rows of the scores belong to.
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          uint32_t r[4];  // columns 32 k + rw, + 8 of both 16-column halves
          ldmatrix_b8_x2_trans(vbase + swizzled<D>(t0 + (lane & 15), 2 * k + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(r[2 * h], a0, a2);
            e4m3x4_to_f16x4(r[2 * h + 1], a1, a3);
            // The tensor cores cut their fp32 sums off, always toward zero (2 10^-5 after
            // 32 768 tokens): a tile's sum is added with a rounding.
            float t4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 1; w >= 0; --w) mma_f16_16816(t4, a0, a1, a2, a3, b[w][0], b[w][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][h][e] += t4[e];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(t));
    }

    // The denominators of a warp's 16 tokens lie in the 8 lanes of a quad index.
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    if (!ok) break;
    // Merge the consumer warps' states in shared memory, once all have read the
    // unit's before.
    if (i > 0 && !warp_wait(m_empty, uint32_t(i - 1) & 1u, ok)) break;
#pragma unroll
    for (int k = 0; k < KC; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float *base = sm_o + (warp * 8 + 2 * qd) * S::OUT_STRIDE + 32 * k + 16 * h + rw;
        base[0] = o[k][h][0];
        base[S::OUT_STRIDE] = o[k][h][1];
        base[8] = o[k][h][2];
        base[S::OUT_STRIDE + 8] = o[k][h][3];
      }
    if (rw == 0) {
      sm_m[warp * 8 + 2 * qd] = m0;
      sm_m[warp * 8 + 2 * qd + 1] = m1;
      sm_l[warp * 8 + 2 * qd] = l0;
      sm_l[warp * 8 + 2 * qd + 1] = l1;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(m_full);
    if (!warp_wait(m_full, uint32_t(i) & 1u, ok)) break;
    const size_t row0 = size_t(c.s) * p.num_q_heads + c.kvh * G;  // the group's first row of out
    for (int k = threadIdx.x * 4; k < G * D; k += kWarps * 128) {  // four columns each
      const int g = k / D, col = k % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w * 8 + g]);
      float L = 0.0f;
      float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_ftz(sm_m[w * 8 + g] - M);  // 0 for a warp that saw no token
        const float4 v = *reinterpret_cast<const float4 *>(sm_o + (w * 8 + g) * S::OUT_STRIDE + col);
        L = fmaf(sm_l[w * 8 + g], f, L);
        O.x = fmaf(v.x, f, O.x), O.y = fmaf(v.y, f, O.y), O.z = fmaf(v.z, f, O.z), O.w = fmaf(v.w, f, O.w);
      }
      if (c.np == 1) {
        IO *to = static_cast<IO *>(p.out) + (row0 + g) * D + col;
        *reinterpret_cast<decltype(raw4(to)) *>(to) = narrow4(make_float4(O.x / L, O.y / L, O.z / L, O.w / L), IO());
      } else {
        const size_t slot = (row0 + g) * p.num_partitions + c.part;
        *reinterpret_cast<float4 *>(p.ws_acc + slot * D + col) = O;
        if (col == 0) {
          p.ws_m[slot] = merge_max(M, L);
          p.ws_l[slot] = L;
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(m_empty);
  }
  if (!ok && lane == 0) timeout();
}

// The codes of a pool, [N * B, Hk, D] bytes; a load is one head's rows of a block.
template <int D>
bool encode_codes(CUtensorMap *map, const void *pool, const pk_cache_desc &d) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(d.num_kv_heads),
                              cuuint64_t(d.num_blocks) * cuuint64_t(d.block_size)};
  const cuuint64_t strides[2] = {cuuint64_t(D), cuuint64_t(D) * cuuint64_t(d.num_kv_heads)};
  const cuuint32_t box[3] = {D, 1, cuuint32_t(d.block_size)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(pool), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename IO, int D, int BS>
pk_status launch(const RowsParams &p, const pk_cache_desc &d, cudaStream_t stream) {
  using S = Shape<IO, D, BS>;
  CUtensorMap kmap, vmap;
  if (!encode_codes<D>(&kmap, p.k_cache, d) || !encode_codes<D>(&vmap, p.v_cache, d)) return PK_ERR_CUDA;
  auto kern = attn_e4m3_kernel<IO, D, BS>;
  static std::atomic<uint64_t> ready{0};
  if (!smem_ready(kern, S::SMEM_BYTES, ready)) return PK_ERR_CUDA;
  const dim3 g = rows_grid(p);
  const int64_t units = int64_t(g.x) * g.y * g.z;
  if (units > INT32_MAX) return PK_ERR_UNSUPPORTED;
  kern<<<unsigned(units), kThreads, S::SMEM_BYTES, stream>>>(p, kmap, vmap);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

template <typename IO, int D>
pk_status run(const RowsParams &p, const pk_cache_desc &d, cudaStream_t stream) {
  const pk_status st = d.block_size == 8    ? launch<IO, D, 8>(p, d, stream)
                       : d.block_size == 16 ? launch<IO, D, 16>(p, d, stream)
                                            : launch<IO, D, 32>(p, d, stream);
  if (st != PK_OK || p.num_partitions == 1) return st;
  return launch_rows_merge<IO, D>(p, stream);
}

}  // namespace

// The launch bounds ask for 3, and the shared memory allows them (head_dim 128:
// 3 x 72 KB, fp32 queries 76); the planner fills that many.
extern "C" int pkx_e4m3_resident_ctas(int, int) { return 3; }

extern "C" pk_status pk_paged_attention_decode_e4m3(
    void *out, const void *q, pk_dtype io_dtype, const void *k_cache, const void *v_cache,
    const uint8_t *kv_exp, const int32_t *block_tables, const int32_t *context_lens, float scale,
    int32_t num_seqs, int32_t num_q_heads, int32_t max_blocks_per_seq, int32_t max_context_len,
    int32_t partition_size, const int32_t *work_items, int32_t num_items, void *workspace,
    size_t workspace_bytes, const pk_cache_desc *desc, void *stream) {
  if (!desc) return PK_ERR_INVALID_ARG;
  if (desc->dtype != PK_E4M3 || (io_dtype != PK_F32 && io_dtype != PK_BF16))
    return PK_ERR_UNSUPPORTED;
  const int32_t part = pk_paged_attention_resolve_partition(num_seqs, num_q_heads, max_context_len,
                                                            partition_size, desc);
  if (part < 0) return PK_ERR_INVALID_ARG;
  if (desc->block_size != 8 && desc->block_size != 16 && desc->block_size != 32)
    return PK_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PK_OK;
  if (!kv_exp || !aligned16(kv_exp)) return PK_ERR_INVALID_ARG;
  RowsParams p{};
  pk_status st = rows_params(p, out, q, k_cache, v_cache, block_tables, context_lens, scale, num_seqs,
                             num_seqs, 1, num_q_heads, max_blocks_per_seq, max_context_len, part,
                             work_items, num_items, workspace, workspace_bytes, *desc);
  if (st != PK_OK) return st;
  p.kv_exp = kv_exp;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (io_dtype == PK_F32) return desc->head_dim == 128 ? run<float, 128>(p, *desc, s) : run<float, 64>(p, *desc, s);
  return desc->head_dim == 128 ? run<__nv_bfloat16, 128>(p, *desc, s)
                               : run<__nv_bfloat16, 64>(p, *desc, s);
}

}  // namespace pk
