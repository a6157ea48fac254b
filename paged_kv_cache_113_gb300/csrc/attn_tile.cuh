// The products of one warp's 16-token tile with up to eight rows of query, on mma.sync
// tensor cores (bf16): shared by decode attention and its form with changed scores. K and V
// lie in shared memory as D / 64 slabs of `slab` bytes (128-byte rows, 128B-swizzled); the
// tile is rows row0 .. row0 + 15.
#pragma once

#include "pk_device.cuh"

namespace pk {

// S^T = K_tile (16 x D) * Q^T (D x 8), as two independent accumulation chains (even and odd
// k-steps), to be added: lanes hold tokens lane / 4 and + 8, rows 2 (lane % 4) and + 1.
template <int KSTEPS>
__device__ __forceinline__ void tile_scores(uint32_t kbase, int slab, int row0, const uint32_t (&qb)[KSTEPS][2],
                                            float (&sacc)[2][4], int lane) {
  const int mi = lane >> 3, r8 = lane & 7;
#pragma unroll
  for (int e = 0; e < 4; ++e) sacc[0][e] = sacc[1][e] = 0.0f;
#pragma unroll
  for (int ks = 0; ks < KSTEPS; ++ks) {
    const int r = row0 + (mi & 1) * 8 + r8;
    const int chunk = ks * 2 + (mi >> 1);
    const uint32_t a = kbase + (chunk >> 3) * slab + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
    uint32_t a0, a1, a2, a3;
    ldmatrix_x4(a, a0, a1, a2, a3);
    mma_bf16_16816(sacc[ks & 1], a0, a1, a2, a3, qb[ks][0], qb[ks][1]);
  }
}

// O^T (D x 8) += V^T (D x 16 tokens) * P^T, the weights as a pair w + r of bf16 (01: of tokens
// lane / 4, 23: of those + 8): all w products first, then all r products, so consecutive MMAs
// never share an accumulator.
template <int KSTEPS>
__device__ __forceinline__ void tile_values(uint32_t vbase, int slab, int row0, uint32_t w01, uint32_t w23, uint32_t r01,
                                            uint32_t r23, float (&o)[KSTEPS][4], int lane) {
  const int mi = lane >> 3, r8 = lane & 7;
  // P^T (16 tokens x 8 heads) as the B operand: transpose the C fragments.
  const uint32_t b0 = movmatrix_trans(w01);
  const uint32_t b1 = movmatrix_trans(w23);
  const uint32_t e0 = movmatrix_trans(r01);
  const uint32_t e1 = movmatrix_trans(r23);
  uint32_t va[KSTEPS][4];
#pragma unroll
  for (int mt = 0; mt < KSTEPS; ++mt) {
    const int r = row0 + (mi >> 1) * 8 + r8;
    const int chunk = mt * 2 + (mi & 1);
    const uint32_t a = vbase + (chunk >> 3) * slab + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
    ldmatrix_x4_trans(a, va[mt][0], va[mt][1], va[mt][2], va[mt][3]);
  }
#pragma unroll
  for (int mt = 0; mt < KSTEPS; ++mt)
    mma_bf16_16816(o[mt], va[mt][0], va[mt][1], va[mt][2], va[mt][3], b0, b1);
#pragma unroll
  for (int mt = 0; mt < KSTEPS; ++mt)
    mma_bf16_16816(o[mt], va[mt][0], va[mt][1], va[mt][2], va[mt][3], e0, e1);
}

}  // namespace pk
