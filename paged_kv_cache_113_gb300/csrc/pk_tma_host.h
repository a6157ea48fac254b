// Host side of TMA: the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

#include "pagedkv.h"

namespace pk {

// cuTensorMapEncodeTiled of the loaded driver, or null.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// A [N*B, Hk, D] bf16 view of one pool; each load is a box of B token rows of
// one head and 64 elements (128 bytes), swizzled 128B in shared memory.
inline bool encode_bf16_pool(CUtensorMap *map, const void *pool, const pk_cache_desc &d) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cuuint64_t(d.head_dim), cuuint64_t(d.num_kv_heads),
                              cuuint64_t(d.num_blocks) * cuuint64_t(d.block_size)};
  const cuuint64_t strides[2] = {cuuint64_t(d.head_dim) * 2,
                                 cuuint64_t(d.num_kv_heads) * cuuint64_t(d.head_dim) * 2};
  const cuuint32_t box[3] = {64, 1, cuuint32_t(d.block_size)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(pool), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pk
