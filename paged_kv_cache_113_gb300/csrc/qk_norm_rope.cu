// Queries' and keys' per-head RMS norm, the position rotation and the cache
// write of a step's new tokens in one pass (pk_qk_norm_rope_and_cache).
//
// For each token i and query or key head, x being the head's d values:
//     y = x * (mean(x^2) + eps)^(-1/2) * w                 (with weights)
//     (a, b) -> (a c - b s, b c + a s)    over the first rotary_dim elements,
//                         c, s = cos_sin[positions[i]]; the rest unchanged.
// Everything between the load and the store is fp32 and each result is
// rounded once. The key goes to k_out and to its slot of the cache, the value
// to its slot.
//
// Pure data movement bounds it: every input is read once and every output
// written once, and a head costs about 7 operations per element.
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "pagedkv.h"
#include "pk_device.cuh"

namespace {

__device__ int g_qk_norm_rope_error;

struct RopeParams {
  const void *q, *k, *v;        // token i's heads at i * stride elements
  int64_t q_stride, k_stride, v_stride;
  void *q_out, *k_out;          // [T, Hq, d], [T, Hk, d] or null
  const void *q_weight, *k_weight;  // [d] or null (no norm)
  const float *cos_sin;         // [max_position, rot]: rot / 2 cosines, then sines
  const int64_t *positions;     // [T]
  const int64_t *slots;         // [T] or null (no cache write)
  void *k_cache, *v_cache;      // [N, B, Hk, d]
  int64_t num_slots;
  float eps;
  int32_t num_tokens, hq, hk, d, rot, max_position, interleaved;
  int32_t heads;                // heads of a token that have work: Hq + Hk (+ Hk values)
};

// A head is LANES lanes of eight elements each (LANES a power of two; lanes
// past the head's end carry zeros). Rotated pairs that lie in other lanes are
// exchanged with shuffles: rotary_dim / 2 is a multiple of eight, so a pair's
// two halves sit at the same place of two lanes.
template <typename T, int LANES>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(RopeParams p) {
  const int64_t unit = int64_t(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
  const int lane = threadIdx.x % LANES, e0 = lane * 8;
  const int64_t tok = unit / p.heads;
  const int head = int(unit % p.heads);
  bool live = tok < p.num_tokens;
  int64_t pos = 0, slot = -1;
  if (live && p.rot) {
    pos = __ldg(p.positions + tok);
    if (pos < 0 || pos >= p.max_position) {
      if (lane == 0 && head == 0) pk::record_error(&g_qk_norm_rope_error, PK_DEVERR_POSITION, tok);
      live = false;
    }
  }
  const bool is_q = head < p.hq, is_k = !is_q && head < p.hq + p.hk;
  const int h = is_q ? head : (is_k ? head - p.hq : head - p.hq - p.hk);
  if (live && !is_q && p.slots) {
    slot = __ldg(p.slots + tok);
    if (slot >= p.num_slots) {
      if (lane == 0 && is_k && h == 0)
        pk::record_error(&g_qk_norm_rope_error, PK_DEVERR_SLOT, tok);
      slot = -1;
    }
  }
  const bool on = live && e0 < p.d;
  const T *src = static_cast<const T *>(is_q ? p.q : (is_k ? p.k : p.v)) +
                 tok * (is_q ? p.q_stride : (is_k ? p.k_stride : p.v_stride)) + int64_t(h) * p.d + e0;
  float x[8] = {};
  if (on) pk::load8(src, x);
  // Every lane of the warp takes part in the shuffles, whatever its head is.
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const void *w = is_q ? p.q_weight : (is_k ? p.k_weight : nullptr);
  if (w && on) {
    const float r = 1.0f / sqrtf(ss / float(p.d) + p.eps);
    float g[8];
    pk::load8(static_cast<const T *>(w) + e0, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * g[i];
  }
  const int half = p.rot / 2;
  const bool turn = on && (is_q || is_k) && e0 < p.rot;
  if (p.interleaved) {
    if (turn) {
      const float *cs = p.cos_sin + pos * p.rot + e0 / 2;
      const float4 c = __ldg(reinterpret_cast<const float4 *>(cs));
      const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + half));
      const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * cc[i] - b * sn[i];
        x[2 * i + 1] = b * cc[i] + a * sn[i];
      }
    }
  } else {
    const bool upper = e0 >= half;
    const int other = e0 < p.rot ? (upper ? lane - half / 8 : lane + half / 8) : lane;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], other, LANES);
    if (turn) {
      const float *cs = p.cos_sin + pos * p.rot + (upper ? e0 - half : e0);
      float c[8], s[8];
      pk::load8(cs, c);
      pk::load8(cs + half, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * c[i] + (upper ? y[i] : -y[i]) * s[i];
    }
  }
  if (!on) return;
  const int64_t row = (tok * (is_q ? p.hq : p.hk) + h) * p.d + e0;
  if (is_q) {
    pk::store8(static_cast<T *>(p.q_out) + row, x);
    return;
  }
  if (is_k && p.k_out) pk::store8(static_cast<T *>(p.k_out) + row, x);
  if (slot >= 0)  // a value reaches here as it was loaded: the round trip through fp32 is exact
    pk::store8(static_cast<T *>(is_k ? p.k_cache : p.v_cache) + (slot * p.hk + h) * p.d + e0, x);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T>
pk_status launch(const RopeParams &p, cudaStream_t stream) {
  const int lanes = p.d / 8;
  auto go = [&](auto lanes_c) {
    constexpr int L = decltype(lanes_c)::value;
    const int64_t units = int64_t(p.num_tokens) * p.heads;
    const int64_t ctas = (units + 256 / L - 1) / (256 / L);
    if (ctas > INT32_MAX) return PK_ERR_UNSUPPORTED;
    qk_norm_rope_kernel<T, L><<<unsigned(ctas), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
  };
  if (lanes <= 8) return go(std::integral_constant<int, 8>());
  if (lanes <= 16) return go(std::integral_constant<int, 16>());
  return go(std::integral_constant<int, 32>());
}

}  // namespace

extern "C" int pkx_take_qk_norm_rope_error(cudaStream_t stream) {
  return pk::take_error_word(g_qk_norm_rope_error, stream);
}

extern "C" pk_status pk_qk_norm_rope_and_cache(
    void *q_out, void *k_out, const void *q, const void *k, const void *v, int64_t q_stride,
    int64_t k_stride, int64_t v_stride, const void *q_weight, const void *k_weight, float eps,
    const float *cos_sin, const int64_t *positions, int32_t max_position, int32_t rotary_dim,
    int32_t interleaved, const int64_t *slot_mapping, int32_t num_tokens, int32_t num_q_heads,
    void *k_cache, void *v_cache, const pk_cache_desc *desc, void *stream) {
  const bool cache = slot_mapping != nullptr;
  if (!desc || desc->num_kv_heads <= 0 || desc->head_dim <= 0 || num_q_heads <= 0 || num_tokens < 0)
    return PK_ERR_INVALID_ARG;
  if (cache && (desc->num_blocks <= 0 || desc->block_size <= 0)) return PK_ERR_INVALID_ARG;
  if (desc->dtype != PK_F32 && desc->dtype != PK_BF16) return PK_ERR_UNSUPPORTED;
  const int64_t esz = desc->dtype == PK_F32 ? 4 : 2;
  const int32_t d = desc->head_dim, hk = desc->num_kv_heads;
  if (d % 16 != 0 || d > 256) return PK_ERR_UNSUPPORTED;
  if (rotary_dim < 0 || rotary_dim > d || rotary_dim % 16 != 0) return PK_ERR_INVALID_ARG;
  if (int64_t(num_q_heads) * d > INT32_MAX || int64_t(hk) * d > INT32_MAX) return PK_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f)) return PK_ERR_INVALID_ARG;
  if (num_tokens == 0) return PK_OK;
  if (!q_out || !q || !k || (q_weight == nullptr) != (k_weight == nullptr)) return PK_ERR_INVALID_ARG;
  if (rotary_dim > 0 && (!cos_sin || !positions || max_position <= 0)) return PK_ERR_INVALID_ARG;
  if (cache ? (!v || !k_cache || !v_cache) : !k_out) return PK_ERR_INVALID_ARG;
  if (q_stride < int64_t(num_q_heads) * d || k_stride < int64_t(hk) * d ||
      (cache && v_stride < int64_t(hk) * d))
    return PK_ERR_INVALID_ARG;
  const void *ptrs[] = {q_out, k_out, q, k, cache ? v : nullptr, q_weight, k_weight, cos_sin,
                        cache ? k_cache : nullptr, cache ? v_cache : nullptr};
  for (const void *ptr : ptrs)
    if (!aligned16(ptr)) return PK_ERR_INVALID_ARG;
  if (q_stride * esz % 16 != 0 || k_stride * esz % 16 != 0 || (cache && v_stride * esz % 16 != 0))
    return PK_ERR_INVALID_ARG;
  // In place only where a head's result replaces exactly that head.
  if ((q_out == q && q_stride != int64_t(num_q_heads) * d) ||
      (k_out == k && k_stride != int64_t(hk) * d))
    return PK_ERR_INVALID_ARG;
  RopeParams p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.slots = slot_mapping;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.num_slots = int64_t(desc->num_blocks) * desc->block_size;
  p.eps = eps;
  p.num_tokens = num_tokens;
  p.hq = num_q_heads;
  p.hk = hk;
  p.d = d;
  p.rot = rotary_dim;
  p.max_position = max_position;
  p.interleaved = interleaved ? 1 : 0;
  p.heads = num_q_heads + hk + (cache ? hk : 0);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return desc->dtype == PK_F32 ? launch<float>(p, s) : launch<__nv_bfloat16>(p, s);
}
