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
// Data movement bounds it: every input is read once and every output written
// once, and a head costs about 7 operations per element. What decides is how much
// a warp has under way before its first result: 8192 tokens of 32 + 2 x 8 heads
// of 128 (bf16, 222 MB with the rotations) take 44.8 us, 4.96 TB/s, with four rounds of loads first;
// 67.6 us with one, 55.3 with two, 53.3 with eight (registers leave too few warps).
// A decode step's 64 tokens take 2.3 us on the device: latency, not bytes.
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
  float inv_d;
  uint32_t warps;               // warps of a token
  int32_t heads;                // heads of a token that have work: Hq + Hk (+ Hk values)
};

// Rounds per warp: 4 from this many heads on, else 1. Fewer heads leave SMs idle
// and one round is the shorter way through; more are bounded by the bytes under
// way. Device times with one and four rounds, bf16, 48 heads of 128 a token: 768
// heads 1.9 and 2.9 us, 12 288 heads 4.06 and 4.09, 16 320 heads 5.0 and 4.7,
// 24 576 heads 6.5 and 5.4, 393 216 heads 65 and 42.
constexpr int64_t kManyHeads = 16384;

// A head is d / 8 of LANES lanes (a power of two), each with two chunks of four
// elements that hold whole pairs, so that the rotation stays in the lane: with
// halves apart, chunks 4 l and rotary_dim / 2 + 4 l; with neighbouring pairs, and
// past the rotated elements, two chunks side by side. Either way the lane's four
// cosines and sines are those from 4 l on. A warp holds 32 / LANES heads of one
// token at a time and does U such rounds, all loaded before the first is
// computed; the token's cosines and sines are loaded once.
template <typename T, int LANES, int U>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(RopeParams p) {
  constexpr int HPW = 32 / LANES;  // heads of a round
  using Raw = decltype(pk::raw4(static_cast<const T *>(nullptr)));
  const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5), warps = p.warps;
  const uint32_t t = unit / warps;
  if (t >= uint32_t(p.num_tokens)) return;
  const int64_t tok = t;
  const int lane = threadIdx.x % LANES;
  const int first = int(unit - t * warps) * HPW * U + (threadIdx.x & 31) / LANES;
  const int64_t pos = p.rot ? __ldg(p.positions + tok) : 0;
  int64_t slot = p.slots ? __ldg(p.slots + tok) : -1;
  const bool in = lane * 8 < p.d, turn = lane * 8 < p.rot;
  const bool apart = turn && !p.interleaved;
  const int ea = apart ? 4 * lane : 8 * lane, eb = apart ? p.rot / 2 + 4 * lane : 8 * lane + 4;
  // Bases such that head * d leads to the head, whichever of the three it is.
  const T *const in_q = static_cast<const T *>(p.q) + tok * p.q_stride;
  const T *const in_k = static_cast<const T *>(p.k) + tok * p.k_stride - p.hq * p.d;
  const T *const in_v = static_cast<const T *>(p.v) + tok * p.v_stride - (p.hq + p.hk) * p.d;
  Raw ra[U], rb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int head = first + u * HPW;
    ra[u] = rb[u] = Raw{};
    if (!in || head >= p.heads) continue;
    const T *src = (head < p.hq ? in_q : (head < p.hq + p.hk ? in_k : in_v)) + head * p.d;
    ra[u] = pk::raw4(src + ea);
    rb[u] = pk::raw4(src + eb);
  }
  if (p.rot && (pos < 0 || pos >= p.max_position)) {  // the whole token: recorded and skipped
    if ((threadIdx.x & 31) == 0 && first == 0)
      pk::record_error(&g_qk_norm_rope_error, PK_DEVERR_POSITION, tok);
    return;
  }
  if (slot >= p.num_slots) {
    if ((threadIdx.x & 31) == 0 && first == 0)
      pk::record_error(&g_qk_norm_rope_error, PK_DEVERR_SLOT, tok);
    slot = -1;
  }
  float4 c, s;
  if (turn) {
    const float *cs = p.cos_sin + pos * p.rot + 4 * lane;
    c = __ldg(reinterpret_cast<const float4 *>(cs));
    s = __ldg(reinterpret_cast<const float4 *>(cs + p.rot / 2));
  }
  T *const to_q = static_cast<T *>(p.q_out) + tok * p.hq * p.d;
  T *const to_k = p.k_out ? static_cast<T *>(p.k_out) + (tok * p.hk - p.hq) * p.d : nullptr;
  T *const cache_k = static_cast<T *>(p.k_cache) + (slot * p.hk - p.hq) * p.d;
  T *const cache_v = static_cast<T *>(p.v_cache) + (slot * p.hk - p.hq - p.hk) * p.d;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int head = first + u * HPW;
    const bool is_q = head < p.hq, on = in && head < p.heads;
    if (__all_sync(0xffffffffu, head >= p.hq + p.hk)) {  // values, or nothing: as they are
      if (on && slot >= 0) {
        *reinterpret_cast<Raw *>(cache_v + head * p.d + ea) = ra[u];
        *reinterpret_cast<Raw *>(cache_v + head * p.d + eb) = rb[u];
      }
      continue;
    }
    const bool value = head >= p.hq + p.hk;
    float4 a = pk::widen4(ra[u]), b = pk::widen4(rb[u]);
    if (p.q_weight) {  // every lane of the warp takes part in the shuffles
      float ss = a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w;
      ss += b.x * b.x + b.y * b.y + b.z * b.z + b.w * b.w;
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!value && on) {
        const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
        const T *w = static_cast<const T *>(is_q ? p.q_weight : p.k_weight);
        const float4 ga = pk::widen4(pk::raw4(w + ea)), gb = pk::widen4(pk::raw4(w + eb));
        a.x *= r * ga.x, a.y *= r * ga.y, a.z *= r * ga.z, a.w *= r * ga.w;
        b.x *= r * gb.x, b.y *= r * gb.y, b.z *= r * gb.z, b.w *= r * gb.w;
      }
    }
    if (!on) continue;
    if (turn && !value) {
      const float4 x = a, y = b;
      if (apart) {
        a = make_float4(x.x * c.x - y.x * s.x, x.y * c.y - y.y * s.y, x.z * c.z - y.z * s.z, x.w * c.w - y.w * s.w);
        b = make_float4(y.x * c.x + x.x * s.x, y.y * c.y + x.y * s.y, y.z * c.z + x.z * s.z, y.w * c.w + x.w * s.w);
      } else {
        a = make_float4(x.x * c.x - x.y * s.x, x.y * c.x + x.x * s.x, x.z * c.y - x.w * s.y, x.w * c.y + x.z * s.y);
        b = make_float4(y.x * c.z - y.y * s.z, y.y * c.z + y.x * s.z, y.z * c.w - y.w * s.w, y.w * c.w + y.z * s.w);
      }
    }
    const Raw oa = value ? ra[u] : pk::narrow4(a, T()), ob = value ? rb[u] : pk::narrow4(b, T());
    auto put = [&](T *to) {
      *reinterpret_cast<Raw *>(to + head * p.d + ea) = oa;
      *reinterpret_cast<Raw *>(to + head * p.d + eb) = ob;
    };
    if (is_q) {
      put(to_q);
    } else {
      if (to_k && !value) put(to_k);
      if (slot >= 0) put(value ? cache_v : cache_k);
    }
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T>
pk_status launch(RopeParams p, cudaStream_t stream) {
  auto go = [&](auto lanes_c, auto rounds_c) {
    constexpr int L = decltype(lanes_c)::value, U = decltype(rounds_c)::value;
    p.warps = (p.heads + 32 / L * U - 1) / (32 / L * U);
    const int64_t units = int64_t(p.num_tokens) * p.warps;
    if (units > INT32_MAX) return PK_ERR_UNSUPPORTED;
    qk_norm_rope_kernel<T, L, U><<<unsigned((units + 7) / 8), 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
  };
  using std::integral_constant;
  auto by_lanes = [&](auto rounds_c) {
    if (p.d <= 64) return go(integral_constant<int, 8>(), rounds_c);
    if (p.d <= 128) return go(integral_constant<int, 16>(), rounds_c);
    return go(integral_constant<int, 32>(), rounds_c);
  };
  return int64_t(p.num_tokens) * p.heads >= kManyHeads ? by_lanes(integral_constant<int, 4>())
                                                       : by_lanes(integral_constant<int, 1>());
}

}  // namespace

extern "C" int *pkx_qk_norm_rope_error_word() { return pk::error_word(g_qk_norm_rope_error); }

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
  p.inv_d = 1.0f / float(d);
  p.interleaved = interleaved ? 1 : 0;
  p.heads = num_q_heads + hk + (cache ? hk : 0);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return desc->dtype == PK_F32 ? launch<float>(p, s) : launch<__nv_bfloat16>(p, s);
}
