// The 8-bit cache: new tokens' K/V quantised as they are written
// (pk_reshape_and_cache_e4m3), read back (pk_gather_cache_e4m3), and the
// copy-on-write block copy (pk_copy_blocks_e4m3).
//
// A row is one token's K or V of one KV head, d values. It is held as d e4m3
// codes and one power of two:
//     e = the smallest integer >= -100 with 448 * 2^e >= max |x|   (finite x)
//     code = e4m3(x * 2^-e), nearest even;      value = code * 2^e
// and kv_exp holds e + 127. A power of two loses no precision against a scale
// of max / 448 (e4m3 is a floating format: at most one step of its 2^15 range
// is given up), the product x * 2^-e is exact, so each code is one rounding of
// its input whatever computes it, every value is exact in bf16, and values that
// are written again stay what they are.
//
// Data movement bounds all three kernels. A row of K and the same row of V are
// loaded before either is converted. Written, a lane has 16 elements of each: the
// row's magnitude is a maximum over the bits, two bf16 at a time, and 16 codes are
// stored at once. 16 000 tokens of 8 heads of 128 (bf16) take 18.6 us, 5.3 TB/s, and
// 32 768 take 31.4, 6.4 TB/s; widening each value first and testing it for infinity
// took 23.9 for the former, bounded by instructions, and eight elements a lane 22.5.
// Read back, a lane has the elements of 16 bytes of the result, of two rows, so that
// a warp's stores are whole lines: 32 768 such tokens take 34.8 us, 5.8 TB/s, as fp32
// 56; 16 codes a lane took 37.4 and 74, one row a lane 38.5 and 64, four 36.9 and 56.
// Copied, 4096 pairs of blocks of 16 such tokens (270 MB moved) take 59 us, 4.6 TB/s:
// a thread has one 16-byte vector; 64 pairs 7.4 us.
// Up to some hundred tokens a call is bounded by its launch.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "pagedkv.h"
#include "pk_device.cuh"

namespace {

__device__ int g_cache_e4m3_error;

struct RowParams {
  const void *k, *v;           // [T, Hk, d] rows of token i at i * stride elements
  int64_t k_stride, v_stride;
  void *k_out, *v_out;         // read back: [T, Hk, d]
  const int64_t *slots;        // [T]
  uint8_t *k_cache, *v_cache;  // [N, B, Hk, d]
  uint8_t *kv_exp;             // [N, Hk, B, 2]
  int64_t num_slots;
  int32_t num_tokens, hk, d, block_size;
};

// LANES lanes of E elements hold a head's row of K and its row of V, both of
// which are loaded before either is converted.
struct Place {
  int64_t tok, slot, exp;  // exp: index of the pair of exponents
  int h, e0;
};

template <int LANES, int E>
__device__ __forceinline__ bool place_of(const RowParams &p, uint32_t unit, Place &at) {
  const uint32_t t = unit / uint32_t(p.hk);
  at.tok = t;
  at.h = int(unit - t * p.hk);
  at.e0 = (threadIdx.x % LANES) * E;
  if (at.tok >= p.num_tokens) return false;
  at.slot = __ldg(p.slots + at.tok);
  if (at.slot >= p.num_slots) {
    if (at.e0 == 0 && at.h == 0) pk::record_error(&g_cache_e4m3_error, PK_DEVERR_SLOT, at.tok);
    return false;
  }
  if (at.slot < 0) return false;
  const int64_t block = int32_t(at.slot) / p.block_size;  // slots fit 32 bits
  at.exp = (block * p.hk + at.h) * p.block_size + (at.slot - block * p.block_size);
  return at.e0 < p.d;
}

// A lane's 16 values of a row, as they are stored.
struct Row16F {
  float4 x[4];
  __device__ __forceinline__ void load(const float *p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = reinterpret_cast<const float4 *>(p)[i];
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return i & 1 ? make_float2(x[i / 2].z, x[i / 2].w) : make_float2(x[i / 2].x, x[i / 2].y);
  }
  // The largest magnitude as the bits of an fp32 (their order is the values').
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = pair(i);
      t = max(t, max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu));
    }
    return t;
  }
};
struct Row16B {
  uint4 x[2];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    x[0] = reinterpret_cast<const uint4 *>(p)[0];
    x[1] = reinterpret_cast<const uint4 *>(p)[1];
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4 &v = x[i / 4];
    return i % 4 == 0 ? v.x : (i % 4 == 1 ? v.y : (i % 4 == 2 ? v.z : v.w));
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2(pk::bf16_lo(word(i)), pk::bf16_hi(word(i)));
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;  // two 16-bit maxima
#pragma unroll
    for (int i = 0; i < 8; ++i) t = __vmaxu2(t, word(i) & 0x7fff7fffu);
    return max(t << 16, t & 0xffff0000u);
  }
};
template <typename T>
struct Row16Of;
template <>
struct Row16Of<float> {
  using Type = Row16F;
};
template <>
struct Row16Of<__nv_bfloat16> {
  using Type = Row16B;
};

// The exponent e of a row of LANES lanes, and the lane's codes. Infinities and
// NaN are rare: whether the warp has any is asked first.
template <int LANES, typename Row>
__device__ __forceinline__ int quantize16(const Row &row, uint4 &codes) {
  constexpr uint32_t INF = 0x7f800000u;
  uint32_t top = row.top();
  const bool odd = __any_sync(0xffffffffu, top >= INF);
  if (odd) {  // the largest finite magnitude
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = row.pair(i);
      const uint32_t a = __float_as_uint(v.x) & 0x7fffffffu, b = __float_as_uint(v.y) & 0x7fffffffu;
      top = max(top, max(a < INF ? a : 0u, b < INF ? b : 0u));
    }
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  // With top = f * 2^E, 1 <= f < 2: e = E - 8 where f <= 1.75 = 448 / 256, else
  // E - 7. Adding 0x1fffff carries into the exponent exactly where f > 1.75.
  const int e = top == 0 ? 0 : max(int((top + 0x1fffffu) >> 23) - 127 - 8, -100);
  const float s = __uint_as_float(uint32_t(127 - e) << 23);  // 2^-e: e is in [-100, 120]
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 v = row.pair(i);
    v.x *= s;
    v.y *= s;
    if (odd) {  // infinities become the NaN code too: the conversion would saturate them
      if (!(fabsf(row.pair(i).x) <= 3.402823466e38f)) v.x = __uint_as_float(0x7fc00000u);
      if (!(fabsf(row.pair(i).y) <= 3.402823466e38f)) v.y = __uint_as_float(0x7fc00000u);
    }
    w[i] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
  }
  codes = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  return e;
}

template <typename T, int LANES>
__global__ void __launch_bounds__(256) quantize_kernel(RowParams p) {
  Place at;
  const bool on = place_of<LANES, 16>(p, blockIdx.x * (256 / LANES) + threadIdx.x / LANES, at);
  typename Row16Of<T>::Type k{}, v{};
  if (on) {
    k.load(static_cast<const T *>(p.k) + at.tok * p.k_stride + int64_t(at.h) * p.d + at.e0);
    v.load(static_cast<const T *>(p.v) + at.tok * p.v_stride + int64_t(at.h) * p.d + at.e0);
  }
  uint4 kc, vc;
  const int ke = quantize16<LANES>(k, kc), ve = quantize16<LANES>(v, vc);
  if (!on) return;
  const int64_t to = (at.slot * p.hk + at.h) * p.d + at.e0;
  *reinterpret_cast<uint4 *>(p.k_cache + to) = kc;
  *reinterpret_cast<uint4 *>(p.v_cache + to) = vc;
  if (at.e0 == 0)
    *reinterpret_cast<uint16_t *>(p.kv_exp + at.exp * 2) = uint16_t((ke + 127) | (ve + 127) << 8);
}

// Two codes as fp32 values.
__device__ __forceinline__ float2 values_of(uint32_t pair, float s) {
  const float2 f =
      __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(pair & 0xffffu), __NV_E4M3)));
  return make_float2(f.x * s, f.y * s);
}
__device__ __forceinline__ void store_values(float *dst, uint32_t c, uint32_t exp) {
  const float s = __uint_as_float(exp << 23);
  const float2 a = values_of(c, s), b = values_of(c >> 16, s);
  *reinterpret_cast<float4 *>(dst) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_values(__nv_bfloat16 *dst, const uint2 &c, uint32_t exp) {
  const float s = __uint_as_float(exp << 23);
  const float2 x[4] = {values_of(c.x, s), values_of(c.x >> 16, s), values_of(c.y, s), values_of(c.y >> 16, s)};
  *reinterpret_cast<uint4 *>(dst) = make_uint4(pk::pack_bf16x2(x[0].x, x[0].y), pk::pack_bf16x2(x[1].x, x[1].y),
                                               pk::pack_bf16x2(x[2].x, x[2].y), pk::pack_bf16x2(x[3].x, x[3].y));
}

constexpr int kGatherRows = 2;  // of a lane, all loaded before the first is stored

// A lane writes 16 bytes of a row, so that a warp's stores are whole lines.
template <typename T, int LANES>
__global__ void __launch_bounds__(256) gather_kernel(RowParams p) {
  constexpr int E = 16 / int(sizeof(T)), U = kGatherRows;
  using Codes = typename std::conditional<E == 4, uint32_t, uint2>::type;
  Place at[U];
  bool on[U];
  Codes k[U], v[U];
  uint32_t e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    on[u] = place_of<LANES, E>(p, (blockIdx.x * U + u) * (256 / LANES) + threadIdx.x / LANES, at[u]);
    if (!on[u]) continue;
    const int64_t from = (at[u].slot * p.hk + at[u].h) * p.d + at[u].e0;
    k[u] = __ldg(reinterpret_cast<const Codes *>(p.k_cache + from));
    v[u] = __ldg(reinterpret_cast<const Codes *>(p.v_cache + from));
    e[u] = __ldg(reinterpret_cast<const uint16_t *>(p.kv_exp + at[u].exp * 2));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!on[u]) continue;
    const int64_t to = (at[u].tok * p.hk + at[u].h) * p.d + at[u].e0;
    store_values(static_cast<T *>(p.k_out) + to, k[u], e[u] & 0xffu);
    store_values(static_cast<T *>(p.v_out) + to, v[u], e[u] >> 8);
  }
}

// grid.x = pair, grid.y = 0 K codes / 1 V codes / 2 exponents, grid.z = chunk
// of 16-byte vectors (bytes where the exponents of a block are no multiple).
__global__ void __launch_bounds__(256) copy_blocks_e4m3_kernel(
    uint8_t *k_cache, uint8_t *v_cache, uint8_t *kv_exp, const int64_t *__restrict__ pairs,
    int32_t num_blocks, int64_t code_bytes, int64_t exp_bytes) {
  const int64_t src = pairs[2 * blockIdx.x], dst = pairs[2 * blockIdx.x + 1];
  if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
      pk::record_error(&g_cache_e4m3_error, PK_DEVERR_PAIR, blockIdx.x);
    return;
  }
  const int64_t n = blockIdx.y == 2 ? exp_bytes : code_bytes;
  uint8_t *pool = blockIdx.y == 0 ? k_cache : (blockIdx.y == 1 ? v_cache : kv_exp);
  const uint8_t *from = pool + src * n;
  uint8_t *to = pool + dst * n;
  const int64_t i = int64_t(blockIdx.z) * 256 + threadIdx.x;
  if (n % 16 == 0) {
    if (i < n / 16) reinterpret_cast<uint4 *>(to)[i] = reinterpret_cast<const uint4 *>(from)[i];
  } else {
    for (int64_t j = 16 * i; j < min(n, 16 * i + 16); ++j) to[j] = from[j];
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pk_status check_desc_e4m3(const pk_cache_desc *d) {
  if (!d || d->num_blocks <= 0 || d->block_size <= 0 || d->num_kv_heads <= 0 || d->head_dim <= 0)
    return PK_ERR_INVALID_ARG;
  if (d->dtype != PK_E4M3) return PK_ERR_UNSUPPORTED;
  if (d->head_dim % 16 != 0 || d->head_dim > 256) return PK_ERR_UNSUPPORTED;
  if (int64_t(d->num_kv_heads) * d->head_dim > INT32_MAX ||
      int64_t(d->num_blocks) * d->block_size > INT32_MAX)
    return PK_ERR_UNSUPPORTED;
  return PK_OK;
}

// Calls f with the lanes that a row takes at E elements each, and with the grid for
// `rows` rows a lane.
template <int E, typename F>
pk_status by_lanes(const RowParams &p, int rows, F f) {
  const int64_t units = int64_t(p.num_tokens) * p.hk;
  auto go = [&](auto c) {
    constexpr int L = decltype(c)::value;
    const int64_t per = 256 / L * rows, ctas = (units + per - 1) / per;
    if (units > INT32_MAX) return PK_ERR_UNSUPPORTED;
    f(c, unsigned(ctas));
    return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
  };
  if (p.d <= 64) return go(std::integral_constant<int, 64 / E>());
  if (p.d <= 128) return go(std::integral_constant<int, 128 / E>());
  return go(std::integral_constant<int, 256 / E>());
}

}  // namespace

extern "C" int *pkx_cache_e4m3_error_word() { return pk::error_word(g_cache_e4m3_error); }

extern "C" {

pk_status pk_reshape_and_cache_e4m3(const void *k, const void *v, pk_dtype src_dtype,
                                    int64_t k_stride, int64_t v_stride,
                                    const int64_t *slot_mapping, int32_t num_tokens, void *k_cache,
                                    void *v_cache, uint8_t *kv_exp, const pk_cache_desc *desc,
                                    void *stream) {
  pk_status st = check_desc_e4m3(desc);
  if (st != PK_OK) return st;
  if (num_tokens < 0) return PK_ERR_INVALID_ARG;
  if (src_dtype != PK_F32 && src_dtype != PK_BF16) return PK_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PK_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache || !kv_exp) return PK_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(kv_exp))
    return PK_ERR_INVALID_ARG;
  const int64_t row = int64_t(desc->num_kv_heads) * desc->head_dim;
  const int64_t esz = src_dtype == PK_F32 ? 4 : 2;
  if (k_stride < row || v_stride < row || k_stride * esz % 16 != 0 || v_stride * esz % 16 != 0)
    return PK_ERR_INVALID_ARG;
  RowParams p{};
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slot_mapping;
  p.k_cache = static_cast<uint8_t *>(k_cache);
  p.v_cache = static_cast<uint8_t *>(v_cache);
  p.kv_exp = kv_exp;
  p.num_slots = int64_t(desc->num_blocks) * desc->block_size;
  p.num_tokens = num_tokens;
  p.hk = desc->num_kv_heads;
  p.d = desc->head_dim;
  p.block_size = desc->block_size;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_lanes<16>(p, 1, [&](auto c, unsigned ctas) {
    constexpr int L = decltype(c)::value;
    if (src_dtype == PK_F32)
      quantize_kernel<float, L><<<ctas, 256, 0, s>>>(p);
    else
      quantize_kernel<__nv_bfloat16, L><<<ctas, 256, 0, s>>>(p);
  });
}

pk_status pk_gather_cache_e4m3(void *k_out, void *v_out, pk_dtype out_dtype,
                               const int64_t *slot_mapping, int32_t num_tokens, const void *k_cache,
                               const void *v_cache, const uint8_t *kv_exp,
                               const pk_cache_desc *desc, void *stream) {
  pk_status st = check_desc_e4m3(desc);
  if (st != PK_OK) return st;
  if (num_tokens < 0) return PK_ERR_INVALID_ARG;
  if (out_dtype != PK_F32 && out_dtype != PK_BF16) return PK_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PK_OK;
  if (!k_out || !v_out || !slot_mapping || !k_cache || !v_cache || !kv_exp) return PK_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(kv_exp))
    return PK_ERR_INVALID_ARG;
  RowParams p{};
  p.k_out = k_out;
  p.v_out = v_out;
  p.slots = slot_mapping;
  p.k_cache = static_cast<uint8_t *>(const_cast<void *>(k_cache));
  p.v_cache = static_cast<uint8_t *>(const_cast<void *>(v_cache));
  p.kv_exp = const_cast<uint8_t *>(kv_exp);
  p.num_slots = int64_t(desc->num_blocks) * desc->block_size;
  p.num_tokens = num_tokens;
  p.hk = desc->num_kv_heads;
  p.d = desc->head_dim;
  p.block_size = desc->block_size;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (out_dtype == PK_F32)
    return by_lanes<4>(p, kGatherRows, [&](auto c, unsigned ctas) {
      gather_kernel<float, decltype(c)::value><<<ctas, 256, 0, s>>>(p);
    });
  return by_lanes<8>(p, kGatherRows, [&](auto c, unsigned ctas) {
    gather_kernel<__nv_bfloat16, decltype(c)::value><<<ctas, 256, 0, s>>>(p);
  });
}

pk_status pk_copy_blocks_e4m3(void *k_cache, void *v_cache, uint8_t *kv_exp,
                              const int64_t *src_dst_pairs, int32_t num_pairs,
                              const pk_cache_desc *desc, void *stream) {
  pk_status st = check_desc_e4m3(desc);
  if (st != PK_OK) return st;
  if (num_pairs < 0) return PK_ERR_INVALID_ARG;
  if (num_pairs == 0) return PK_OK;
  if (!k_cache || !v_cache || !kv_exp || !src_dst_pairs) return PK_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(kv_exp)) return PK_ERR_INVALID_ARG;
  const int64_t tokens = int64_t(desc->block_size) * desc->num_kv_heads;
  const int64_t code_bytes = tokens * desc->head_dim, exp_bytes = tokens * 2;
  const int64_t chunks = (code_bytes / 16 + 255) / 256;
  if (chunks > 65535) return PK_ERR_UNSUPPORTED;
  copy_blocks_e4m3_kernel<<<dim3(unsigned(num_pairs), 3, unsigned(chunks)), 256, 0,
                            static_cast<cudaStream_t>(stream)>>>(
      static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), kv_exp, src_dst_pairs,
      desc->num_blocks, code_bytes, exp_bytes);
  return cudaGetLastError() == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // extern "C"
