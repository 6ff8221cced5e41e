// paged_kv_write_q4 and paged_kv_unpack_q4: rows packed into the 4-bit cache, blocks of it back as values
// (format: q4_common.cuh).
//
// Packing.  Of 64 values: lo = min(0, min x), hi = max(0, max x), scale = bf16(fp32(hi / 15) - fp32(lo / 15)),
// zero = round(-lo / scale), code = round(x / scale) + zero, both clamped to 0 .. 15.  (Zero is on the grid, so
// x / scale is rounded by itself.)  The quotients are rounded to the nearest whole number, halves to the even one,
// as real numbers: with r the nearest to x * (1 / scale) in 32 bits, the remainder x - r * scale is exact wherever
// it decides (r * scale has 13 bits, and next to a half the remainder fits 24), so comparing it with scale / 2
// says whether r is right.  What a value is packed to therefore depends on nothing but the definition.
// A group that holds a value that is not finite gets scale NaN, and all its values are NaN.
#include <float.h>

#include <algorithm>

#include "pa_internal.h"
#include "q4_common.cuh"

namespace pa {

constexpr int kQ4Threads = 256;
constexpr int kQ4Vals = 8;                          // values of a thread
constexpr int kQ4Lanes = kQ4Group / kQ4Vals;        // threads of a group

// Eight consecutive values as 32-bit numbers.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    Elt<T>::unpack(ld_stream16(p), x);
  } else {
    float lo[4], hi[4];
    Elt<float>::unpack(ld_stream16(p), lo);
    Elt<float>::unpack(ld_stream16(p + 4), hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = lo[i];
      x[4 + i] = hi[i];
    }
  }
}

// The whole number nearest to x / s (halves to the even one), exactly; |x / s| < 2^20, inv = 1 / s in 32 bits.
__device__ __forceinline__ int q4_round(float x, float s, float inv) {
  float r = rintf(x * inv);
  const float e = fmaf(-r, s, x), h = 0.5f * s;
  const bool odd = ((int)r & 1) != 0;
  if (e > h || (odd && e == h)) r += 1.f;
  else if (e < -h || (odd && e == -h)) r -= 1.f;
  return (int)r;
}

// Packs the eight values of a thread; the kQ4Lanes threads of a group (a part of a warp, all of it here) work
// together.  Returns the codes; pair: the group's (scale, zero).
__device__ __forceinline__ uint32_t q4_pack8(const float (&x)[8], uint32_t& pair) {
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int off = 1; off < kQ4Lanes; off <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  const float s = __bfloat162float(__float2bfloat16_rn(__fsub_rn(__fdiv_rn(hi, 15.f), __fdiv_rn(lo, 15.f))));
  if (!(s <= FLT_MAX)) {  // a value that is not finite
    pair = 0x7fc0u;       // NaN, 0
    return 0u;
  }
  if (s < FLT_MIN) {  // nothing but zeros, or next to nothing
    pair = 0u;
    return 0u;
  }
  const float inv = 1.f / s;
  const int z = min(max(q4_round(-lo, s, inv), 0), 15);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) codes |= (uint32_t)min(max(q4_round(x[i], s, inv) + z, 0), 15) << (4 * i);
  pair = (__float_as_uint(s) >> 16) | (__float_as_uint((float)z) & 0xffff0000u);
  return codes;
}

// Thread (token, KV head and group, eighth of it), K and V.  Bound by HBM.
template <typename T>
__global__ void __launch_bounds__(kQ4Threads) kv_write_q4_kernel(const Q4WriteArgs a) {
  const int64_t idx = (int64_t)blockIdx.x * kQ4Threads + threadIdx.x;
  // (whole groups: the lanes of one are all here or all past the end; rows are computed even if nothing is written,
  // so that the lanes of a warp stay together)
  const int64_t t = min(idx / a.row_lanes, a.n_tokens - 1);
  const int c = (int)(idx - idx / a.row_lanes * a.row_lanes);
  int64_t slot = __ldg(a.slot_mapping + t);
  if (idx >= a.n_tokens * a.row_lanes) slot = -1;
  if (slot >= a.total_slots) {
    if (c == 0) raise_error(a.err, PA_DEVERR_SLOT);
    slot = -1;
  }
  const int64_t src = (t * a.row_lanes + c) * kQ4Vals;
  float xk[8], xv[8];
  load8(static_cast<const T*>(a.k_new) + src, xk);
  load8(static_cast<const T*>(a.v_new) + src, xv);
  uint32_t pk, pv;
  const uint32_t ck = q4_pack8(xk, pk), cv = q4_pack8(xv, pv);
  if (slot < 0) return;
  const int64_t dst = slot * a.row_lanes + c;
  static_cast<uint32_t*>(a.k_codes)[dst] = ck;
  static_cast<uint32_t*>(a.v_codes)[dst] = cv;
  if (c % kQ4Lanes == 0) {
    static_cast<uint32_t*>(a.k_params)[dst / kQ4Lanes] = pk;
    static_cast<uint32_t*>(a.v_params)[dst / kQ4Lanes] = pv;
  }
}

cudaError_t launch_kv_write_q4(const Q4WriteArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  const int64_t blocks = (a.n_tokens * a.row_lanes + kQ4Threads - 1) / kQ4Threads;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  switch (dt) {
    case PA_BF16: kv_write_q4_kernel<__nv_bfloat16><<<(unsigned)blocks, kQ4Threads, 0, s>>>(a); break;
    case PA_FP16: kv_write_q4_kernel<__half><<<(unsigned)blocks, kQ4Threads, 0, s>>>(a); break;
    case PA_FP32: kv_write_q4_kernel<float><<<(unsigned)blocks, kQ4Threads, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  ++*launches;
  return cudaGetLastError();
}

// ------------------------------------------------------------------------------------------------
template <typename T>
struct Largest;
template <>
struct Largest<__nv_bfloat16> { static constexpr float kValue = 3.3895313892515355e38f; };
template <>
struct Largest<__half> { static constexpr float kValue = 65504.f; };
template <>
struct Largest<float> { static constexpr float kValue = FLT_MAX; };

// Eight values of a thread to memory.  The largest codes of a group may stand for a little more than the type's
// largest number (the scale is rounded): they become that.
template <typename T>
__device__ __forceinline__ void unpack8(uint32_t codes, uint32_t pair, T* p) {
  const float s = q4_scale(pair), z = q4_zero(pair);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = s * ((float)((codes >> (4 * i)) & 15u) - z);
    x[i] = max_nan(min_nan(v, Largest<T>::kValue), -Largest<T>::kValue);
  }
  alignas(16) T y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = Elt<T>::from_float(x[i]);
#pragma unroll
  for (int i = 0; i < (int)sizeof(y) / 16; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(y)[i];
}

constexpr int kQ4Unroll = 2;  // words of K and of V in flight per thread

// CTA (block pair, slice of it).  Bound by HBM: 72 bytes read and 256 written per row of 128 bf16 values.
template <typename T>
__global__ void __launch_bounds__(kQ4Threads) kv_unpack_q4_kernel(const Q4UnpackArgs a, const int slices) {
  const int64_t pair = blockIdx.x / slices;
  const int slice = (int)(blockIdx.x - pair * slices);
  const int64_t src = __ldg(a.pairs + 2 * pair), dst = __ldg(a.pairs + 2 * pair + 1);
  if (src < 0 || src >= a.cache_blocks || dst < 0 || dst >= a.num_blocks) {
    if (slice == 0 && threadIdx.x == 0) raise_error(a.err, PA_DEVERR_COPY_PAIR);
    return;
  }
  const uint32_t* kc = static_cast<const uint32_t*>(a.k_codes) + src * a.block_words;
  const uint32_t* vc = static_cast<const uint32_t*>(a.v_codes) + src * a.block_words;
  const uint32_t* kp = static_cast<const uint32_t*>(a.k_params) + src * (a.block_words / kQ4Lanes);
  const uint32_t* vp = static_cast<const uint32_t*>(a.v_params) + src * (a.block_words / kQ4Lanes);
  T* ko = static_cast<T*>(a.k_pool) + dst * a.block_stride;
  T* vo = static_cast<T*>(a.v_pool) + dst * a.block_stride;
  for (int w0 = slice * kQ4Threads * kQ4Unroll + threadIdx.x; w0 < a.block_words; w0 += slices * kQ4Threads * kQ4Unroll) {
    uint32_t c[kQ4Unroll][2], p[kQ4Unroll][2];
#pragma unroll
    for (int u = 0; u < kQ4Unroll; ++u) {
      const int w = w0 + u * kQ4Threads;
      if (w < a.block_words) {
        c[u][0] = __ldg(kc + w);
        c[u][1] = __ldg(vc + w);
        p[u][0] = __ldg(kp + w / kQ4Lanes);
        p[u][1] = __ldg(vp + w / kQ4Lanes);
      }
    }
#pragma unroll
    for (int u = 0; u < kQ4Unroll; ++u) {
      const int w = w0 + u * kQ4Threads;
      if (w < a.block_words) {
        unpack8<T>(c[u][0], p[u][0], ko + (int64_t)w * kQ4Vals);
        unpack8<T>(c[u][1], p[u][1], vo + (int64_t)w * kQ4Vals);
      }
    }
  }
}

cudaError_t launch_kv_unpack_q4(const Q4UnpackArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  if (a.n_pairs == 0) return cudaSuccess;
  const int slices = std::max(1, (a.block_words + kQ4Threads * kQ4Unroll - 1) / (kQ4Threads * kQ4Unroll));
  const int64_t grid = a.n_pairs * slices;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  switch (dt) {
    case PA_BF16: kv_unpack_q4_kernel<__nv_bfloat16><<<(unsigned)grid, kQ4Threads, 0, s>>>(a, slices); break;
    case PA_FP16: kv_unpack_q4_kernel<__half><<<(unsigned)grid, kQ4Threads, 0, s>>>(a, slices); break;
    case PA_FP32: kv_unpack_q4_kernel<float><<<(unsigned)grid, kQ4Threads, 0, s>>>(a, slices); break;
    default: return cudaErrorInvalidValue;
  }
  ++*launches;
  return cudaGetLastError();
}

}  // namespace pa
