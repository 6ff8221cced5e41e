// paged_kv_write_q4 and paged_kv_unpack_q4: rows packed into the 4-bit cache, blocks of it back as values
// (format: q4_common.cuh).
//
// Packing.  Of 64 values: lo = min(0, min x), hi = max(0, max x), scale = bf16(fp32(hi r) - fp32(lo r)), r = fp32(1 / 15),
// zero = round(-lo / scale), code = round(x / scale) + zero, both clamped to 0 .. 15.  (Zero is on the grid, so
// x / scale is rounded by itself.)  The quotients are rounded to the nearest whole number, halves to the even one, as real
// numbers, so that what a value is packed to depends on nothing but the definition:
//   16-bit values.  Their quotient by a scale of 8 bits is a half or at least 2^-12 away from one, so its fp32 rounding
//     decides.  That is formed from the rounded reciprocal and one exact remainder (Markstein's division): q = x / s
//     rounded, q += (x - q s) / s.
//   fp32 values.  With r the nearest to x * (1 / scale) in 32 bits, the remainder x - r * scale is exact wherever it
//     decides (r * scale has 13 bits, and next to a half the remainder fits 24), so comparing it with scale / 2 says
//     whether r is right.
// A group that holds a value that is not finite gets scale NaN, and all its values are NaN.
#include <float.h>

#include <algorithm>

#include "pa_internal.h"
#include "q4_common.cuh"

namespace pa {

constexpr int kQ4Threads = 256;
constexpr int kPackVals = 32;                       // values of a thread that packs
constexpr int kPackLanes = kQ4Group / kPackVals;    // threads of a group
constexpr int kPackCtas = 3;                        // CTAs of an SM, which take parts in turn
constexpr int kQ4Vals = 16;                         // the same for unpacking
constexpr int kQ4Lanes = kQ4Group / kQ4Vals;

// A thread's consecutive values.
template <typename T, int kWords>
__device__ __forceinline__ void load_raw(const T* p, bool aligned32, uint32_t (&v)[kWords]) {
#pragma unroll
  for (int i = 0; i < kWords; i += 8)
    ld_stream32(reinterpret_cast<const uint32_t*>(p) + i, *reinterpret_cast<uint32_t(*)[8]>(&v[i]), aligned32);
}

// They as 32-bit numbers, and the smallest and the largest of them and 0 (NaN if one is).
template <typename T>
__device__ __forceinline__ void unpack_raw(const uint32_t (&v)[kPackVals * sizeof(T) / 4], float (&x)[kPackVals], float& lo,
                                           float& hi) {
  constexpr int kVec = Elt<T>::kVec, kWords = kPackVals * (int)sizeof(T) / 4;
#pragma unroll
  for (int i = 0; i < kPackVals / kVec; ++i)
    Elt<T>::unpack(make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]), *reinterpret_cast<float(*)[kVec]>(&x[i * kVec]));
  if constexpr (sizeof(T) == 2) {  // two at a time
    uint32_t a = 0u, b = 0u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(v[i]));
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(v[i]));
      } else {
        asm("min.NaN.f16x2 %0, %0, %1;" : "+r"(a) : "r"(v[i]));
        asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(b) : "r"(v[i]));
      }
    }
    float f[8];
    Elt<T>::unpack(make_uint4(a, b, 0u, 0u), f);
    lo = min_nan(f[0], f[1]);
    hi = max_nan(f[2], f[3]);
  } else {
    lo = hi = 0.f;
#pragma unroll
    for (int i = 0; i < kPackVals; ++i) {
      lo = min_nan(lo, x[i]);
      hi = max_nan(hi, x[i]);
    }
  }
}

// The whole number nearest to x / s (halves to the even one), exactly; |x / s| < 2^20, inv = 1 / s in 32 bits.
__device__ __forceinline__ float q4_round(float x, float s, float inv) {
  float r = rintf(x * inv);
  const float e = fmaf(-r, s, x), h = 0.5f * s;
  const bool odd = ((int)r & 1) != 0;
  if (e > h || (odd && e == h)) r += 1.f;
  else if (e < -h || (odd && e == -h)) r -= 1.f;
  return r;
}

// Packs the values of a thread; the kPackLanes threads of a group (a part of a warp, all of it here) work
// together; lo, hi: of its own values.  Returns the codes; pair: the group's (scale, zero); kShort: values of at most 11 bits.
template <bool kShort>
__device__ __forceinline__ uint4 q4_pack(float (&x)[kPackVals], float lo, float hi, uint32_t& pair) {
#pragma unroll
  for (int off = 1; off < kPackLanes; off <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  const float s = __bfloat162float(__float2bfloat16_rn(__fsub_rn(__fmul_rn(hi, 1.f / 15.f), __fmul_rn(lo, 1.f / 15.f))));
  if (!(s <= FLT_MAX)) {  // a value that is not finite
    pair = 0x7fc0u;       // NaN, 0
    return make_uint4(0u, 0u, 0u, 0u);
  }
  if (s < FLT_MIN) {  // nothing but zeros, or next to nothing
    pair = 0u;
    return make_uint4(0u, 0u, 0u, 0u);
  }
  const float inv = 1.f / s;
  const float z = fminf(fmaxf(q4_round(-lo, s, inv), 0.f), 15.f);
  pair = (__float_as_uint(s) >> 16) | (__float_as_uint(z) & 0xffff0000u);
  // Added to a number, 1.5 * 2^23 rounds it to a whole one, which is then in the sum's low bits: codes are put together
  // from those, and what 1.5 * 2^23 and zero add to all eight of a word is taken off at the end.  None is below 0: the
  // smallest rounds to -zero.
  constexpr float kWhole = 12582912.f;
  const float top = kWhole + 15.f - z;
  float c[kPackVals];
  if constexpr (kShort) {
    // (remainders of numbers of 2^-60 and less would not be exact: both sides times 2^64)
    const bool tiny = s < 8.6736174e-19f;
    const float s1 = tiny ? s * 18446744073709551616.f : s, inv1 = tiny ? inv * 5.4210109e-20f : inv;
    if (tiny) {
#pragma unroll
      for (int i = 0; i < kPackVals; ++i) x[i] *= 18446744073709551616.f;
    }
#pragma unroll
    for (int i = 0; i < kPackVals; ++i) {
      const float q = x[i] * inv1;
      c[i] = fmaf(fmaf(-q, s1, x[i]), inv1, q) + kWhole;
    }
  } else {
    // all rounded again by q4_round where the remainder of one of them is not below half a scale
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < kPackVals; ++i) {
      c[i] = fmaf(x[i], inv, kWhole);
      most = fmaxf(most, fabsf(fmaf(-(c[i] - kWhole), s, x[i])));
    }
    if (most >= 0.5f * s) {
#pragma unroll
      for (int i = 0; i < kPackVals; ++i) c[i] = q4_round(x[i], s, inv) + kWhole;
    }
  }
  const uint32_t off = (__float_as_uint(kWhole) - (uint32_t)(int)z) * 0x11111111u;
  uint32_t w[kPackVals / 8];
#pragma unroll
  for (int k = 0; k < kPackVals / 8; ++k) {
    w[k] = 0u;
#pragma unroll
    for (int i = 7; i >= 0; --i) w[k] = w[k] * 16u + __float_as_uint(fminf(c[8 * k + i], top));
    w[k] -= off;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Thread (token, KV head and group, half of it); blockIdx.y: K or V.  Bound by the instructions to issue (14 a value, 25 us
// for 67 million values) next to HBM (256 bytes read and 72 written a row of 128 bf16 values, also 25 us), so each thread
// fetches the values of its next part before it packs this one.  32,768 tokens of 8 x 128 bf16 values take 35 us (4.9
// TB/s of what is read and written), fp32 61 us (5.0); 16 values a thread took 46 us, 32 without fetching ahead 40.
template <typename T>
__global__ void __launch_bounds__(kQ4Threads) kv_write_q4_kernel(const Q4WriteArgs a, const int64_t total) {
  const T* src = static_cast<const T*>(blockIdx.y ? a.v_new : a.k_new);
  const bool wide = (reinterpret_cast<uintptr_t>(src) & 31u) == 0;
  const int64_t stride = (int64_t)gridDim.x * kQ4Threads;
  // (the threads of a group are all here or all past the end, and what writes nothing computes all the same, so that
  // the lanes of a warp stay together)
  int64_t i = (int64_t)blockIdx.x * kQ4Threads + threadIdx.x;
  uint32_t raw[kPackVals * sizeof(T) / 4];
  int64_t slot = -1;
  int c = 0;
  auto fetch = [&](int64_t at) {  // values and slot of part `at`
    const bool here = at < total;
    if (!here) at = 0;
    int64_t t;
    if (total <= 0xffffffffLL) {
      t = (unsigned)at / (unsigned)a.row_lanes;
    } else {
      t = at / a.row_lanes;
    }
    c = (int)(at - t * a.row_lanes);
    load_raw(src + at * kPackVals, wide, raw);
    slot = __ldg(a.slot_mapping + t);
    if (slot >= a.total_slots && here && c == 0 && blockIdx.y == 0) raise_error(a.err, PA_DEVERR_SLOT);
    if (!here || slot >= a.total_slots) slot = -1;
  };
  const int64_t warp0 = i - (threadIdx.x & 31);
  if (warp0 >= total) return;
  fetch(i);
  for (int64_t w = warp0; w < total; w += stride) {
    float x[kPackVals], lo, hi;
    unpack_raw<T>(raw, x, lo, hi);
    const int64_t dst = slot * a.row_lanes + c;
    const bool writes = slot >= 0, first = c % kPackLanes == 0;
    i += stride;
    if (w + stride < total) fetch(i);
    uint32_t pair;
    const uint4 codes = q4_pack<sizeof(T) == 2>(x, lo, hi, pair);
    if (!writes) continue;
    static_cast<uint4*>(blockIdx.y ? a.v_codes : a.k_codes)[dst] = codes;
    if (first) static_cast<uint32_t*>(blockIdx.y ? a.v_params : a.k_params)[dst / kPackLanes] = pair;
  }
}

template <typename T>
static cudaError_t launch_write(const Q4WriteArgs& a, cudaStream_t s) {
  const int64_t total = a.n_tokens * a.row_lanes, need = (total + kQ4Threads - 1) / kQ4Threads;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)std::min<int64_t>(need, (int64_t)sms * kPackCtas / 2), 2);
  kv_write_q4_kernel<T><<<grid, kQ4Threads, 0, s>>>(a, total);
  return cudaGetLastError();
}

cudaError_t launch_kv_write_q4(const Q4WriteArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  if (a.n_tokens == 0) return cudaSuccess;
  cudaError_t e = cudaErrorInvalidValue;
  if (dt == PA_BF16) e = launch_write<__nv_bfloat16>(a, s);
  if (dt == PA_FP16) e = launch_write<__half>(a, s);
  if (dt == PA_FP32) e = launch_write<float>(a, s);
  ++*launches;
  return e;
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

// Sixteen values of a thread to memory.  The largest codes of a group may stand for a little more than the type's
// largest number (the scale is rounded): they become that.  bf16: 128 + code of two values by two logical instructions,
// minus 128 + zero, times the scale, all in bf16 pairs, which round once, at the end (code - zero is exact).
template <typename T>
__device__ __forceinline__ void unpack16(const uint2& codes, uint32_t pair, T* p, bool aligned32) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  const float s = q4_scale(pair), z = q4_zero(pair);
  if constexpr (sizeof(T) == 2) {
    uint32_t y[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w = k ? codes.y : codes.x;
      uint32_t q[4];  // values i and i + 4
      if constexpr (kBf16) {
        const uint32_t s2 = __byte_perm(pair, pair, 0x1010), top = 0x7f7f7f7fu;
        uint32_t b2;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(b2) : "r"(__byte_perm(pair, pair, 0x3232)), "r"(0x43004300u));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
          asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(b2));
          asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(s2));
          asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(top));
          asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(top | 0x80008000u));
          q[i] = v;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x64006400u;  // 1024 + code
          const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&v));
          const float lo = s * (c.x - (1024.f + z)), hi = s * (c.y - (1024.f + z));
          constexpr float kTop = Largest<T>::kValue;
          const __half2 h = __floats2half2_rn(max_nan(min_nan(lo, kTop), -kTop), max_nan(min_nan(hi, kTop), -kTop));
          q[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      y[4 * k] = __byte_perm(q[0], q[1], 0x5410);
      y[4 * k + 1] = __byte_perm(q[2], q[3], 0x5410);
      y[4 * k + 2] = __byte_perm(q[0], q[1], 0x7632);
      y[4 * k + 3] = __byte_perm(q[2], q[3], 0x7632);
    }
    st_global32(p, y, aligned32);
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = s * (__uint_as_float((((k ? codes.y : codes.x) >> (4 * i)) & 15u) | 0x4b000000u) - (8388608.f + z));
        y[i] = __float_as_uint(max_nan(min_nan(v, FLT_MAX), -FLT_MAX));
      }
      st_global32(p + 8 * k, y, aligned32);
    }
  }
}

constexpr int kQ4Unroll = 2;  // words of K and of V in flight per thread

// CTA (block pair, slice of it).  Bound by HBM: 72 bytes read and 256 written per row of 128 bf16 values.  2,048 blocks of 16
// x 8 x 128 bf16 values take 28 us (6.15 TB/s), fp32 48 us (6.4).
template <typename T>
__global__ void __launch_bounds__(kQ4Threads) kv_unpack_q4_kernel(const Q4UnpackArgs a, const int slices) {
  const int64_t pair = blockIdx.x / slices;
  const int slice = (int)(blockIdx.x - pair * slices);
  const int64_t src = __ldg(a.pairs + 2 * pair), dst = __ldg(a.pairs + 2 * pair + 1);
  if (src < 0 || src >= a.cache_blocks || dst < 0 || dst >= a.num_blocks) {
    if (slice == 0 && threadIdx.x == 0) raise_error(a.err, PA_DEVERR_COPY_PAIR);
    return;
  }
  const uint2* kc = static_cast<const uint2*>(a.k_codes) + src * a.block_words;
  const uint2* vc = static_cast<const uint2*>(a.v_codes) + src * a.block_words;
  const uint32_t* kp = static_cast<const uint32_t*>(a.k_params) + src * (a.block_words / kQ4Lanes);
  const uint32_t* vp = static_cast<const uint32_t*>(a.v_params) + src * (a.block_words / kQ4Lanes);
  T* ko = static_cast<T*>(a.k_pool) + dst * a.block_stride;
  T* vo = static_cast<T*>(a.v_pool) + dst * a.block_stride;
  const bool wide = ((reinterpret_cast<uintptr_t>(ko) | reinterpret_cast<uintptr_t>(vo)) & 31u) == 0;
  for (int w0 = slice * kQ4Threads * kQ4Unroll + threadIdx.x; w0 < a.block_words; w0 += slices * kQ4Threads * kQ4Unroll) {
    uint2 c[kQ4Unroll][2];
    uint32_t p[kQ4Unroll][2];
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
        unpack16<T>(c[u][0], p[u][0], ko + (int64_t)w * kQ4Vals, wide);
        unpack16<T>(c[u][1], p[u][1], vo + (int64_t)w * kQ4Vals, wide);
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
