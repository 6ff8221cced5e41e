// The 4-bit cache's format, shared by the kernels that pack, unpack and read it.
//
// A row (token, KV head) of head_dim values is head_dim / 2 bytes of codes, the even dimension in a byte's low
// half, and per group of 64 values a pair (scale, zero) of bf16: value = scale * (code - zero), code and zero
// whole numbers in 0 .. 15.  Codes and pairs lie in pools of their own, [num_blocks][block_size][n_kv_heads][..].
#pragma once

#include "pa_common.cuh"

namespace pa {

constexpr int kQ4Group = 64;  // values that share a scale and a zero

// Minimum and maximum that keep a NaN (fminf and fmaxf drop it).
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale and zero of a (scale, zero) pair.
__device__ __forceinline__ float q4_scale(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float q4_zero(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }

}  // namespace pa
