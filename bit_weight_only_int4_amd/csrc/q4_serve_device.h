// q4_serve_device.h -- device helpers shared by the cache, attention and
// log-probability kernels: element types, exponentials, cross-lane steps.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_kv.h"
#include "q4serve.h"

namespace q4 {

typedef __bf16 bf16;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
  return (float)x;
}
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  return (T)x;  // one rounding to nearest even
}

// 2^x on the transcendental unit (about 1 ulp; 2^-inf = 0, NaN stays NaN)
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_fast(float x) { return __builtin_amdgcn_logf(x); }

__device__ __forceinline__ uint32_t abs_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ float bits_f32(uint32_t b) { return __builtin_bit_cast(float, b); }
__device__ __forceinline__ uint32_t f32_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

// What a page's scale makes of its codes: a negative one is no scale, and NaN
// like one that is (the kernels' maxima and digits take values of one sign).
__device__ __forceinline__ float scale_or_nan(float s) {
  return s >= 0.0f ? s : bits_f32(0x7fc00000u);
}

// Magnitudes are compared as their bit patterns, which order like the
// numbers and put NaN above infinity, so that neither is lost in a maximum.
__device__ __forceinline__ uint32_t wave_umax(uint32_t x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x = umax(x, (uint32_t)__shfl_xor((int)x, m, 64));
  return x;
}

}  // namespace q4
