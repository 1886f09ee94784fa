// q4_experts_device.h -- what the matrix kernels of packed experts share: the
// binary16 forms of codes and activations, and the steps around MFMA.
//
// A packed word holds 8 codes of one row, which become operands in the order of
// nibbles 0, 4, 1, 5, 2, 6, 3, 7 (unpack_word: nine operations, exact);
// activations are laid out in it.  The nibbles n = c + 8 masked out of a word
// are subnormal operands after five operations, and a product's start value
// could take the 8 off again; but MFMA aligns products by their operands'
// exponents, so a subnormal's leading zeros cost low bits of the sum (logits
// to 1e-5 of their size where exact codes give 2e-7), and the time is the same.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_device.h"
#include "q4_serve_device.h"

namespace q4 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Nibble at position i of an operand.
__device__ __forceinline__ constexpr int operand_nibble(int i) { return (i >> 1) + 4 * (i & 1); }

// and the position of a nibble
__device__ __forceinline__ constexpr int operand_place(int nibble) {
  return nibble < 4 ? 2 * nibble : 2 * nibble - 7;
}

__device__ __forceinline__ h8 codes_of(uint32_t w, const Magic& mg) {
  h2 c[4];
  unpack_word(w, mg, c);
  return h8{c[0][0], c[0][1], c[1][0], c[1][1], c[2][0], c[2][1], c[3][0], c[3][1]};
}

// Exponent that puts a row's largest magnitude (its bits; finite) into
// [2^14, 2^15); 0 for a row of zeros.
__device__ __forceinline__ int row_exponent(uint32_t max_bits) {
  if (max_bits == 0) return 0;
  // frexp: max = f * 2^k, f in [0.5, 1)
  return 15 - __builtin_amdgcn_frexp_expf(bits_f32(max_bits));
}

// k with 2^(k - 1) <= the magnitude < 2^k; 0 for 0.
__device__ __forceinline__ int top_exponent(uint32_t bits) {
  return bits ? __builtin_amdgcn_frexp_expf(bits_f32(bits)) : 0;
}

__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = abs_bits(x);
  return b < 0x7f800000u ? b : 0u;
}

// The two binary16 numbers of a scaled element: x = hi + lo to 22 bits (or hi
// alone to 11).  Of an infinity lo is NaN.
__device__ __forceinline__ _Float16 part_hi(float x) { return (_Float16)x; }
__device__ __forceinline__ _Float16 part_lo(float x, _Float16 hi) {
  return (_Float16)__builtin_fmaf(-(float)hi, 1.0f, x);
}

// A product about to be split, rounded to fp32 here: the compiler may otherwise
// round it to binary16 at once for one use and twice for another, and the
// parts no longer belong together.
__device__ __forceinline__ float settled(float x) {
  asm("" : "+v"(x));
  return x;
}

// The slot ids at [0, n) that an expert index is taken from.
__device__ __forceinline__ bool id_ok(int32_t id, int32_t experts) {
  return (uint32_t)id < (uint32_t)experts;
}

// A barrier for what the waves exchange in LDS; loads stay under way.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// MFMA results read after a loop: the compiler's own waits count only from
// within the block (a 16x16x32 product read right after a loop's last one came
// back unfinished here), so the wait is spelled out.
// The accumulators are operands, so that the wait stays behind their products.
template <typename V>
__device__ __forceinline__ void settle(V (&a)[2][2]) {
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7"
               : "+v"(a[0][0]), "+v"(a[0][1]), "+v"(a[1][0]), "+v"(a[1][1]));
}
template <typename V>
__device__ __forceinline__ void settle(V (&a)[2][1]) {
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" : "+v"(a[0][0]), "+v"(a[1][0]));
}
template <typename V>
__device__ __forceinline__ void settle(V (&a)[1][2]) {
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" : "+v"(a[0][0]), "+v"(a[0][1]));
}

// e^x to an ulp or two for x <= 88: the argument in base 2 keeps what its
// product rounds off.
__device__ __forceinline__ float exp_full(float x) {
  const float t = x * kLog2e;
  // infinities have no remainder
  const float r = t - t == 0.0f ? __builtin_fmaf(x, 1.925963033500899e-8f, __builtin_fmaf(x, kLog2e, -t)) : 0.0f;
  const float e = exp2_fast(t);
  return __builtin_fmaf(e, r * kLn2, e);
}

__device__ __forceinline__ float sigmoid(float z) {
  const float e = exp_full(z < 0.0f ? z : -z);  // <= 1
  return (z < 0.0f ? e : 1.0f) / (1.0f + e);
}

}  // namespace q4
