// Float32 arithmetic on two values at a time, and 16-bit elements two to a word.
#pragma once

#include "train_common.cuh"

namespace demo {

template <typename T>
constexpr bool is_bf16 = false;
template <>
constexpr bool is_bf16<__nv_bfloat16> = true;

// ----------------------------------------------------------------------------
// Two float32 operations in one instruction
// ----------------------------------------------------------------------------

// Each half rounds as the scalar operation does.  Kernels that sum and scale 16-bit elements are bound by the
// instructions an element takes, not by HBM, without it.
typedef float2 F2;

__device__ __forceinline__ F2 f2(float lo, float hi) { return make_float2(lo, hi); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return __ffma2_rn(a, b, c); }
// The largest magnitude of m (not negative), a and b; NaN if one is.
__device__ __forceinline__ float max_abs_nan(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}

// The same passing over a NaN.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}

// ----------------------------------------------------------------------------
// 16-bit elements
// ----------------------------------------------------------------------------

// Two 16-bit elements in a word, the first in its low half.
template <typename T>
__device__ __forceinline__ F2 widen(uint32_t w) {
  if constexpr (is_bf16<T>) return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t narrow(F2 v) {
  if constexpr (is_bf16<T>) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&r);
}
}  // namespace demo
