// What the training operators (dropout, block-scaled 8-bit quantization, products) share:
// element types, the dropout mask, and the scale and codes of a block of 128.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "demo_common.cuh"
#include "train_launch.h"

namespace demo {

// ----------------------------------------------------------------------------
// Elements in 16 or 32 bits, computed with in float32
// ----------------------------------------------------------------------------

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// N consecutive elements as one access of N * sizeof(T) bytes (at most 16, aligned to its size).
template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
  T e[N];
};

// Launch with programmatic stream serialisation: the kernel's blocks may be placed while the stream's
// previous kernel ends, and wait for it (kernel_begin) before they touch memory.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t st,
                              const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ void kernel_begin() {
  griddep_launch_dependents();
  griddep_wait();
}

// ----------------------------------------------------------------------------
// The dropout mask: 16 bits per element of a counter-based hash
// ----------------------------------------------------------------------------

// h(g) = sm(key ^ g) gives the four elements of group g = row * ceil(cols / 4) + col / 4 sixteen
// bits each; an element is kept where its bits are at least `threshold` = round(65536 p).  Sixteen
// bits keep the hash at about six integer operations per element (32 bits each would double it and
// make the bfloat16 kernel issue-bound); p is taken to the nearest 1/65536, and the kept values'
// factor is that of the p actually applied, so the expected value is exact.
struct DropMask {
  uint64_t key;
  uint32_t threshold;  // 0 keeps everything, 65536 nothing
  float scale;         // 65536 / (65536 - threshold)

  __device__ __forceinline__ uint64_t group(uint64_t g) const { return splitmix64(key ^ g); }
  __device__ __forceinline__ bool keep(uint64_t h, int lane) const {
    return ((static_cast<uint32_t>(h >> (16 * lane))) & 0xffffu) >= threshold;
  }
  // All four elements of a group, with one comparison of 32 bits each: a half's high 16 bits compare as
  // they are, its low ones after a shift (a threshold of 65536 has no such form).
  __device__ __forceinline__ void keep4(uint64_t h, bool (&keep)[4]) const {
    const uint32_t lo = static_cast<uint32_t>(h), hi = static_cast<uint32_t>(h >> 32), t = threshold << 16;
    const bool any = threshold < 65536u;
    keep[0] = any && (lo << 16) >= t;
    keep[1] = any && lo >= t;
    keep[2] = any && (hi << 16) >= t;
    keep[3] = any && hi >= t;
  }
  // A dropped element is 0 whatever it held, an infinity or a NaN included.
  __device__ __forceinline__ float apply(float v, uint64_t h, int lane) const {
    return keep(h, lane) ? v * scale : 0.0f;
  }
};

inline __device__ DropMask drop_mask(const DropParams& d) { return DropMask{d.key, d.threshold, d.scale}; }

// ----------------------------------------------------------------------------
// Block scales and codes
// ----------------------------------------------------------------------------

// Exponent of the block scale: the smallest e >= -126 with amax <= 2^e * (largest finite code),
// 0 for a block of zeros.  `bits` are the float32 bits of amax (finite, not negative).  Both
// formats' largest code is 1.75 * 2^top, so e = exponent(amax) - top, one more when amax's
// significand is above 1.75.
__device__ __forceinline__ int scale_exponent(uint32_t bits, int top) {
  if (bits == 0) return 0;
  // 0x1fffff carries into the exponent where the significand's bits are above 0x600000 (1.75)
  const int e = static_cast<int>((bits + 0x1fffffu) >> 23) - 127 - top;
  return e < -126 ? -126 : e;
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// A scale as the tensor core takes it, an exponent byte (UE8M0).  A quantized matrix's scales are 0 or
// powers of two from 2^-126 to 2^127; any other would lose its significand or sign without a word, so it
// becomes the byte of NaN, in every product.  (Turned left by nine bits, a power of two is its exponent,
// and whatever has a sign or a significand is above 255.)  0 is taken for 2^-127.
constexpr uint32_t kScaleNaN = 255;
__device__ __forceinline__ uint32_t scale_byte(float s) {
  const uint32_t bits = __float_as_uint(s), r = __funnelshift_l(bits, bits, 9);
  return r < kScaleNaN ? r : kScaleNaN;
}

// A non-finite element becomes a NaN code (neither format's codes saturate silently); it does not
// take part in its block's scale (fmaxf passes over a NaN).
__device__ __forceinline__ float finite_or_nan(float v) {
  return fabsf(v) <= 3.402823466e38f ? v : __uint_as_float(0x7fc00000u);
}

// Two codes, `lo` in the low byte; nearest even.  Block scaling keeps |v| at or below the largest
// code, so saturation never applies.
template <int FMT>
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, FMT == kE4M3 ? __NV_E4M3 : __NV_E5M2);
}

template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return codes2<FMT>(a, b) | (codes2<FMT>(c, d) << 16);
}

}  // namespace demo
