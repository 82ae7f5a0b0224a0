// x w^T for a few rows of x (tokens being generated) and w in 8-bit floating point, block-scaled: one
// kernel that quantizes x, multiplies and scales, bound by reading w once.
//
// A warp multiplies 16 rows of w at a time (the instruction's 16 x 32 operand) by up to 8 T tokens,
// one block of 128 along k after another; the warps of a CTA share its rows and take the blocks in
// turn, so that a short k still fills the machine with reads, and join their sums in order through
// shared memory.  w goes straight from global memory to the registers the instruction reads: its k
// order is free as long as both operands agree, so lane (g, c) takes 16 consecutive codes of row g at
// 16 c and at 64 + 16 c, whole 16-byte loads, a block ahead of the arithmetic.  Lane (g, c) likewise
// quantizes 32 elements of token g, the four lanes of a token sharing the block's maximum.  Every CTA
// repeats that (at most 32 tokens), which is cheaper than a kernel of its own before this one.
//
// The block's 128 products accumulate in the instruction's float32, blocks in IEEE float32.
#include "train_common.cuh"

namespace demo {

namespace {

constexpr int kLinearMaxWarps = 16;

// D += A B, 16 x 8, K = 32 codes, float32 accumulators.
template <int WFMT>
__device__ __forceinline__ void mma_f8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if constexpr (WFMT == kE4M3)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e5m2.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 consecutive elements of a token as float32, zero from `live` on.
template <typename T, bool VEC>
__device__ __forceinline__ void load16(const T* p, long long live, float* v) {
  constexpr int N = 16 / static_cast<int>(sizeof(T));
  if (VEC && live >= 16) {
#pragma unroll
    for (int i = 0; i < 16 / N; ++i) {
      const Vec<T, N> q = reinterpret_cast<const Vec<T, N>*>(p)[i];
#pragma unroll
      for (int e = 0; e < N; ++e) v[N * i + e] = to_f32(q.e[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = e < live ? to_f32(p[e]) : 0.0f;
  }
}

template <typename T, bool VEC, int WFMT, int TILES>
__global__ void __launch_bounds__(32 * kLinearMaxWarps) linear_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ float part[];  // [warps][8 TILES tokens][16 rows]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const long long n0 = static_cast<long long>(blockIdx.x) * 16;
  // rows past the end repeat the last one (their results are not written)
  const long long r0 = n0 + g < p.n ? n0 + g : p.n - 1, r1 = n0 + g + 8 < p.n ? n0 + g + 8 : p.n - 1;
  const long long kp = static_cast<long long>(p.kb) * kBlock, ldw = (p.n + 3) / 4 * 4;
  const uint8_t* w0 = static_cast<const uint8_t*>(p.w) + r0 * kp + 16 * c;
  const uint8_t* w1 = static_cast<const uint8_t*>(p.w) + r1 * kp + 16 * c;
  kernel_begin();

  float sum[TILES][4];
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[t][e] = 0.0f;
  uint4 a[2][2];  // [row][half] of the block to come
  float s0 = 0.0f, s1 = 0.0f;
  const auto fetch = [&](int kb) {
    const long long at = static_cast<long long>(kb) * kBlock;
    a[0][0] = *reinterpret_cast<const uint4*>(w0 + at);
    a[0][1] = *reinterpret_cast<const uint4*>(w0 + at + 64);
    a[1][0] = *reinterpret_cast<const uint4*>(w1 + at);
    a[1][1] = *reinterpret_cast<const uint4*>(w1 + at + 64);
    s0 = p.w_scales[kb * ldw + r0];
    s1 = p.w_scales[kb * ldw + r1];
  };
  if (warp < p.kb) fetch(warp);
  for (int kb = warp; kb < p.kb; kb += warps) {
    uint32_t b[TILES][2][4];
    float sx[TILES];
    const long long k0 = static_cast<long long>(kb) * kBlock + 16 * c;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int m = 8 * t + g;
      float v[32];
      const T* x = static_cast<const T*>(p.x) + m * p.ldx + k0;
      load16<T, VEC>(x, m < p.m ? p.k - k0 : 0, v);
      load16<T, VEC>(x + 64, m < p.m ? p.k - k0 - 64 : 0, v + 16);
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        v[e] = finite_or_nan(v[e]);
        top = fmaxf(top, fabsf(v[e]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = scale_exponent(__float_as_uint(top), fmt_top(kE4M3));
      const float inv = pow2f(-e);
      sx[t] = pow2f(e);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        b[t][q >> 2][q & 3] = codes4<kE4M3>(v[4 * q] * inv, v[4 * q + 1] * inv, v[4 * q + 2] * inv, v[4 * q + 3] * inv);
    }
    const uint4 x00 = a[0][0], x01 = a[0][1], x10 = a[1][0], x11 = a[1][1];
    const float t0 = s0, t1 = s1;
    if (kb + warps < p.kb) fetch(kb + warps);
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      mma_f8<WFMT>(d, x00.x, x10.x, x00.y, x10.y, b[t][0][0], b[t][0][1]);
      mma_f8<WFMT>(d, x00.z, x10.z, x00.w, x10.w, b[t][0][2], b[t][0][3]);
      mma_f8<WFMT>(d, x01.x, x11.x, x01.y, x11.y, b[t][1][0], b[t][1][1]);
      mma_f8<WFMT>(d, x01.z, x11.z, x01.w, x11.w, b[t][1][2], b[t][1][3]);
      // this lane's results are rows g, g + 8 and tokens 2 c, 2 c + 1, whose scales lanes 8 c, 8 c + 4 hold
      const float u0 = __shfl_sync(0xffffffffu, sx[t], 8 * c), u1 = __shfl_sync(0xffffffffu, sx[t], 8 * c + 4);
      sum[t][0] = fmaf(d[0] * t0, u0, sum[t][0]);
      sum[t][1] = fmaf(d[1] * t0, u1, sum[t][1]);
      sum[t][2] = fmaf(d[2] * t1, u0, sum[t][2]);
      sum[t][3] = fmaf(d[3] * t1, u1, sum[t][3]);
    }
  }
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    float* q = part + (warp * 8 * TILES + 8 * t + 2 * c) * 16 + g;
    q[0] = sum[t][0];
    q[16] = sum[t][1];
    q[8] = sum[t][2];
    q[24] = sum[t][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * TILES * 16; i += blockDim.x) {
    const int m = i >> 4;
    const long long n = n0 + (i & 15);
    if (m >= p.m || n >= p.n) continue;
    float v = part[i];
    for (int w = 1; w < warps; ++w) v += part[w * 8 * TILES * 16 + i];
    const long long at = m * p.ldo + n;
    if (p.out_dtype == kF32)
      static_cast<float*>(p.out)[at] = v;
    else if (p.out_dtype == kBF16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
    else
      static_cast<__half*>(p.out)[at] = __float2half_rn(v);
  }
}

struct LinearShape {
  unsigned grid, threads;
  size_t smem;
  int tiles;
  cudaStream_t st;
};

template <typename T, bool VEC, int WFMT>
cudaError_t launch_tiles(const LinearParams& p, const LinearShape& s) {
  auto* kernel = s.tiles == 1   ? linear_kernel<T, VEC, WFMT, 1>
                 : s.tiles == 2 ? linear_kernel<T, VEC, WFMT, 2>
                                : linear_kernel<T, VEC, WFMT, 4>;
  return launch_overlapped(kernel, s.grid, s.threads, s.smem, s.st, p);
}

template <typename T>
cudaError_t launch_linear_t(const LinearParams& p, int w_fmt, const LinearShape& s) {
  const bool vec = (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 && (p.m == 1 || p.ldx * sizeof(T) % 16 == 0);
  if (w_fmt == kE4M3) return vec ? launch_tiles<T, true, kE4M3>(p, s) : launch_tiles<T, false, kE4M3>(p, s);
  return vec ? launch_tiles<T, true, kE5M2>(p, s) : launch_tiles<T, false, kE5M2>(p, s);
}

}  // namespace

cudaError_t launch_linear(const LinearParams& p, int dtype, int w_fmt, int sms, cudaStream_t st) {
  const long long ctas = (p.n + 15) / 16;
  // Eight warps a CTA fill the machine's reads when there are CTAs for every SM, sixteen when not.
  int warps = ctas > sms ? 8 : kLinearMaxWarps;
  if (warps > p.kb) warps = p.kb > 0 ? p.kb : 1;
  LinearShape s;
  s.tiles = p.m <= 8 ? 1 : p.m <= 16 ? 2 : 4;
  s.grid = static_cast<unsigned>(ctas);
  s.threads = 32 * warps;
  s.smem = static_cast<size_t>(warps) * 8 * s.tiles * 16 * sizeof(float);
  s.st = st;
  if (dtype == kF32) return launch_linear_t<float>(p, w_fmt, s);
  if (dtype == kBF16) return launch_linear_t<__nv_bfloat16>(p, w_fmt, s);
  return launch_linear_t<__half>(p, w_fmt, s);
}

}  // namespace demo
