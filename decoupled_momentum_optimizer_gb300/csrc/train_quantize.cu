// Quantization of a matrix to 8-bit floating point with one power-of-two scale for each block of
// 128, by rows, by columns (the codes of the transpose) or both from one read of the matrix:
//
//   v[r][c]  = x[r][c], then relu, dropout and a gate if asked
//   s        = the smallest power of two >= 2^-126 with max |v| over the block <= s * largest code
//   code     = v / s rounded to nearest even      (division by a power of two is exact)
//
// A block is 128 consecutive elements of a row (row form) or of a column (column form), or a whole
// 128 x 128 tile.  The feed-forward layer's relu and dropout, or their gradient (the gate h > 0 and
// the same dropout mask), run in registers on the way, so the activation between them and the
// quantized product is never stored in 16 or 32 bits.
//
// A CTA owns a 128 x 128 tile and keeps it in registers: warp w holds rows 8 w .. 8 w + 7, lane l
// their columns 4 l .. 4 l + 3, all row loads in flight at once; 64 registers a thread let two tiles of
// sixteen warps share an SM (8 warps of 16 rows with 120 registers: 72 us where this took 62).
// A row's block is one warp's 128 elements (one warp-wide maximum each; lane i then works out row i's
// scale for all), a column's block is 8 registers of a lane and the 16 warps' maxima in shared memory,
// a thread per column.  Infinities and NaN are found by a multiply-add with 0 per element and mended
// only where there are any.  Row codes leave as 128 contiguous bytes per row; column codes are packed 8
// rows at a time from the same registers, and leave through a swizzled 16 KB tile in shared memory as
// 128 contiguous bytes per column.
//
// Measured, both forms: 8192 x 2048 float32 tiles 16 us (6.2 TB/s, HBM's rate); 8192 x 8192 bfloat16 55 us
// (4.8 TB/s; 62 with bounds checked in whole tiles too), with relu and dropout 82 us (68 without the
// hash).  Nothing is saturated there: the integer and compare pipe is 65% busy (17 of 32 instructions an
// element), issue slots 61%, HBM 33%; a tile is loaded, computed and stored in turn, and only the SM's
// other CTA overlaps that.
#include "train_common.cuh"

namespace demo {

constexpr int kQuantWarps = 16, kQuantThreads = 32 * kQuantWarps;
constexpr int kPer = kBlock / kQuantWarps;  // rows of a warp

struct QuantShared {
  float colmax[kQuantWarps][kBlock];  // each warp's column maxima
  float colinv[kBlock];               // 1 / each column's scale
  uint32_t warpmax[kQuantWarps];
  uint2 codes[kBlock * kQuantWarps];  // column codes, 16 units of 8 rows per column, swizzled
};

__device__ __forceinline__ float relu_nan(float v) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load4(const T* p, int live, float (&v)[4]) {
  if (VEC) {
    if (live > 0) {  // whole groups of four only: see launch_quantize
      const Vec<T, 4> q = *reinterpret_cast<const Vec<T, 4>*>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = to_f32(q.e[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = 0.0f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < live ? to_f32(p[e]) : 0.0f;
  }
}

template <typename T, int FMT, bool VEC, bool GATE>
__global__ void __launch_bounds__(kQuantThreads, 2) quantize_kernel(const __grid_constant__ QuantParams p) {
  __shared__ QuantShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned tile_r = blockIdx.x / p.col_blocks, tile_c = blockIdx.x - tile_r * p.col_blocks;
  const long long r0 = static_cast<long long>(tile_r) * kBlock + kPer * warp;
  const long long c0 = static_cast<long long>(tile_c) * kBlock + 4 * lane;
  const int live_rows = p.rows - r0 >= kPer ? kPer : p.rows > r0 ? static_cast<int>(p.rows - r0) : 0;
  const int live_cols = p.cols - c0 >= 4 ? 4 : p.cols > c0 ? static_cast<int>(p.cols - c0) : 0;
  kernel_begin();
  float v[kPer][4];
  const T* x = static_cast<const T*>(p.x) + r0 * p.ldx + c0;
  const T* gate = GATE ? static_cast<const T*>(p.gate) + r0 * p.ldg + c0 : nullptr;
  // a whole tile (for every thread of the CTA) needs no bounds
  const bool whole = VEC && static_cast<long long>(tile_r + 1) * kBlock <= p.rows &&
                     static_cast<long long>(tile_c + 1) * kBlock <= p.cols;
  if (whole) {
    Vec<T, 4> a[kPer], h[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      a[i] = *reinterpret_cast<const Vec<T, 4>*>(x + i * p.ldx);
      if constexpr (GATE) h[i] = *reinterpret_cast<const Vec<T, 4>*>(gate + i * p.ldg);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = !GATE || to_f32(h[i].e[e]) > 0.0f ? to_f32(a[i].e[e]) : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      load4<T, VEC>(x + i * p.ldx, i < live_rows ? live_cols : 0, v[i]);
      if constexpr (GATE) {
        float h[4];
        load4<T, VEC>(gate + i * p.ldg, i < live_rows ? live_cols : 0, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = h[e] > 0.0f ? v[i][e] : 0.0f;
      }
    }
  }
  if (p.relu) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = relu_nan(v[i][e]);
  }
  if (p.drop.threshold != 0) {
    const DropMask d = drop_mask(p.drop);
    const unsigned long long G = static_cast<unsigned long long>((p.cols + 3) / 4);
    unsigned long long g = static_cast<unsigned long long>(r0) * G + static_cast<unsigned long long>(c0 / 4);
#pragma unroll
    for (int i = 0; i < kPer; ++i, g += G) {
      bool keep[4];
      d.keep4(d.group(g), keep);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = keep[e] ? v[i][e] * d.scale : 0.0f;
    }
  }
  {
    float odd = 0.0f;  // NaN once an element is infinite or NaN
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) odd = fmaf(v[i][e], 0.0f, odd);
    if (__any_sync(0xffffffffu, odd != odd)) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = finite_or_nan(v[i][e]);
    }
  }

  constexpr int top = fmt_top(FMT);
  // Float bits of non-negative values order as unsigned integers.  (fmaxf passes over a NaN.)
  uint32_t rowbits[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    rowbits[i] = __float_as_uint(
        fmaxf(fmaxf(fmaxf(fabsf(v[i][0]), fabsf(v[i][1])), fmaxf(fabsf(v[i][2]), fabsf(v[i][3]))), 0.0f));
  int tile_e = 0;
  if (p.tiles) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = umax32(m, rowbits[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) sh.warpmax[warp] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < kQuantWarps; ++w) m = umax32(m, sh.warpmax[w]);
    tile_e = scale_exponent(m, top);
  }
  if (p.codes_rows != nullptr) {
    const long long kp = static_cast<long long>(p.col_blocks) * kBlock;
    uint8_t* dst = static_cast<uint8_t*>(p.codes_rows) + r0 * kp + c0;
    int mine = tile_e;  // lane i: the exponent of row i
    if (!p.tiles) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t r = __reduce_max_sync(0xffffffffu, rowbits[i]);
        if (lane == i) m = r;
      }
      mine = scale_exponent(m, top);
    }
    const float inverse = pow2f(-mine);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float inv = __shfl_sync(0xffffffffu, inverse, i);
      if (i < live_rows) *reinterpret_cast<uint32_t*>(dst) = codes4<FMT>(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv);
      dst += kp;
    }
    // rows past the matrix up to the scales' stride hold 1
    const long long lds = (p.rows + 3) / 4 * 4;
    if (lane < kPer && r0 + lane < lds)
      p.scales_rows[static_cast<long long>(tile_c) * lds + r0 + lane] = r0 + lane < p.rows ? pow2f(mine) : 1.0f;
  }
  if (p.codes_cols != nullptr) {
    float4 m = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!p.tiles) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        m.x = fmaxf(m.x, fabsf(v[i][0]));
        m.y = fmaxf(m.y, fabsf(v[i][1]));
        m.z = fmaxf(m.z, fabsf(v[i][2]));
        m.w = fmaxf(m.w, fabsf(v[i][3]));
      }
    }
    *reinterpret_cast<float4*>(&sh.colmax[warp][4 * lane]) = m;
    __syncthreads();
    if (threadIdx.x < kBlock) {  // a thread per column
      float c = 0.0f;
#pragma unroll
      for (int w = 0; w < kQuantWarps; ++w) c = fmaxf(c, sh.colmax[w][threadIdx.x]);
      const int e = p.tiles ? tile_e : scale_exponent(__float_as_uint(c), top);
      sh.colinv[threadIdx.x] = pow2f(-e);
      const long long lds = (p.cols + 3) / 4 * 4, col = static_cast<long long>(tile_c) * kBlock + threadIdx.x;
      if (col < lds)  // columns past the matrix up to the scales' stride hold 1
        p.scales_cols[static_cast<long long>(tile_r) * lds + col] = col < p.cols ? pow2f(e) : 1.0f;
    }
    __syncthreads();
    const float4 q4 = *reinterpret_cast<const float4*>(&sh.colinv[4 * lane]);
    const float inv[4] = {q4.x, q4.y, q4.z, q4.w};
    // Column 4 l + e, unit `warp` (its rows 8 w ..): stored at unit w ^ (l & 15), so that the sixteen
    // lanes of an 8-byte store phase reach different banks.
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sh.codes[(4 * lane + e) * kQuantWarps + (warp ^ (lane & 15))] =
          make_uint2(codes4<FMT>(v[0][e] * inv[e], v[1][e] * inv[e], v[2][e] * inv[e], v[3][e] * inv[e]),
                     codes4<FMT>(v[4][e] * inv[e], v[5][e] * inv[e], v[6][e] * inv[e], v[7][e] * inv[e]));
    __syncthreads();
    const long long rp = static_cast<long long>(p.row_blocks) * kBlock;
    const long long col0 = static_cast<long long>(tile_c) * kBlock;
    const int unit = threadIdx.x & 7;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = (threadIdx.x >> 3) + 64 * j, k = (c >> 2) & 15;
      if (col0 + c < p.cols) {
        const uint2 lo = sh.codes[c * kQuantWarps + ((2 * unit) ^ k)], hi = sh.codes[c * kQuantWarps + ((2 * unit + 1) ^ k)];
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.codes_cols) + (col0 + c) * rp +
                                  static_cast<long long>(tile_r) * kBlock + 16 * unit) =
            make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
}

template <typename T, int FMT>
static cudaError_t launch_quantize_t(const QuantParams& p, cudaStream_t st) {
  const unsigned grid = p.row_blocks * p.col_blocks;
  const auto at = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & (4 * sizeof(T) - 1)) == 0; };
  // Accesses of four elements where every row's groups of four are aligned and whole.
  const bool vec = p.cols % 4 == 0 && p.ldx % 4 == 0 && at(p.x) &&
                   (p.gate == nullptr || (p.ldg % 4 == 0 && at(p.gate)));
  auto* kernel = p.gate != nullptr ? (vec ? quantize_kernel<T, FMT, true, true> : quantize_kernel<T, FMT, false, true>)
                                   : (vec ? quantize_kernel<T, FMT, true, false> : quantize_kernel<T, FMT, false, false>);
  return launch_overlapped(kernel, grid, kQuantThreads, 0, st, p);
}

cudaError_t launch_quantize(const QuantParams& p, int dtype, int fmt, cudaStream_t st) {
  if (fmt == kE4M3) {
    if (dtype == kF32) return launch_quantize_t<float, kE4M3>(p, st);
    if (dtype == kBF16) return launch_quantize_t<__nv_bfloat16, kE4M3>(p, st);
    return launch_quantize_t<__half, kE4M3>(p, st);
  }
  if (dtype == kF32) return launch_quantize_t<float, kE5M2>(p, st);
  if (dtype == kBF16) return launch_quantize_t<__nv_bfloat16, kE5M2>(p, st);
  return launch_quantize_t<__half, kE5M2>(p, st);
}

}  // namespace demo
