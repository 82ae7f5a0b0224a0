// Dropout with a counter-based mask that is never stored, with or without a residual added:
//
//   out[r][c] = residual[r][c] + (keep(r, c) ? x[r][c] * 65536 / (65536 - T) : 0)
//
// keep(r, c) is 16 bits of a splitmix64 hash of (seed, step, site, position) compared with T (see
// DropMask), the framework's shared-seed generator, so a backward pass, a replica or a resumed run
// recomputes the same mask from four numbers.  The gradient with respect to x is the same map
// applied to dy, without a residual.
//
// One pass, bound by HBM: 2 or 3 accesses of the element's size per element against about a dozen
// integer and float operations.  One hash covers four elements, so every thread owns whole groups
// of four.  Four access patterns:
//   flat      rows end to end and whole groups per row: positions are flat, 16-byte accesses
//   rows      rows of whole 16-byte units, any stride: a thread per unit
//   segments  rows of any alignment: a warp covers 128 columns with 32-wide accesses, each lane
//             hashes one group, and the lanes pass the hashes round
//   groups    rows of less than 64 elements, where a segment would leave lanes idle
// Measured on 32768 x 2048 bfloat16: flat 40.0 us (6.7 TB/s), with a residual 57.2 us (7.0 TB/s), rows of
// 2056 elements 48 us, of 2051 (segments) 95 us, for its accesses of one element.
#include "train_common.cuh"

namespace demo {

constexpr int kDropThreads = 256;

template <typename T, bool RES>
__device__ __forceinline__ T drop_one(const DropMask& d, T x, T res, uint64_t h, int lane) {
  float v = d.apply(to_f32(x), h, lane);
  if constexpr (RES) v += to_f32(res);
  return from_f32<T>(v);
}

// Elements per 16-byte access, and accesses per thread (all loads are issued before any store).
template <typename T>
constexpr int kPer16 = 16 / static_cast<int>(sizeof(T));
constexpr int kFlatUnroll = 4;

template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_flat(const __grid_constant__ DropoutParams p, long long n) {
  constexpr int N = kPer16<T>;
  using V = Vec<T, N>;
  const DropMask d = drop_mask(p.drop);
  kernel_begin();
  const long long units = n / N;
  const V* x = static_cast<const V*>(p.x);
  const V* res = static_cast<const V*>(p.residual);
  V* out = static_cast<V*>(p.out);
  const long long base = static_cast<long long>(blockIdx.x) * (kDropThreads * kFlatUnroll) + threadIdx.x;
  V a[kFlatUnroll], b[kFlatUnroll];
#pragma unroll
  for (int j = 0; j < kFlatUnroll; ++j) {
    const long long u = base + j * kDropThreads;
    if (u < units) {
      a[j] = x[u];
      if constexpr (RES) b[j] = res[u];
    }
  }
#pragma unroll
  for (int j = 0; j < kFlatUnroll; ++j) {
    const long long u = base + j * kDropThreads;
    if (u < units) {
      V o;
#pragma unroll
      for (int q = 0; q < N / 4; ++q) {
        const uint64_t h = d.group(static_cast<uint64_t>(u) * (N / 4) + q);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o.e[4 * q + e] = drop_one<T, RES>(d, a[j].e[4 * q + e], RES ? b[j].e[4 * q + e] : T(), h, e);
      }
      out[u] = o;
    }
  }
  // The last group of a 16-bit tensor whose size is not a multiple of 8.
  if (N > 4 && n % N != 0 && base == 0) {
    const uint64_t h = d.group(static_cast<uint64_t>(n / 4 - 1));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const long long i = n - 4 + e;
      static_cast<T*>(p.out)[i] = drop_one<T, RES>(
          d, static_cast<const T*>(p.x)[i], RES ? static_cast<const T*>(p.residual)[i] : T(), h, e);
    }
  }
}

// Row of item i where a row has `per` items; 64-bit division only where the numbers need it.
__device__ __forceinline__ long long row_of(long long i, long long per) {
  return i < (1ll << 32) && per < (1ll << 32)
             ? static_cast<long long>(static_cast<uint32_t>(i) / static_cast<uint32_t>(per))
             : i / per;
}

// A thread per 16 bytes of a row.
template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_rows(const __grid_constant__ DropoutParams p, long long per_row) {
  constexpr int N = kPer16<T>;
  using V = Vec<T, N>;
  const DropMask d = drop_mask(p.drop);
  kernel_begin();
  const long long u = static_cast<long long>(blockIdx.x) * kDropThreads + threadIdx.x;
  if (u >= p.rows * per_row) return;
  const long long row = row_of(u, per_row);
  const long long c0 = (u - row * per_row) * N;
  const V a = *reinterpret_cast<const V*>(static_cast<const T*>(p.x) + row * p.ldx + c0);
  V b, o;
  if constexpr (RES) b = *reinterpret_cast<const V*>(static_cast<const T*>(p.residual) + row * p.ldr + c0);
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const uint64_t h = d.group(static_cast<uint64_t>(u) * (N / 4) + q);
#pragma unroll
    for (int e = 0; e < 4; ++e) o.e[4 * q + e] = drop_one<T, RES>(d, a.e[4 * q + e], RES ? b.e[4 * q + e] : T(), h, e);
  }
  *reinterpret_cast<V*>(static_cast<T*>(p.out) + row * p.ldo + c0) = o;
}

// A thread per group, element by element: rows of less than 64 elements.
template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_groups(const __grid_constant__ DropoutParams p, long long G) {
  const DropMask d = drop_mask(p.drop);
  kernel_begin();
  const long long g = static_cast<long long>(blockIdx.x) * kDropThreads + threadIdx.x;
  if (g >= p.rows * G) return;
  const long long row = row_of(g, G);
  const long long c0 = (g - row * G) * 4;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx + c0;
  const T* res = RES ? static_cast<const T*>(p.residual) + row * p.ldr + c0 : nullptr;
  T* out = static_cast<T*>(p.out) + row * p.ldo + c0;
  const uint64_t h = d.group(static_cast<uint64_t>(g));
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c0 + e < p.cols) out[e] = drop_one<T, RES>(d, x[e], RES ? res[e] : T(), h, e);
}

template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads)
    dropout_segments(const __grid_constant__ DropoutParams p, long long G, long long per_row) {
  const DropMask d = drop_mask(p.drop);
  kernel_begin();
  const int lane = threadIdx.x & 31;
  const long long s = static_cast<long long>(blockIdx.x) * (kDropThreads / 32) + (threadIdx.x >> 5);
  if (s >= p.rows * per_row) return;  // whole warps
  const long long row = row_of(s, per_row);
  const long long c0 = (s - row * per_row) * 128;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx + c0;
  const T* res = RES ? static_cast<const T*>(p.residual) + row * p.ldr + c0 : nullptr;
  T* out = static_cast<T*>(p.out) + row * p.ldo + c0;
  const int live = p.cols - c0 < 128 ? static_cast<int>(p.cols - c0) : 128;
  T a[4], b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (32 * j + lane < live) {
      a[j] = x[32 * j + lane];
      if constexpr (RES) b[j] = res[32 * j + lane];
    }
  }
  const uint64_t own = d.group(static_cast<uint64_t>(row * G + c0 / 4 + lane));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t h = __shfl_sync(0xffffffffu, own, 8 * j + (lane >> 2));
    if (32 * j + lane < live)
      out[32 * j + lane] = drop_one<T, RES>(d, a[j], RES ? b[j] : T(), h, lane & 3);
  }
}

template <typename T, bool RES>
static cudaError_t launch_dropout_t(const DropoutParams& p, cudaStream_t st) {
  const auto at = [](const void* q, size_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; };
  const auto all_at = [&](size_t a) { return at(p.x, a) && at(p.out, a) && (!RES || at(p.residual, a)); };
  const long long G = (p.cols + 3) / 4;
  const bool flat = (p.rows == 1 || (p.ldx == p.cols && p.ldo == p.cols && (!RES || p.ldr == p.cols))) &&
                    p.cols % 4 == 0 && all_at(16);
  constexpr int N = kPer16<T>;
  const bool units = all_at(16) && p.cols % N == 0 && p.ldx % N == 0 && p.ldo % N == 0 && (!RES || p.ldr % N == 0);
  const auto blocks = [](long long items, long long per) { return static_cast<unsigned>((items + per - 1) / per); };
  if (flat) {
    const long long n = p.rows * p.cols;
    return launch_overlapped(dropout_flat<T, RES>, blocks(n / N + 1, kDropThreads * kFlatUnroll), kDropThreads, 0, st, p,
                             n);  // at least one block, for the last group
  }
  if (units)
    return launch_overlapped(dropout_rows<T, RES>, blocks(p.rows * (p.cols / N), kDropThreads), kDropThreads, 0, st, p,
                             p.cols / N);
  // A warp per segment would leave most of its lanes idle on short rows.
  if (p.cols < 64)
    return launch_overlapped(dropout_groups<T, RES>, blocks(p.rows * G, kDropThreads), kDropThreads, 0, st, p, G);
  const long long per_row = (p.cols + 127) / 128;
  return launch_overlapped(dropout_segments<T, RES>, blocks(p.rows * per_row, kDropThreads / 32), kDropThreads, 0, st, p,
                           G, per_row);
}

cudaError_t launch_dropout(const DropoutParams& p, int dtype, cudaStream_t st) {
  const bool res = p.residual != nullptr;
  if (dtype == kF32) return res ? launch_dropout_t<float, true>(p, st) : launch_dropout_t<float, false>(p, st);
  if (dtype == kBF16)
    return res ? launch_dropout_t<__nv_bfloat16, true>(p, st) : launch_dropout_t<__nv_bfloat16, false>(p, st);
  return res ? launch_dropout_t<__half, true>(p, st) : launch_dropout_t<__half, false>(p, st);
}

}  // namespace demo
