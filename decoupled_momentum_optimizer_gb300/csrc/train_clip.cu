// The norm over all gradients of a model, and the gradients scaled to a largest norm:
//
//   norm = sqrt(sum over the tensors and their elements of g^2)
//   out  = g * f,  f = max_norm / norm where max_norm < norm < infinity, else 1
//
// Bound by HBM: one read for the norm, another read and a write where something is scaled.  The tensors'
// addresses and sizes are kernel parameters, so a list of them is one launch and no copy.  A tensor is
// cut into chunks of 32 KB of whole 16-byte accesses (its first and last access may be partial), and CTAs take
// every gridDim.x-th chunk of the list: which elements a thread sums, and in which order the sums are joined,
// follow from the sizes and the grid alone.
//
// A thread squares and sums the 32 or 64 elements of a chunk in float32 (sums of four or eight, then a tree) and
// adds that to a float64 sum: float64 for every element would take 1.9 ms for 2^30 elements (two lanes an SM),
// three times what HBM takes.  A chunk sum that overflows, or that is so small that squares may have been lost
// below float32's range, is done again in float64 from the registers the elements are in, so the norm is right
// over all of float32's range.
//
// 193 float32 tensors of 157 million elements: the norm 94 us (6.7 TB/s), clipped into others 300 us; in bfloat16 157
// us.  (The second read starts at the first one's end, for what L2 still holds: in order 302 and 165 us.)
// 2^27 bfloat16 elements that need no clipping 46.5 us, of 39.4 for their bytes.  Lists of up to 64 chunks are one
// cluster's, in one launch: shorter calls where nothing is scaled, longer ones where something is and in graphs.
#include <cooperative_groups.h>

#include <type_traits>

#include "train_pairs.cuh"

namespace demo {

namespace cg = cooperative_groups;

constexpr int kClipThreads = 256, kClipUnroll = 8, kClipChunk = kClipThreads * kClipUnroll;  // in 16-byte accesses
// CTAs an SM: what 64 or 84 registers a thread leave room for (16-bit elements spill with 64).  2^27 elements,
// the norm: float32 80 us (6.7 TB/s, three CTAs the same), bfloat16 44 us (6.1 TB/s; 71 with four).
template <typename T>
constexpr int kClipCtas = sizeof(T) == 4 ? 4 : 3;

template <typename T>
constexpr int kClipN = 16 / static_cast<int>(sizeof(T));

// A chunk of a tensor: accesses [first, ...) counted from the 16-byte boundary at or below its start, `off`
// elements before it.
template <typename T>
struct Chunk {
  const T* base;  // element 0 of access 0 (may lie before the tensor)
  long long off, end, first;  // the tensor is elements off .. end - 1 from base
  int tensor;

  // `lane` counts the kClipThreads threads of the chunk.
  template <int CAP>
  __device__ __forceinline__ Chunk(const ClipParams<CAP>& p, unsigned chunk, unsigned lane) {
    int lo = 0, hi = p.count - 1;  // the last tensor that starts at or before the chunk
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.start[mid] <= chunk)
        lo = mid;
      else
        hi = mid - 1;
    }
    tensor = lo;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p.g[lo]);
    off = static_cast<long long>((a & 15) / sizeof(T));
    base = reinterpret_cast<const T*>(a & ~static_cast<uintptr_t>(15));
    end = off + p.n[lo];
    first = static_cast<long long>(chunk - p.start[lo]) * kClipChunk + lane;
  }
  __device__ __forceinline__ long long access(int u) const { return first + u * kClipThreads; }
  __device__ __forceinline__ bool whole(long long v) const {
    return v * kClipN<T> >= off && (v + 1) * kClipN<T> <= end;
  }
  // Elements of a partial access, 0 around the tensor.
  __device__ __forceinline__ uint4 load_part(long long v) const {
    Vec<T, kClipN<T>> q;
#pragma unroll
    for (int e = 0; e < kClipN<T>; ++e) {
      const long long i = v * kClipN<T> + e;
      q.e[e] = i >= off && i < end ? base[i] : from_f32<T>(0.0f);
    }
    return *reinterpret_cast<const uint4*>(&q);
  }
  __device__ __forceinline__ void load(uint4 (&x)[kClipUnroll]) const {
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) {
      const long long v = access(u);
      x[u] = make_uint4(0, 0, 0, 0);
      if (whole(v))
        x[u] = reinterpret_cast<const uint4*>(base)[v];
      else if (v * kClipN<T> < end)
        x[u] = load_part(v);
    }
  }
};

// Elements 2 i and 2 i + 1 of an access.
template <typename T>
__device__ __forceinline__ F2 pair_of(const uint4& x, int i) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (sizeof(T) == 2) return widen<T>(w[i]);
  return f2(__uint_as_float(w[(2 * i) & 3]), __uint_as_float(w[(2 * i + 1) & 3]));
}

// The sum of a CTA's threads' values, for all of them.
template <int THREADS>
__device__ __forceinline__ double cta_sum(double v, double* sh) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = sh[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) t += sh[w];
  return t;
}

// A thread's sum of squares of its elements of a chunk.
template <typename T>
__device__ __forceinline__ double chunk_squares(const Chunk<T>& chunk) {
  uint4 x[kClipUnroll];
  chunk.load(x);
  F2 s[kClipUnroll];
#pragma unroll
  for (int u = 0; u < kClipUnroll; ++u) {
    s[u] = f2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kClipN<T> / 2; ++i) {
      const F2 v = pair_of<T>(x[u], i);
      s[u] = fma2(v, v, s[u]);
    }
  }
#pragma unroll
  for (int d = 1; d < kClipUnroll; d *= 2)
#pragma unroll
    for (int u = 0; u < kClipUnroll; u += 2 * d) s[u] = add2(s[u], s[u + d]);
  const float sum = s[0].x + s[0].y;
  // At 2^-90 the squares lost below 2^-149, 64 of them, are 2^-53 of the sum.
  if (sum >= 0x1p-90f && sum <= 0x1p120f) return static_cast<double>(sum);
  uint32_t any = 0;
#pragma unroll
  for (int u = 0; u < kClipUnroll; ++u) any |= x[u].x | x[u].y | x[u].z | x[u].w;
  double t = 0.0;
  if (any != 0) {
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) {
#pragma unroll
      for (int i = 0; i < kClipN<T> / 2; ++i) {
        const F2 v = pair_of<T>(x[u], i);
        t += static_cast<double>(v.x) * v.x + static_cast<double>(v.y) * v.y;
      }
    }
  }
  return t;
}

template <typename T, int CAP>
__global__ void __launch_bounds__(kClipThreads, kClipCtas<T>) squares_kernel(const __grid_constant__ ClipParams<CAP> p) {
  __shared__ double sh[kClipThreads / 32];
  kernel_begin();
  double total = 0.0;
  for (unsigned c = blockIdx.x; c < p.chunks; c += gridDim.x) total += chunk_squares(Chunk<T>(p, c, threadIdx.x));
  total = cta_sum<kClipThreads>(total, sh);
  if (threadIdx.x == 0) p.parts[blockIdx.x] = total;
}

// The norm from the CTAs' sums, for all threads of a CTA.
__device__ __forceinline__ float norm_of(const double* parts, int count, double* sh) {
  double v = 0.0;
  for (int i = threadIdx.x; i < count; i += kClipThreads) v += parts[i];
  return static_cast<float>(sqrt(cta_sum<kClipThreads>(v, sh)));
}

__global__ void __launch_bounds__(kClipThreads) norm_kernel_of_parts(const double* parts, int count, float* norm) {
  __shared__ double sh[kClipThreads / 32];
  kernel_begin();
  const float n = norm_of(parts, count, sh);
  if (threadIdx.x == 0) *norm = n;
}

// What a norm becomes of: the factor, 1 where nothing is clipped.
__device__ __forceinline__ float clip_factor(double max_norm, float norm) {
  const bool some = static_cast<double>(norm) > max_norm && norm <= 3.402823466e38f;
  return some ? static_cast<float>(max_norm / static_cast<double>(norm)) : 1.0f;
}

// A thread's elements of a chunk times f.  With f = 1 the elements themselves, a NaN's payload included, where O is
// their type.
template <typename T, typename O, int CAP>
__device__ __forceinline__ void scale_chunk(const ClipParams<CAP>& p, const Chunk<T>& chunk, float f) {
  const bool copy = f == 1.0f;
  uint4 x[kClipUnroll];
  chunk.load(x);
  O* out = static_cast<O*>(p.out[chunk.tensor]);
  const bool aligned = ((reinterpret_cast<uintptr_t>(out) - static_cast<uintptr_t>(chunk.off) * sizeof(O)) & 15) == 0;
#pragma unroll
  for (int u = 0; u < kClipUnroll; ++u) {
    const long long v = chunk.access(u), i0 = v * kClipN<T> - chunk.off;
    if (chunk.whole(v) && aligned) {
      if constexpr (std::is_same_v<T, float> || !std::is_same_v<T, O>) {
        float4* to = reinterpret_cast<float4*>(out + i0);
#pragma unroll
        for (int k = 0; k < kClipN<T> / 4; ++k) {
          const F2 a = mul2(pair_of<T>(x[u], 2 * k), f2(f, f)), b = mul2(pair_of<T>(x[u], 2 * k + 1), f2(f, f));
          to[k] = copy && std::is_same_v<T, O> ? *reinterpret_cast<const float4*>(&x[u]) : make_float4(a.x, a.y, b.x, b.y);
        }
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = narrow<T>(mul2(pair_of<T>(x[u], i), f2(f, f)));
        *reinterpret_cast<uint4*>(out + i0) = copy ? x[u] : make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else if (v * kClipN<T> < chunk.end) {
#pragma unroll
      for (int e = 0; e < kClipN<T>; ++e) {
        if (i0 + e >= 0 && i0 + e < chunk.end - chunk.off) {
          const F2 g = pair_of<T>(x[u], e / 2);
          if constexpr (std::is_same_v<T, O>) {
            if (copy) {
              out[i0 + e] = chunk.base[chunk.off + i0 + e];
              continue;
            }
          }
          out[i0 + e] = from_f32<O>((e % 2 ? g.y : g.x) * f);
        }
      }
    }
  }
}

template <typename T, typename O, int CAP>
__global__ void __launch_bounds__(kClipThreads, kClipCtas<T>) scale_kernel(const __grid_constant__ ClipParams<CAP> p) {
  __shared__ double sh[kClipThreads / 32];
  __shared__ float factor;
  kernel_begin();
  const float norm = p.given ? *p.norm : norm_of(p.all_parts, p.part_count, sh);
  if (threadIdx.x == 0) {
    if (!p.given && blockIdx.x == 0 && p.first_launch) *p.norm = norm;
    factor = clip_factor(p.max_norm, norm);
  }
  __syncthreads();
  const float f = factor;
  if (f == 1.0f && p.in_place) return;
  // Backwards: what the norm read last is still in L2.
  for (unsigned i = blockIdx.x; i < p.chunks; i += gridDim.x)
    scale_chunk<T, O>(p, Chunk<T>(p, p.chunks - 1 - i, threadIdx.x), f);
}

// A few chunks in one launch: a cluster's CTAs add up each other's sums in CTA order, and scale what they read.  A call of
// a short list takes the longer of the device's time and its issue, about 3 us a launch; from a graph two launches are
// faster, as they overlap and have a CTA for each chunk (see kSmallChunks for both sides).
constexpr int kSmallThreads = 512, kSmallCtas = 8, kSmallTeams = kSmallCtas * (kSmallThreads / kClipThreads);

template <typename T, typename O>
__global__ void __launch_bounds__(kSmallThreads) small_clip_kernel(const __grid_constant__ ClipParams<kClipFew> p) {
  __shared__ double sh[kSmallThreads / 32];
  __shared__ double mine;
  __shared__ float factor;
  cg::cluster_group cluster = cg::this_cluster();
  const unsigned team = cluster.block_rank() * (kSmallThreads / kClipThreads) + threadIdx.x / kClipThreads;
  const unsigned lane = threadIdx.x % kClipThreads;
  kernel_begin();
  double total = 0.0;
  for (unsigned c = team; c < p.chunks; c += kSmallTeams) total += chunk_squares(Chunk<T>(p, c, lane));
  total = cta_sum<kSmallThreads>(total, sh);
  if (threadIdx.x == 0) mine = total;
  cluster.sync();
  if (threadIdx.x == 0) {
    double v[kSmallCtas];
#pragma unroll
    for (int r = 0; r < kSmallCtas; ++r) v[r] = *cluster.map_shared_rank(&mine, r);
#pragma unroll
    for (int r = 1; r < kSmallCtas; ++r) v[0] += v[r];
    const float norm = static_cast<float>(sqrt(v[0]));
    if (cluster.block_rank() == 0) *p.norm = norm;
    factor = p.only_norm ? 1.0f : clip_factor(p.max_norm, norm);
  }
  cluster.sync();  // the factor is there, and nobody reads this CTA's sum any more
  const float f = factor;
  if (p.only_norm || (f == 1.0f && p.in_place)) return;
  for (unsigned c = team; c < p.chunks; c += kSmallTeams) scale_chunk<T, O>(p, Chunk<T>(p, c, lane), f);
}

namespace {

unsigned clip_grid(unsigned chunks, int dtype, int sms) {
  const int ctas = sms * (dtype == kF32 ? kClipCtas<float> : kClipCtas<__half>);
  const unsigned most = static_cast<unsigned>(ctas < kClipParts ? ctas : kClipParts);
  return chunks < most ? chunks : most;
}

template <typename T, typename O, int CAP>
cudaError_t launch_scale_t(const ClipParams<CAP>& p, int sms, cudaStream_t st) {
  return launch_overlapped(scale_kernel<T, O, CAP>, clip_grid(p.chunks, sizeof(T) == 4 ? kF32 : kF16, sms), kClipThreads, 0, st, p);
}

}  // namespace

long long clip_chunks(uintptr_t address, long long n, int size) {
  const long long per = 16 / size, off = static_cast<long long>(address & 15) / size;
  return ((off + n + per - 1) / per + kClipChunk - 1) / kClipChunk;
}

int clip_parts(unsigned chunks, int dtype, int sms) { return static_cast<int>(clip_grid(chunks, dtype, sms)); }

template <int CAP>
cudaError_t launch_squares(const ClipParams<CAP>& p, int dtype, int sms, cudaStream_t st) {
  auto* kernel = dtype == kF32    ? squares_kernel<float, CAP>
                 : dtype == kBF16 ? squares_kernel<__nv_bfloat16, CAP>
                                  : squares_kernel<__half, CAP>;
  return launch_overlapped(kernel, clip_grid(p.chunks, dtype, sms), kClipThreads, 0, st, p);
}

cudaError_t launch_norm_of_parts(const double* parts, int count, float* norm, cudaStream_t st) {
  return launch_overlapped(norm_kernel_of_parts, 1, kClipThreads, 0, st, parts, count, norm);
}

template <typename T, typename O>
static cudaError_t launch_small_t(const ClipParams<kClipFew>& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSmallCtas);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kSmallCtas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, small_clip_kernel<T, O>, p);
}

cudaError_t launch_small_clip(const ClipParams<kClipFew>& p, int dtype, int out_dtype, cudaStream_t st) {
  if (dtype == kF32) return launch_small_t<float, float>(p, st);
  if (dtype == kBF16)
    return out_dtype == kF32 ? launch_small_t<__nv_bfloat16, float>(p, st) : launch_small_t<__nv_bfloat16, __nv_bfloat16>(p, st);
  return out_dtype == kF32 ? launch_small_t<__half, float>(p, st) : launch_small_t<__half, __half>(p, st);
}

template <int CAP>
cudaError_t launch_scale(const ClipParams<CAP>& p, int dtype, int out_dtype, int sms, cudaStream_t st) {
  if (dtype == kF32) return launch_scale_t<float, float>(p, sms, st);
  if (dtype == kBF16)
    return out_dtype == kF32 ? launch_scale_t<__nv_bfloat16, float>(p, sms, st)
                             : launch_scale_t<__nv_bfloat16, __nv_bfloat16>(p, sms, st);
  return out_dtype == kF32 ? launch_scale_t<__half, float>(p, sms, st) : launch_scale_t<__half, __half>(p, sms, st);
}

template cudaError_t launch_squares(const ClipParams<kClipFew>&, int, int, cudaStream_t);
template cudaError_t launch_squares(const ClipParams<kClipTensors>&, int, int, cudaStream_t);
template cudaError_t launch_scale(const ClipParams<kClipFew>&, int, int, int, cudaStream_t);
template cudaError_t launch_scale(const ClipParams<kClipTensors>&, int, int, int, cudaStream_t);

}  // namespace demo
