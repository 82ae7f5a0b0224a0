// Root-mean-square norm of rows, with the residual's addition before it, into 16 or 32 bits and / or
// 8-bit codes with a scale for each block of 128; and its gradient.
//
//   s      = x + residual, rounded to the type it is stored in
//   rstd   = 1 / sqrt(mean(s^2) + eps), the float32 nearest to it
//   v      = (s rstd) w, two float32 products;  out = v rounded, codes = v / scale rounded
//   with dy the result's gradient, xh = s rstd and c = mean(dy w xh):
//   dx     = rstd (dy w - xh c) + past,   dw = sum over the rows of dy xh
//
// Codes change by a step, and a scale by a factor of two, where v crosses a border.  So that they are a
// function of the row alone, and the fused kernel, the column form and a replica that cuts the row
// otherwise agree, the mean square is not a float32 sum: squares are exact (a product of 8 or 11 bits, or a
// product and its error by a multiply-add), their sum is a pair of floats joined by Knuth's two-sum (seven
// additions an element, where float64 would be 110 us of the SM's two lanes for 32768 x 2048), and one
// Newton step in pairs makes rstd right to about 2^-40 before its rounding.  Rows whose mean square is
// outside 2^-60 .. 2^60 are summed again in float64 from the registers they are in.
#include "train_common.cuh"

namespace demo {

// How a row lies in the registers of its W warps.  Unit j of warp w covers 32 N columns, from
// (j W + w) 32 N on; lane l holds N consecutive ones as one 16-byte access, or, where rows are not whole
// aligned accesses, N columns 32 apart (N = 4, so that a block of 128 is one unit of one warp).
template <typename T>
constexpr bool is_bf16 = false;
template <>
constexpr bool is_bf16<__nv_bfloat16> = true;

template <typename T, bool VEC>
constexpr int kNormN = VEC ? 16 / static_cast<int>(sizeof(T)) : 4;

template <bool VEC, int N>
__device__ __forceinline__ int norm_column(int base, int lane, int e) {
  return VEC ? base + lane * N + e : base + 32 * e + lane;
}

// Two 16-bit elements in a word, the first in its low half.
template <typename T>
__device__ __forceinline__ float half_of(uint32_t w, int e) {
  if constexpr (sizeof(T) == 2) {
    const uint16_t h = static_cast<uint16_t>(e & 1 ? w >> 16 : w);
    if constexpr (is_bf16<T>) return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
    return __half2float(__ushort_as_half(h));
  }
  return 0.0f;
}

template <typename T>
__device__ __forceinline__ uint32_t halves(float lo, float hi) {
  if constexpr (is_bf16<T>) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A lane's N elements of a unit: whole accesses of 16 bits stay packed in words (as an array of 16-bit
// elements they took a register each: 152 instead of 89 a thread), all others are float32.
template <typename T, bool VEC, int N>
struct Unit {
  static constexpr bool kPacked = VEC && sizeof(T) == 2;
  static constexpr int kWords = kPacked ? N / 2 : N;
  uint32_t w[kWords];

  __device__ __forceinline__ float get(int e) const {
    if constexpr (kPacked) return half_of<T>(w[e / 2], e);
    return __uint_as_float(w[e]);
  }
  // The float32 values rounded to T.
  __device__ __forceinline__ void round(const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (kPacked)
        w[i] = halves<T>(v[2 * i], v[2 * i + 1]);
      else
        w[i] = __float_as_uint(to_f32(from_f32<T>(v[i])));
    }
  }
  // N elements of a row at `base`, zero past its end.  CONST: memory that the kernel does not write.
  template <bool CONST = false>
  __device__ __forceinline__ void load(const T* row, int base, int lane, int cols) {
    if constexpr (VEC) {
      if (base + lane * N < cols) {
        const uint4* q = reinterpret_cast<const uint4*>(row + base + lane * N);
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 v = CONST ? __ldg(q + i) : q[i];
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int c = norm_column<VEC, N>(base, lane, e);
        w[e] = c < cols ? __float_as_uint(to_f32(CONST ? __ldg(row + c) : row[c])) : 0u;
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int base, int lane, int cols) const {
    if constexpr (VEC) {
      if (base + lane * N < cols) *reinterpret_cast<uint4*>(row + base + lane * N) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int c = norm_column<VEC, N>(base, lane, e);
        if (c < cols) row[c] = from_f32<T>(get(e));
      }
    }
  }
};

// hi + lo, with lo below hi's last place.
struct Pair {
  float hi, lo;
  __device__ __forceinline__ void add(float b) {
    const float s = hi + b, t = s - hi;
    lo += (hi - (s - t)) + (b - t);
    hi = s;
  }
  // The order of the two does not matter, so lanes that exchange their pairs agree.
  __device__ __forceinline__ void join(Pair o) {
    const float s = hi + o.hi, t = s - hi;
    lo = (lo + o.lo) + ((hi - (s - t)) + (o.hi - t));
    hi = s;
  }
};

__device__ __forceinline__ Pair lane_sum(Pair p) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    p.join(Pair{__shfl_xor_sync(0xffffffffu, p.hi, d), __shfl_xor_sync(0xffffffffu, p.lo, d)});
  return p;
}

__device__ __forceinline__ double lane_sum(double v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

constexpr float kPairLow = 0x1p-60f, kPairHigh = 0x1p60f;

// sum / cols + eps; `fits` says whether the pairs' bounds hold for it.
__device__ __forceinline__ Pair mean_eps(const NormParams& p, Pair sum, bool* fits) {
  Pair m;
  m.hi = sum.hi * p.inv_hi;
  m.lo = __fmaf_rn(sum.hi, p.inv_hi, -m.hi) + (sum.hi * p.inv_lo + sum.lo * p.inv_hi);
  m.add(p.eps_hi);
  m.lo += p.eps_lo;
  const float h = m.hi + m.lo;  // back to lo below hi's last place
  m.lo -= h - m.hi;
  m.hi = h;
  *fits = sum.hi <= kPairHigh && m.hi >= kPairLow && m.hi <= kPairHigh;  // false for NaN
  return m;
}

// 1 / sqrt(m): r0 (1 + (1 - m r0^2) / 2) with the difference exact to about 2^-46 and |difference| below 2^-21.
__device__ __forceinline__ float rsqrt_pair(Pair m) {
  const float r = rsqrtf(m.hi);
  const float t = r * r, te = __fmaf_rn(r, r, -t);
  const float q = m.hi * t, qe = __fmaf_rn(m.hi, t, -q);
  const float d = (1.0f - q) - (qe + (m.hi * te + m.lo * t));
  return __fmaf_rn(0.5f * r, d, r);
}

// ----------------------------------------------------------------------------
// Forward
// ----------------------------------------------------------------------------

// A row is W warps' registers: one warp (eight rows to a CTA) up to 64 elements a lane in 16 bits and 32 in
// 32 bits, else one CTA for the row.
constexpr int kNormUnits = 8;
constexpr int kNormThreads = 256, kNormWide = 1024;

template <typename T, typename W, bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kNormThreads ? 2 : 1) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int N = kNormN<T, VEC>;
  __shared__ Pair part[THREADS / 32];
  __shared__ double wide[THREADS / 32];
  const int lane = threadIdx.x & 31, warps = p.warps;
  const int in_cta = threadIdx.x >> 5;
  const int warp = warps == 1 ? 0 : in_cta;  // of the row
  const long long row = warps == 1 ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + in_cta : blockIdx.x;
  const int cols = static_cast<int>(p.cols);
  kernel_begin();
  if (row >= p.rows) return;  // one warp to a row only: whole warps, and no barrier follows
  Unit<T, VEC, N> s[kNormUnits];
  {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
#pragma unroll
    for (int j = 0; j < kNormUnits; ++j) {
      const int base = (j * warps + warp) * 32 * N;
      if (base < cols) s[j].load(x, base, lane, cols);
    }
    if (p.residual != nullptr) {
      const T* res = static_cast<const T*>(p.residual) + row * p.ldr;
      Unit<T, VEC, N> r[kNormUnits];
#pragma unroll
      for (int j = 0; j < kNormUnits; ++j) {
        const int base = (j * warps + warp) * 32 * N;
        if (base < cols) r[j].load(res, base, lane, cols);
      }
      T* total = static_cast<T*>(p.total) + row * p.ldt;
#pragma unroll
      for (int j = 0; j < kNormUnits; ++j) {
        const int base = (j * warps + warp) * 32 * N;
        if (base < cols) {
          float v[N];
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] = s[j].get(e) + r[j].get(e);
          s[j].round(v);
          if (p.total != nullptr) s[j].store(total, base, lane, cols);
        }
      }
    }
  }
  Pair sum{0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < kNormUnits; ++j) {
    if ((j * warps + warp) * 32 * N < cols) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float v = s[j].get(e), q = v * v;
        if constexpr (sizeof(T) == 4) sum.lo += __fmaf_rn(v, v, -q);
        sum.add(q);
      }
    }
  }
  sum = lane_sum(sum);
  if (warps > 1) {
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    sum = lane_sum(lane < warps ? part[lane] : Pair{0.0f, 0.0f});
  }
  bool fits;
  const Pair m = mean_eps(p, sum, &fits);
  float rstd;
  if (fits) {
    rstd = rsqrt_pair(m);
  } else {  // the same for all of the row's warps
    double total = 0.0;
#pragma unroll
    for (int j = 0; j < kNormUnits; ++j) {
      if ((j * warps + warp) * 32 * N < cols) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const double v = s[j].get(e);
          total += v * v;
        }
      }
    }
    total = lane_sum(total);
    if (warps > 1) {
      if (lane == 0) wide[warp] = total;
      __syncthreads();
      total = lane_sum(lane < warps ? wide[lane] : 0.0);
    }
    rstd = static_cast<float>(1.0 / sqrt(total * p.inv + p.eps));
  }
  if (p.rstd != nullptr && warp == 0 && lane == 0) p.rstd[row] = rstd;
  if (p.out == nullptr && p.codes == nullptr) return;

  const W* weight = static_cast<const W*>(p.weight);
  T* out = static_cast<T*>(p.out) + row * p.ldo;
  const int kp = static_cast<int>(p.col_blocks) * kBlock;
  uint8_t* codes = static_cast<uint8_t*>(p.codes) + row * kp;
  const long long lds = (p.rows + 3) / 4 * 4;
#pragma unroll
  for (int j = 0; j < kNormUnits; ++j) {
    const int base = (j * warps + warp) * 32 * N;
    if (base < cols) {
      Unit<W, VEC, N> w;
      w.template load<true>(weight, base, lane, cols);
      float v[N];
#pragma unroll
      for (int e = 0; e < N; ++e)  // 0 past the row, also where rstd is NaN
        v[e] = norm_column<VEC, N>(base, lane, e) < cols ? s[j].get(e) * rstd * w.get(e) : 0.0f;
      if (p.out != nullptr) {
        Unit<T, VEC, N> o;
        o.round(v);
        o.store(out, base, lane, cols);
      }
      if (p.codes != nullptr) {
        float odd = 0.0f;  // NaN once an element is infinite or NaN
#pragma unroll
        for (int e = 0; e < N; ++e) odd = fmaf(v[e], 0.0f, odd);
        if (odd != odd) {
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] = finite_or_nan(v[e]);
        }
        float m4 = 0.0f;  // fmaxf passes over a NaN
#pragma unroll
        for (int e = 0; e < N; ++e) m4 = fmaxf(m4, fabsf(v[e]));
        // A block of 128 is 16 lanes of eight columns, or a whole warp.
        uint32_t bits = __float_as_uint(m4);
        if constexpr (N == 8) {
#pragma unroll
          for (int d = 8; d > 0; d >>= 1) bits = umax32(bits, __shfl_xor_sync(0xffffffffu, bits, d));
        } else {
          bits = __reduce_max_sync(0xffffffffu, bits);
        }
        const int exponent = scale_exponent(bits, fmt_top(p.fmt));
        const float inv = pow2f(-exponent);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] *= inv;
        const int c0 = norm_column<VEC, N>(base, lane, 0);
        if constexpr (VEC) {
          if (c0 < kp) {
            uint32_t q[N / 4];
#pragma unroll
            for (int e = 0; e < N; e += 4)
              q[e / 4] = p.fmt == kE4M3 ? codes4<kE4M3>(v[e], v[e + 1], v[e + 2], v[e + 3])
                                        : codes4<kE5M2>(v[e], v[e + 1], v[e + 2], v[e + 3]);
            if constexpr (N == 8)
              *reinterpret_cast<uint2*>(codes + c0) = make_uint2(q[0], q[1]);
            else
              *reinterpret_cast<uint32_t*>(codes + c0) = q[0];
          }
        } else {
          const uint32_t q = p.fmt == kE4M3 ? codes4<kE4M3>(v[0], v[1], v[2], v[3]) : codes4<kE5M2>(v[0], v[1], v[2], v[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) codes[c0 + 32 * e] = static_cast<uint8_t>(q >> (8 * e));
        }
        const bool first = (lane & (N == 8 ? 15 : 31)) == 0;
        if (first && c0 < kp) {
          float* scale = p.scales + static_cast<long long>(c0 / kBlock) * lds;
          scale[row] = pow2f(exponent);
          if (row == p.rows - 1)  // rows past the matrix up to the scales' stride hold 1
            for (long long r = p.rows; r < lds; ++r) scale[r] = 1.0f;
        }
      }
    }
  }
}

namespace {

bool whole(const void* q, long long ld, int n) {
  return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld % n == 0;
}

// The fewest warps whose registers hold a row; with rows for less than eight warps an SM, up to one
// access a lane, so that one token's row is on its way at once.
int norm_warps(long long rows, long long cols, int n, int units, int sms) {
  const long long all = (cols + 32 * n - 1) / (32 * n);
  const long long least = (all + units - 1) / units;
  long long w = least;
  while (2 * w <= 8 && 2 * w <= all && rows * w < 8LL * sms) w *= 2;
  return static_cast<int>(w);
}

template <typename T, typename W, bool VEC>
cudaError_t launch_norm_v(NormParams& p, int sms, cudaStream_t st) {
  p.warps = norm_warps(p.rows, p.cols, kNormN<T, VEC>, kNormUnits, sms);
  if (p.warps == 1)
    return launch_overlapped(norm_kernel<T, W, VEC, kNormThreads>,
                             static_cast<unsigned>((p.rows + kNormThreads / 32 - 1) / (kNormThreads / 32)), kNormThreads, 0,
                             st, p);
  auto* kernel = p.warps <= kNormThreads / 32 ? norm_kernel<T, W, VEC, kNormThreads> : norm_kernel<T, W, VEC, kNormWide>;
  return launch_overlapped(kernel, static_cast<unsigned>(p.rows), 32 * p.warps, 0, st, p);
}

template <typename T, typename W>
cudaError_t launch_norm_t(NormParams& p, int sms, cudaStream_t st) {
  constexpr int n = kNormN<T, true>;
  const bool vec = p.cols % n == 0 && whole(p.x, p.ldx, n) && whole(p.weight, 0, n) &&
                   (p.residual == nullptr || whole(p.residual, p.ldr, n)) &&
                   (p.total == nullptr || whole(p.total, p.ldt, n)) && (p.out == nullptr || whole(p.out, p.ldo, n));
  return vec ? launch_norm_v<T, W, true>(p, sms, st) : launch_norm_v<T, W, false>(p, sms, st);
}

}  // namespace

cudaError_t launch_norm(NormParams& p, int dtype, int weight_dtype, int sms, cudaStream_t st) {
  if (dtype == kF32) return launch_norm_t<float, float>(p, sms, st);
  if (dtype == kBF16)
    return weight_dtype == kF32 ? launch_norm_t<__nv_bfloat16, float>(p, sms, st)
                                : launch_norm_t<__nv_bfloat16, __nv_bfloat16>(p, sms, st);
  return weight_dtype == kF32 ? launch_norm_t<__half, float>(p, sms, st) : launch_norm_t<__half, __half>(p, sms, st);
}

// ----------------------------------------------------------------------------
// Gradient
// ----------------------------------------------------------------------------

// One read of dy and s makes both gradients: a row's group of W warps holds it in registers, sums
// dy w xh over it, writes dx and adds dy xh to each lane's own columns of dw, which stay in
// registers over all rows of the group.  At the end the CTA's groups are joined in shared memory, in their
// order, the CTAs' sums by a second kernel, in theirs: no atomics, the same bits from call to call.
// Lanes hold 32 elements of packed 16 bits, and of anything in rows that need more than 16 warps; 16 of float32
// (32 would spill 276 bytes a thread).
constexpr int kGradThreads = 512, kGradWide = 1024;
template <typename T, bool VEC, int THREADS>
constexpr int kGradUnits = ((VEC && sizeof(T) == 2) || THREADS == kGradWide ? 32 : 16) / kNormN<T, VEC>;

__device__ __forceinline__ void group_barrier(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}

template <typename T, typename W, bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  constexpr int N = kNormN<T, VEC>, U = kGradUnits<T, VEC, THREADS>;
  extern __shared__ float joined[];  // the CTA's dw, where it has several groups
  __shared__ float part[2][THREADS / 32];
  const int lane = threadIdx.x & 31, in_cta = threadIdx.x >> 5, warps = p.warps;
  const int group = in_cta / warps, warp = in_cta - group * warps, groups = (blockDim.x >> 5) / warps;
  const int cols = static_cast<int>(p.cols);
  kernel_begin();
  const W* weight = static_cast<const W*>(p.weight);
  float acc[U][N];
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int e = 0; e < N; ++e) acc[j][e] = 0.0f;
  int turn = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * groups + group; row < p.rows;
       row += static_cast<long long>(gridDim.x) * groups, turn ^= 1) {
    const T* dyr = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* sr = static_cast<const T*>(p.total) + row * p.ldt;
    Unit<T, VEC, N> dy[U], s[U], past[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int base = (j * warps + warp) * 32 * N;
      if (base < cols) {
        dy[j].load(dyr, base, lane, cols);
        s[j].load(sr, base, lane, cols);
      }
    }
    if (p.past != nullptr) {
      const T* pr = static_cast<const T*>(p.past) + row * p.ldp;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int base = (j * warps + warp) * 32 * N;
        if (base < cols) past[j].load(pr, base, lane, cols);
      }
    }
    const float rstd = p.rstd[row];
    float dot = 0.0f;  // sum of dy w xh
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int base = (j * warps + warp) * 32 * N;
      if (base < cols) {
        Unit<W, VEC, N> w;
        w.template load<true>(weight, base, lane, cols);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float d = dy[j].get(e), xh = s[j].get(e) * rstd;
          dot = __fmaf_rn(d * w.get(e), xh, dot);
          acc[j][e] = __fmaf_rn(d, xh, acc[j][e]);
        }
      }
    }
    dot = lane_sum(dot);
    if (warps > 1) {
      // A warp is at most one barrier ahead of the others of its group: two slots are enough.
      if (lane == 0) part[turn][in_cta] = dot;
      group_barrier(group, 32 * warps);
      dot = lane_sum(lane < warps ? part[turn][group * warps + lane] : 0.0f);
    }
    const float c = dot * p.inv;
    T* dxr = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int base = (j * warps + warp) * 32 * N;
      if (base < cols) {
        Unit<W, VEC, N> w;
        w.template load<true>(weight, base, lane, cols);
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float xh = s[j].get(e) * rstd;
          v[e] = __fmaf_rn(-xh, c, dy[j].get(e) * w.get(e)) * rstd;
          if (p.past != nullptr) v[e] += past[j].get(e);
        }
        Unit<T, VEC, N> o;
        o.round(v);
        o.store(dxr, base, lane, cols);
      }
    }
  }
  if (p.dw == nullptr) return;
  // One CTA writes dw itself.
  const bool last = gridDim.x == 1;
  float* dst = last ? p.dw : p.partials + static_cast<long long>(blockIdx.x) * cols;
  for (int g = 0; g < groups; ++g) {
    if (group == g) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int base = (j * warps + warp) * 32 * N;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int col = norm_column<VEC, N>(base, lane, e);
          if (col < cols) {
            const float v = g > 0 ? joined[col] + acc[j][e] : acc[j][e];
            if (g + 1 < groups)
              joined[col] = v;
            else
              dst[col] = last && p.add ? dst[col] + v : v;
          }
        }
      }
    }
    if (groups > 1) __syncthreads();
  }
}

// dw from the CTAs' sums: 32 columns to a CTA, eight warps take every eighth sum.
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(32 * kJoinWarps) norm_dw_kernel(const float* partials, int parts, int cols, float* dw, int add) {
  __shared__ float sh[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  kernel_begin();
  float v = 0.0f;
  if (col < cols) {
#pragma unroll 8
    for (int i = warp; i < parts; i += kJoinWarps) v += partials[static_cast<long long>(i) * cols + col];
  }
  sh[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && col < cols) {
    float t = sh[0][lane];
#pragma unroll
    for (int i = 1; i < kJoinWarps; ++i) t += sh[i][lane];
    dw[col] = add ? dw[col] + t : t;
  }
}

namespace {

template <typename T, typename W, bool VEC, int THREADS>
cudaError_t launch_norm_grad_w(NormGradParams& p, int sms, cudaStream_t st) {
  constexpr int n = kNormN<T, VEC>, u = kGradUnits<T, VEC, THREADS>, most = THREADS / 32;
  const long long units = (p.cols + 32 * n - 1) / (32 * n);
  p.warps = static_cast<int>((units + u - 1) / u);
  if constexpr (THREADS == kGradThreads) {
    if (p.warps > most) return launch_norm_grad_w<T, W, VEC, kGradWide>(p, sms, st);
  }
  long long groups = THREADS == kGradThreads ? most / p.warps : 1;
  if (groups > p.rows) groups = p.rows > 0 ? p.rows : 1;
  const int threads = static_cast<int>(32 * p.warps * groups);
  long long grid = (p.rows + groups - 1) / groups;
  if (grid > sms) grid = sms;
  if (grid > kNormParts) grid = kNormParts;
  if (grid < 1) grid = 1;  // no rows: dw is 0
  const size_t smem = groups > 1 ? static_cast<size_t>(p.cols) * sizeof(float) : 0;
  const cudaError_t e =
      launch_overlapped(norm_grad_kernel<T, W, VEC, THREADS>, static_cast<unsigned>(grid), threads, smem, st, p);
  if (e != cudaSuccess || p.dw == nullptr || grid == 1) return e;
  return launch_overlapped(norm_dw_kernel, static_cast<unsigned>((p.cols + 31) / 32), 32 * kJoinWarps, 0, st,
                           static_cast<const float*>(p.partials), static_cast<int>(grid), static_cast<int>(p.cols), p.dw, p.add);
}

template <typename T, typename W>
cudaError_t launch_norm_grad_t(NormGradParams& p, int sms, cudaStream_t st) {
  constexpr int n = kNormN<T, true>;
  const bool vec = p.cols % n == 0 && whole(p.dy, p.lddy, n) && whole(p.total, p.ldt, n) && whole(p.weight, 0, n) &&
                   whole(p.dx, p.lddx, n) && (p.past == nullptr || whole(p.past, p.ldp, n));
  return vec ? launch_norm_grad_w<T, W, true, kGradThreads>(p, sms, st)
             : launch_norm_grad_w<T, W, false, kGradThreads>(p, sms, st);
}

}  // namespace

cudaError_t launch_norm_grad(NormGradParams& p, int dtype, int weight_dtype, int sms, cudaStream_t st) {
  if (dtype == kF32) return launch_norm_grad_t<float, float>(p, sms, st);
  if (dtype == kBF16)
    return weight_dtype == kF32 ? launch_norm_grad_t<__nv_bfloat16, float>(p, sms, st)
                                : launch_norm_grad_t<__nv_bfloat16, __nv_bfloat16>(p, sms, st);
  return weight_dtype == kF32 ? launch_norm_grad_t<__half, float>(p, sms, st)
                              : launch_norm_grad_t<__half, __half>(p, sms, st);
}

}  // namespace demo
