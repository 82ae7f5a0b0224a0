// Root-mean-square norm of rows, with the residual's addition before it, into 16 or 32 bits and / or 8-bit
// codes with a scale for each block of 128:
//
//   s      = x + residual, rounded to the type it is stored in
//   rstd   = 1 / sqrt(mean(s^2) + eps), the float32 nearest to it
//   v      = (s rstd) w, two float32 products;  out = v rounded, codes = v / scale rounded
//
// Codes change by a step, and a scale by a factor of two, where v crosses a border.  So that they are a
// function of the row alone, and the fused kernel, the column form and a replica that cuts the row
// otherwise agree, the mean square is not a float32 sum but a pair of floats, right to about 2^-40 (float64
// would be 110 us of the SM's two lanes for 32768 x 2048).  A lane's sum H starts at the largest of its
// squares C, so H is never below a square, and Dekker's fast two-sum finds what an addition loses:
//   s = H + v^2,  l = v^2 - (s - H),  L += l,  H = s        (v^2 is exact inside a multiply-add)
// four instructions for two elements; the sum is (H - C) + L.  Lanes and warps are joined by Knuth's two-sum,
// and one Newton step in pairs makes rstd right before its rounding.  Rows whose mean square is outside
// 2^-60 .. 2^60 are summed again in float64 from the registers they are in.
//
// One pass over the row, held in registers.  Bound by HBM: 16384 x 2048 bfloat16 with a residual 29.7 us for the
// sum and rstd alone (6.8 TB/s), 44 us with the result (6.1 TB/s), 81 us in float32 (6.6 TB/s); with row codes
// 45 us (5.2 TB/s), 22 instructions an element, nine of them for the norm itself.  One row of 2048: 2.1 us, the
// launch.  Rows of 2051 (accesses of one element) 84 us.  The column form is a second kernel's (the quantizer's,
// on the sum as L2 still holds it): both forms 62 us, 40 for their bytes.
#include "train_norm.cuh"

namespace demo {

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

__device__ __forceinline__ Pair pair_sum(Pair p, int lanes = 32) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (d < lanes) p.join(Pair{__shfl_xor_sync(0xffffffffu, p.hi, d), __shfl_xor_sync(0xffffffffu, p.lo, d)});
  return p;
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

// 1 / sqrt(m): r (1 + (1 - m r^2) / 2) with the difference exact to about 2^-46 and below 2^-21.
__device__ __forceinline__ float rsqrt_pair(Pair m) {
  const float r = rsqrtf(m.hi);
  const float t = r * r, te = __fmaf_rn(r, r, -t);
  const float q = m.hi * t, qe = __fmaf_rn(m.hi, t, -q);
  const float d = (1.0f - q) - (qe + (m.hi * te + m.lo * t));
  return __fmaf_rn(0.5f * r, d, r);
}

// A row is the registers of W warps with up to UNITS accesses a lane: one warp (eight rows to a CTA of 256
// threads), or one CTA for the row.  UNITS 1 and 4 leave room for more warps an SM where rows are short (65536 x
// 768 bfloat16: 44 us), and K = 4 rows at a time where they are shorter than a unit (1048576 x 64: 68 us, of
// 39.4 for its bytes; one at a time 79).
constexpr int kNormUnits = 8;
constexpr int kNormThreads = 256, kNormWide = 1024;

template <typename T, typename W, bool VEC, int UNITS, int K, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kNormWide ? 1 : UNITS * K == 1 ? 5 : UNITS * K == 4 ? 3 : 2)
    norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int N = kNormN<T, VEC>;
  __shared__ Pair part[THREADS / 32];
  __shared__ double wide[THREADS / 32];
  const int lanes = UNITS == 1 ? p.lanes : 32, warps = K > 1 ? 1 : p.warps;
  const int in_cta = threadIdx.x >> 5, lane = threadIdx.x & (lanes - 1);
  const int warp = warps == 1 ? 0 : in_cta;  // of the row
  const int share = 32 / lanes;              // rows that a warp shares
  long long row0 = blockIdx.x;               // and K - 1 more, every `share`-th
  if (warps == 1) row0 = (row0 * (blockDim.x >> 5) + in_cta) * (share * K) + (threadIdx.x & 31) / lanes;
  const int cols = static_cast<int>(p.cols);
  const Place mine = Place::of<VEC, N>(warp, UNITS == 1 ? 1 : p.per, lane, lanes, cols);
  kernel_begin();
  if (__all_sync(0xffffffffu, row0 >= p.rows)) return;  // one warp to a row only: no barrier follows
  const auto place = [&](int k) {
    Place at = mine;
    if (UNITS == 1 && row0 + k * share >= p.rows) at.reach = 0;
    return at;
  };
  Unit<T, VEC, N> s[K][UNITS];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const T* x = static_cast<const T*>(p.x) + (row0 + k * share) * p.ldx + mine.first;
#pragma unroll
    for (int j = 0; j < UNITS; ++j) s[k][j].load(x, place(k), j);
  }
  if (p.residual != nullptr) {
    Unit<T, VEC, N> r[K][UNITS];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const T* res = static_cast<const T*>(p.residual) + (row0 + k * share) * p.ldr + mine.first;
#pragma unroll
      for (int j = 0; j < UNITS; ++j) r[k][j].load(res, place(k), j);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int j = 0; j < UNITS; ++j) s[k][j].add(r[k][j]);
      if (p.total != nullptr) {
        T* total = static_cast<T*>(p.total) + (row0 + k * share) * p.ldt + mine.first;
#pragma unroll
        for (int j = 0; j < UNITS; ++j) s[k][j].store(total, place(k), j);
      }
    }
  }
  Pair sum[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    // The largest magnitude of the lane; an infinity or NaN is met again in the sum.
    float top = 0.0f;
    if constexpr (Unit<T, VEC, N>::kPacked) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < UNITS; ++j)
#pragma unroll
        for (int i = 0; i < N / 2; ++i) m = packed_max_abs<T>(m, s[k][j].w[i]);
      const F2 v = widen<T>(m);
      top = fmaxf(v.x, v.y);
    } else {
#pragma unroll
      for (int j = 0; j < UNITS; ++j)
#pragma unroll
        for (int i = 0; i < N; i += 2)
          top = fmaxf(fmaxf(top, fabsf(__uint_as_float(s[k][j].w[i]))), fabsf(__uint_as_float(s[k][j].w[i + 1])));
    }
    const float c = top * top;
    const F2 minus = f2(-1.0f, -1.0f);
    F2 H = f2(c, c), L = f2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
      if (UNITS == 1 || mine.unit<VEC, N>(j, lane)) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const F2 v = s[k][j].get2(i), h = fma2(v, v, H);
          L = add2(L, fma2(v, v, fma2(h, minus, H)));  // v^2 - (h - H)
          H = h;
        }
      }
    }
    sum[k] = Pair{H.x, L.x};
    sum[k].add(-c);
    Pair other{H.y, L.y};
    other.add(-c);
    sum[k].join(other);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) sum[k] = pair_sum(sum[k], lanes);
  if (warps > 1) {
    if (lane == 0) part[warp] = sum[0];
    __syncthreads();
    sum[0] = pair_sum(lane < warps ? part[lane] : Pair{0.0f, 0.0f});
  }
  float rstd[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    bool fits;
    const Pair m = mean_eps(p, sum[k], &fits);
    rstd[k] = rsqrt_pair(m);
    if (__any_sync(0xffffffffu, !fits)) {  // the same for all of the row's warps
      double total = 0.0;
#pragma unroll
      for (int j = 0; j < UNITS; ++j) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const F2 v = s[k][j].get2(i);
          total += static_cast<double>(v.x) * v.x + static_cast<double>(v.y) * v.y;
        }
      }
      total = lane_sum(total, lanes);
      if (warps > 1) {
        if (lane == 0) wide[warp] = total;
        __syncthreads();
        total = lane_sum(lane < warps ? wide[lane] : 0.0);
      }
      if (!fits) rstd[k] = static_cast<float>(1.0 / sqrt(total * p.inv + p.eps));
    }
    if (p.rstd != nullptr && warp == 0 && lane == 0 && (UNITS > 1 || row0 + k * share < p.rows)) p.rstd[row0 + k * share] = rstd[k];
  }
  if (p.out == nullptr && p.codes == nullptr) return;

  const W* weight = static_cast<const W*>(p.weight) + mine.first;
  const int kp = static_cast<int>(p.col_blocks) * kBlock;
  const long long lds = (p.rows + 3) / 4 * 4;
#pragma unroll
  for (int j = 0; j < UNITS; ++j) {
    if (UNITS > 1 && !mine.unit<VEC, N>(j, lane)) continue;
    Unit<W, VEC, N> w;
    w.template load<true>(weight, mine, j);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long long row = row0 + k * share;
      const F2 r2 = f2(rstd[k], rstd[k]);
      F2 v[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) v[i] = mul2(mul2(s[k][j].get2(i), r2), w.get2(i));
      if (p.out != nullptr) {
        Unit<T, VEC, N> o;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) o.set2(i, v[i]);
        o.store(static_cast<T*>(p.out) + row * p.ldo + mine.first, place(k), j);
      }
      if (p.codes != nullptr) {
        float u[N], amax = 0.0f;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          u[2 * i] = v[i].x;
          u[2 * i + 1] = v[i].y;
          amax = max_abs_nan(amax, v[i].x, v[i].y);
        }
        if (!(amax <= 3.402823466e38f)) {  // something is not finite, or NaN past the row (0 times a NaN rstd)
          amax = 0.0f;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            u[e] = mine.has<VEC, N>(j, e) ? finite_or_nan(u[e]) : 0.0f;
            amax = fmaxf(amax, fabsf(u[e]));  // passes over a NaN
          }
        }
        // A block of 128 is 16 lanes of eight columns, a whole warp, or all lanes of a short row.
        constexpr int kSpan = kBlock / N < 32 ? kBlock / N : 32;
        uint32_t bits = __float_as_uint(amax);
        if constexpr (UNITS > 1 && kSpan == 32) {
          bits = __reduce_max_sync(0xffffffffu, bits);
        } else {
#pragma unroll
          for (int d = kSpan / 2; d > 0; d >>= 1)
            if (d < lanes) bits = umax32(bits, __shfl_xor_sync(0xffffffffu, bits, d));
        }
        const int exponent = scale_exponent(bits, fmt_top(p.fmt));
        const float inv = pow2f(-exponent);
        const F2 inv2 = f2(inv, inv);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const F2 h = mul2(f2(u[2 * i], u[2 * i + 1]), inv2);
          u[2 * i] = h.x;
          u[2 * i + 1] = h.y;
        }
        uint32_t q[N / 4];
#pragma unroll
        for (int e = 0; e < N; e += 4)
          q[e / 4] = p.fmt == kE4M3 ? codes4<kE4M3>(u[e], u[e + 1], u[e + 2], u[e + 3])
                                    : codes4<kE5M2>(u[e], u[e + 1], u[e + 2], u[e + 3]);
        const int off = mine.offset<VEC, N>(j, 0), c0 = mine.first + off;
        if (UNITS == 1 && lanes < kSpan) {
          // Short rows: the warp clears its rows' one block each before the lanes write what they hold (lane by
          // lane, a row of three columns would take 124 stores of a byte).
          const int row_lane = threadIdx.x & 31;
          const long long first = row - row_lane / lanes, left = p.rows - first;
          uint4* block = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.codes) + first * kBlock);
          const int units16 = (left < share ? static_cast<int>(left < 0 ? 0 : left) : share) * (kBlock / 16);
          for (int u = row_lane; u < units16; u += 32) block[u] = make_uint4(0, 0, 0, 0);
          __syncwarp();
        }
        if (UNITS > 1 || row < p.rows) {
          uint8_t* codes = static_cast<uint8_t*>(p.codes) + row * kp + mine.first;
          if constexpr (VEC) {
            if (c0 < kp) {
              if constexpr (N == 8)
                *reinterpret_cast<uint2*>(codes + off) = make_uint2(q[0], q[1]);
              else
                *reinterpret_cast<uint32_t*>(codes + off) = q[0];
            }
          } else if (UNITS == 1 && lanes == 1) {
            *reinterpret_cast<uint32_t*>(codes) = q[0];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) codes[off + lanes * e] = static_cast<uint8_t>(q[0] >> (8 * e));
          }
          if ((lane & (kSpan - 1)) == 0 && c0 < kp) {
            float* scale = p.scales + static_cast<long long>(c0 / kBlock) * lds;
            scale[row] = pow2f(exponent);
            if (row == p.rows - 1)  // rows past the matrix up to the scales' stride hold 1
              for (long long r = p.rows; r < lds; ++r) scale[r] = 1.0f;
          }
        }
      }
    }
  }
}

namespace {

// The fewest warps whose registers hold a row (more than eight: with four accesses a lane, if 32 warps are
// enough for that, as eight spill in a CTA of 1024 threads); with rows for less than eight warps an SM, up to
// one access a lane, so that one token's row is on its way at once.
int norm_warps(long long rows, long long units, int sms) {
  long long w = (units + kNormUnits - 1) / kNormUnits;
  if (w > 8 && units <= 4 * 32) w = (units + 3) / 4;
  while (2 * w <= 8 && 2 * w <= units && rows * w < 8LL * sms) w *= 2;
  return static_cast<int>(w);
}

template <typename T, typename W, bool VEC>
cudaError_t launch_norm_v(NormParams& p, int sms, cudaStream_t st) {
  constexpr int n = kNormN<T, VEC>;
  const long long units = (p.cols + 32 * n - 1) / (32 * n);
  p.warps = norm_warps(p.rows, units, sms);
  p.per = static_cast<int>((units + p.warps - 1) / p.warps);
  p.lanes = units == 1 ? row_lanes((p.cols + n - 1) / n) : 32;
  // Four short rows at a time where that leaves every SM eight CTAs.
  const bool several = units == 1 && p.rows / (kNormThreads / p.lanes) >= 32LL * sms;
  auto* kernel = several                     ? norm_kernel<T, W, VEC, 1, 4, kNormThreads>
                 : p.warps > kNormThreads / 32 ? (p.per <= 4 ? norm_kernel<T, W, VEC, 4, 1, kNormWide>
                                                             : norm_kernel<T, W, VEC, kNormUnits, 1, kNormWide>)
                 : p.per == 1                 ? norm_kernel<T, W, VEC, 1, 1, kNormThreads>
                 : p.per <= 4                 ? norm_kernel<T, W, VEC, 4, 1, kNormThreads>
                                             : norm_kernel<T, W, VEC, kNormUnits, 1, kNormThreads>;
  if (p.warps > 1) return launch_overlapped(kernel, static_cast<unsigned>(p.rows), 32 * p.warps, 0, st, p);
  const long long rows = kNormThreads / p.lanes * (several ? 4 : 1);  // of a CTA
  return launch_overlapped(kernel, static_cast<unsigned>((p.rows + rows - 1) / rows), kNormThreads, 0, st, p);
}

template <typename T, typename W>
cudaError_t launch_norm_t(NormParams& p, int sms, cudaStream_t st) {
  constexpr int n = kNormN<T, true>;
  const bool vec = p.cols % n == 0 && whole_rows(p.x, p.ldx, n) && whole_rows(p.weight, 0, n) &&
                   (p.residual == nullptr || whole_rows(p.residual, p.ldr, n)) &&
                   (p.total == nullptr || whole_rows(p.total, p.ldt, n)) &&
                   (p.out == nullptr || whole_rows(p.out, p.ldo, n));
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

}  // namespace demo
