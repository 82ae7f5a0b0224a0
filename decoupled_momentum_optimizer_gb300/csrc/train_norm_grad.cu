// The gradient of the root-mean-square norm.  With dy the result's gradient, xh = s rstd and
// c = mean(dy w xh) over the row:
//
//   dx = rstd (dy w - xh c) + past,   dw = sum over the rows of dy xh
//
// One read of dy and s makes both: a row's group of W warps holds it in registers, sums dy w xh over it, writes
// dx and adds dy xh to each lane's own columns of dw, which stay in registers over all rows of the group.  Rows of
// a half or a quarter of the registers are taken two or four at a time, so that as many bytes are on their way
// for short rows as for long ones, and rows of less than a warp share it.  At the end the CTA's groups are joined
// in shared memory, in their order, the CTAs' sums by a second kernel, in theirs: no atomics, the same bits
// from call to call.
//
// Bound by HBM: 32768 x 2048 bfloat16 with `past` 88 us (6.1 TB/s), 16384 x 2048 float32 85 us (6.4 TB/s), 65536 x 768
// bfloat16 69 us; 18 instructions an element, issue slots 32% busy.  (256 threads a CTA and two of those: 91, 86, 71
// us; 384 threads: 95, 91, 76.)  4096 x 8192 bfloat16, where eight warps meet at a barrier for each row, 56 us
// (4.8 TB/s); 16384 x 2051 bfloat16, accesses of one element, 124 us.
#include "train_norm.cuh"

namespace demo {

// U accesses a lane of one row, K rows at a time: 32 elements of packed 16 bits, 16 of others (32 spill 100 to 316
// bytes a thread).  Rows that 16 warps do not hold so have 32 elements a lane of any type, and then up to 32 warps, which
// spill more: 2000 x 12288 float32 108 us (3.6 TB/s), 436 x 12255 bfloat16 36 us (61 with 32 warps).
constexpr int kGradThreads = 512, kGradWide = 1024;
template <typename T, bool VEC, int THREADS>
constexpr int kGradUnits = ((VEC && sizeof(T) == 2) || THREADS == kGradWide ? 32 : 16) / kNormN<T, VEC>;

constexpr int kStagedWarps = 8;  // of a group whose sums pass through shared memory

__device__ __forceinline__ void group_barrier(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}

template <typename T, typename W, bool VEC, int U, int K, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  constexpr int N = kNormN<T, VEC>;
  extern __shared__ float joined[];  // sums over rows on their way
  __shared__ float part[2][K][THREADS / 32];
  const int lanes = U == 1 ? p.lanes : 32, warps = p.warps;
  const int in_cta = threadIdx.x >> 5, lane = threadIdx.x & (lanes - 1);
  const int group = in_cta / warps, warp = in_cta - group * warps, groups = (blockDim.x >> 5) / warps;
  const int cols = static_cast<int>(p.cols);
  const int share = 32 / lanes;  // rows that a warp shares (one where a row has several)
  const Place mine = Place::of<VEC, N>(warp, p.per, lane, lanes, cols);
  kernel_begin();
  const W* weight = static_cast<const W*>(p.weight) + mine.first;
  F2 acc[U][N / 2];
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int i = 0; i < N / 2; ++i) acc[j][i] = f2(0.0f, 0.0f);
  int turn = 0;
  const long long step = static_cast<long long>(groups) * share * K;
  for (long long first = blockIdx.x * step + static_cast<long long>(group) * share * K; first < p.rows;
       first += gridDim.x * step, turn ^= 1) {
    const long long row0 = first + (threadIdx.x & 31) / lanes;  // and every `share`-th
    Unit<T, VEC, N> dy[K][U], s[K][U], past[K][U];
    float rstd[K], dot[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long long row = row0 + k * share;
      Place at = mine;
      if (row >= p.rows) at.reach = 0;
      const T* dyr = static_cast<const T*>(p.dy) + row * p.lddy + at.first;
      const T* sr = static_cast<const T*>(p.total) + row * p.ldt + at.first;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        dy[k][j].load(dyr, at, j);
        s[k][j].load(sr, at, j);
      }
      if (p.past != nullptr) {
        const T* pr = static_cast<const T*>(p.past) + row * p.ldp + at.first;
#pragma unroll
        for (int j = 0; j < U; ++j) past[k][j].load(pr, at, j);
      }
      rstd[k] = row < p.rows ? p.rstd[row] : 0.0f;
    }
    F2 sum[K];
#pragma unroll
    for (int k = 0; k < K; ++k) sum[k] = f2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (U == 1 || mine.unit<VEC, N>(j, lane)) {
        Unit<W, VEC, N> w;
        w.template load<true>(weight, mine, j);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const F2 r2 = f2(rstd[k], rstd[k]);
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            const F2 d = dy[k][j].get2(i), xh = mul2(s[k][j].get2(i), r2);
            sum[k] = fma2(mul2(d, w.get2(i)), xh, sum[k]);
            acc[j][i] = fma2(d, xh, acc[j][i]);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float2 h = sum[k];
      dot[k] = lane_sum(h.x + h.y, lanes);
    }
    if (warps > 1) {
      // A warp is at most one barrier ahead of the others of its group: two slots are enough.
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) part[turn][k][in_cta] = dot[k];
      }
      group_barrier(group, 32 * warps);
#pragma unroll
      for (int k = 0; k < K; ++k) dot[k] = lane_sum(lane < warps ? part[turn][k][group * warps + lane] : 0.0f);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (U == 1 || mine.unit<VEC, N>(j, lane)) {
        Unit<W, VEC, N> w;
        w.template load<true>(weight, mine, j);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const long long row = row0 + k * share;
          const float c = -(dot[k] * p.inv);
          const F2 r2 = f2(rstd[k], rstd[k]), c2 = f2(c, c);
          Unit<T, VEC, N> o;
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            const F2 g = mul2(dy[k][j].get2(i), w.get2(i)), xh = mul2(s[k][j].get2(i), r2);
            F2 v = mul2(fma2(xh, c2, g), r2);
            if (p.past != nullptr) v = add2(v, past[k][j].get2(i));
            o.set2(i, v);
          }
          Place at = mine;
          if (row >= p.rows) at.reach = 0;
          o.store(static_cast<T*>(p.dx) + row * p.lddx + at.first, at, j);
        }
      }
    }
  }
  if (p.dw == nullptr) return;
  if constexpr (U == 1) {  // the rows that the warp shares
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      if (d >= lanes) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) acc[0][i] = add2(acc[0][i], f2(__shfl_xor_sync(0xffffffffu, acc[0][i].x, d),
                                                               __shfl_xor_sync(0xffffffffu, acc[0][i].y, d)));
      }
    }
  }
  // The groups' sums, halving their number: the later half writes, the earlier half adds.  A lane's elements lie
  // 33 floats apart, lanes one apart: no two lanes meet in a bank, here or when the columns are read in order.
  const auto slot = [](int warp, int j, int e, int lane) { return ((warp * U + j) * N + e) * 33 + lane; };
  const int last_lane = threadIdx.x & 31;
  for (int left = groups; left > 1;) {
    const int half = (left + 1) / 2;
    if (group >= half && group < left) {
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e)
          joined[slot((group - half) * warps + warp, j, e, last_lane)] = e % 2 ? acc[j][e / 2].y : acc[j][e / 2].x;
    }
    __syncthreads();
    if (group < left - half) {
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
          acc[j][i] = add2(acc[j][i], f2(joined[slot(group * warps + warp, j, 2 * i, last_lane)],
                                         joined[slot(group * warps + warp, j, 2 * i + 1, last_lane)]));
    }
    __syncthreads();
    left = half;
  }
  // One CTA writes dw itself.
  const bool last = gridDim.x == 1;
  float* dst = last ? p.dw : p.partials + static_cast<long long>(blockIdx.x) * cols;
  if (warps > kStagedWarps) {  // one group, whose registers do not fit
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (mine.has<VEC, N>(j, e)) {
          float* d = dst + mine.first + mine.offset<VEC, N>(j, e);
          const float v = e % 2 ? acc[j][e / 2].y : acc[j][e / 2].x;
          *d = last && p.add ? *d + v : v;
        }
      }
    return;
  }
  if (group == 0) {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) joined[slot(warp, j, e, last_lane)] = e % 2 ? acc[j][e / 2].y : acc[j][e / 2].x;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < cols; c += blockDim.x) {
    const int unit = c / (32 * N), in = c - unit * 32 * N, w = U == 1 ? unit : unit / p.per, j = unit - w * p.per;
    const float v = VEC ? joined[slot(w, j, in % N, in / N)] : joined[slot(w, j, in / lanes, in % lanes)];
    dst[c] = last && p.add ? dst[c] + v : v;
  }
}

// dw from the CTAs' sums: 32 columns to a CTA, sixteen warps take every sixteenth sum.
constexpr int kJoinWarps = 16;

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

template <typename T, typename W, bool VEC, int U, int K, int THREADS>
cudaError_t launch_norm_grad_u(NormGradParams& p, long long units, int sms, cudaStream_t st) {
  p.warps = static_cast<int>((units + U - 1) / U);
  p.lanes = U == 1 && units == 1 ? row_lanes((p.cols + kNormN<T, VEC> - 1) / kNormN<T, VEC>) : 32;
  p.per = static_cast<int>((units + p.warps - 1) / p.warps);
  const long long rows = (32 / p.lanes) * K;  // of a group
  // As many groups as fit, but no more than give every SM a CTA; rows that one CTA takes at once are one
  // CTA's, which needs no second kernel.
  const long long most = THREADS == kGradThreads ? kGradThreads / 32 / p.warps : 1;
  const long long turns = (p.rows + rows - 1) / rows, spread = (turns + sms - 1) / sms;
  const long long groups = turns <= most ? (turns < 1 ? 1 : turns) : spread < most ? spread : most;
  long long grid = (p.rows + groups * rows - 1) / (groups * rows);
  if (grid > sms) grid = sms;
  if (grid > kNormParts) grid = kNormParts;
  if (grid < 1) grid = 1;  // no rows: dw is 0
  // half of the groups' registers, or one group's: 33 KB at most
  const long long kept = p.warps > kStagedWarps ? 0 : groups > 1 ? groups / 2 : 1;
  const size_t smem = p.dw != nullptr ? static_cast<size_t>(kept * p.warps * U * kNormN<T, VEC> * 33) * sizeof(float) : 0;
  const cudaError_t e = launch_overlapped(norm_grad_kernel<T, W, VEC, U, K, THREADS>, static_cast<unsigned>(grid),
                                          static_cast<unsigned>(32 * p.warps * groups), smem, st, p);
  if (e != cudaSuccess || p.dw == nullptr || grid == 1) return e;
  return launch_overlapped(norm_dw_kernel, static_cast<unsigned>((p.cols + 31) / 32), 32 * kJoinWarps, 0, st,
                           static_cast<const float*>(p.partials), static_cast<int>(grid), static_cast<int>(p.cols), p.dw, p.add);
}

template <typename T, typename W, bool VEC>
cudaError_t launch_norm_grad_v(NormGradParams& p, int sms, cudaStream_t st) {
  constexpr int n = kNormN<T, VEC>, most = kGradThreads / 32;
  constexpr int u = kGradUnits<T, VEC, kGradThreads>;
  static_assert(u == 4, "four accesses a lane: rows of one or two units are taken four or two at a time");
  const long long units = (p.cols + 32 * n - 1) / (32 * n);
  if (units == 1) return launch_norm_grad_u<T, W, VEC, 1, 4, kGradThreads>(p, units, sms, st);
  if (units == 2) return launch_norm_grad_u<T, W, VEC, 2, 2, kGradThreads>(p, units, sms, st);
  if (units <= u * most) return launch_norm_grad_u<T, W, VEC, u, 1, kGradThreads>(p, units, sms, st);
  constexpr int wide = kGradUnits<T, VEC, kGradWide>;
  if (units <= wide * most) return launch_norm_grad_u<T, W, VEC, wide, 1, kGradThreads>(p, units, sms, st);
  return launch_norm_grad_u<T, W, VEC, wide, 1, kGradWide>(p, units, sms, st);
}

template <typename T, typename W>
cudaError_t launch_norm_grad_t(NormGradParams& p, int sms, cudaStream_t st) {
  constexpr int n = kNormN<T, true>;
  const bool vec = p.cols % n == 0 && whole_rows(p.dy, p.lddy, n) && whole_rows(p.total, p.ldt, n) &&
                   whole_rows(p.weight, 0, n) && whole_rows(p.dx, p.lddx, n) &&
                   (p.past == nullptr || whole_rows(p.past, p.ldp, n));
  return vec ? launch_norm_grad_v<T, W, true>(p, sms, st) : launch_norm_grad_v<T, W, false>(p, sms, st);
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
