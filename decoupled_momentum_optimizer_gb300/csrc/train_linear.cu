// x w^T for a few rows of x (tokens being generated) and w in 8-bit floating point, block-scaled: one
// kernel that quantizes x, multiplies and scales, bound by reading w once.
//
// One CTA per SM streams its rows of w through shared memory: one thread keeps TMA loads of 16 rows x
// 4 blocks (8 KB, with their scales) under way, up to 128 KB of them, while sixteen warps first quantize
// all of x into shared memory (four lanes a block, 32 elements each; every SM repeats that, behind the
// first stages' arrival) and then multiply.  A group of four warps has a ring of stages of its own and
// owns 16 rows at a time, the instruction's 16 x 32 operand, each warp one of a stage's four blocks;
// the four join their sums in order.  The instruction's k order is free as long as both operands agree,
// so lane (g, c) takes 16 consecutive codes of row g at 16 c and at 64 + 16 c of a block, whole 16-byte
// reads of either operand.
//
// The block's 128 products accumulate in the instruction's float32, blocks in IEEE float32.
//
// Measured on the device with weights larger than L2 in turn: 8192 x 8192, one token 14.7 us (4.7 TB/s),
// 8192 x 2048 5.9 us, eight tokens 6.9 us; about 2.2 us of each is the launch.  Plain loads of w instead of
// TMA stages left HBM idle (10.1 us for 8192 x 2048), and quantizing x in every CTA of a larger grid cost
// up to 18 us more for eight tokens.
#include "train_common.cuh"
#include "train_tensor.cuh"

namespace demo {

namespace {

constexpr int kWarps = 16, kGroups = 4;
constexpr int kThreads = 32 * (kWarps + 1);  // + one that loads
constexpr int kQuad = 4;                     // blocks of a stage, one for each warp of a group
constexpr int kRows = 16;
constexpr int kStages = 16;

struct LinearShared {
  uint8_t w[kStages][kQuad][kRows][kBlock];  // 1024-byte aligned (swizzle atoms)
  float ws[kStages][kQuad][kRows];
  uint64_t full[kStages], empty[kStages];
  volatile uint32_t dead;
  uint32_t pad[3];  // the rest follows, 16-byte aligned
};
static_assert(sizeof(LinearShared) % 16 == 0 && sizeof(LinearShared) + 1024 + kLinearSmem <= 227 * 1024, "shared memory");

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

// 32 elements of a block of a token, every fourth unit of 16 bytes from unit c on; zero from `live` on.
template <typename T>
constexpr int kUnit = 16 / static_cast<int>(sizeof(T));
template <typename T>
constexpr int kUnits = 32 / kUnit<T>;

template <typename T, bool VEC>
__device__ __forceinline__ void load32(const T* block, int c, long long live, Vec<T, kUnit<T>> (&v)[kUnits<T>]) {
  constexpr int N = kUnit<T>;
#pragma unroll
  for (int j = 0; j < kUnits<T>; ++j) {
    const int at = (4 * j + c) * N;
    if (VEC && at + N <= live) {
      v[j] = *reinterpret_cast<const Vec<T, N>*>(block + at);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) v[j].e[e] = at + e < live ? block[at + e] : from_f32<T>(0.0f);
    }
  }
}

// The larger magnitude; a NaN stays.
__device__ __forceinline__ float max_magnitude(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// sum + d s u for two scales s and u.  Either one, or their product, can leave float32's range with d
// where d s u does not; so the sum of the two exponents is applied in two halves.  d times the first is
// exact unless d s u overflows or vanishes itself.
__device__ __forceinline__ float add_scaled(float sum, float d, float s, float u) {
  const uint32_t e = __float_as_uint(s) + __float_as_uint(u);  // exponents alone, 254 at most each
  const uint32_t half = (e >> 1) & 0x7f800000u;
  return fmaf(d * __uint_as_float(half), __uint_as_float(e - half), sum);
}

// Shared memory behind LinearShared: the warps' sums [warp][m][16 rows], x's codes [m][128 kb] (tokens
// of odd number have the halves of every block swapped, so that eight lanes of a 16-byte read reach
// different banks) and scales [m][kb].
template <typename T, bool VEC, int WFMT, int TILES>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t raw[];
  LinearShared& s = *reinterpret_cast<LinearShared*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  float* part = reinterpret_cast<float*>(&s + 1);
  uint8_t* codes = reinterpret_cast<uint8_t*>(part + kWarps * kRows * p.m);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int kp = p.kb * kBlock;
  float* scales = reinterpret_cast<float*>(codes + p.m * kp);
  // This CTA's rows of w, 16 at a time: row blocks blockIdx.x, + gridDim.x, ..; group j takes the j-th,
  // j + 4-th ..  The groups that have any share the stages evenly, each a ring of its own: whoever waits on
  // a stage's barrier has then seen its every phase (a wait by parity passes at once for the phase after
  // one that is still under way).  Stages are asked for in rounds of up to four row blocks, in turn.
  const int row_blocks = static_cast<int>((p.n + kRows - 1) / kRows);
  const int own = (row_blocks - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  const int quads = (p.kb + kQuad - 1) / kQuad;
  const int ring = kStages / (own < kGroups ? own : kGroups);  // stages of a group

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kQuad);
    }
    s.dead = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32 * kWarps && p.kb > 0) {
    prefetch_tmap(&p.w);
    prefetch_tmap(&p.ws);
  }
  __syncthreads();
  kernel_begin();

  if (warp == kWarps) {
    if (elect_one()) {
      bool ok = true;
      int at = 0;          // in every group's ring
      uint32_t phase = 0;
      uint32_t used = 0, last = 0;  // stages that have been asked for, and the phases they were last
      long long loads = 0;
      for (int first = 0; ok && first < own; first += kGroups) {
        const int live = own - first < kGroups ? own - first : kGroups;
        for (int q = 0; ok && q < quads; ++q) {
          for (int j = 0; j < live; ++j) {
            const int slot = j * ring + at;
            if (!(ok = wait_bounded<false>(&s.dead, &s.empty[slot], phase ^ 1u, p.fault))) break;
            const int row = static_cast<int>(blockIdx.x + (first + j) * gridDim.x) * kRows;
            mbar_expect_tx(&s.full[slot], kQuad * kRows * (kBlock + 4) + stall_extra(p.stall_at, blockIdx.x, loads++));
            tma_load_3d(s.w[slot], &p.w, &s.full[slot], 0, row, kQuad * q);
            tma_load_2d(s.ws[slot], &p.ws, &s.full[slot], row, kQuad * q);
            used |= 1u << slot;
            last = (last & ~(1u << slot)) | phase << slot;
          }
          if (++at == ring) {
            at = 0;
            phase ^= 1u;
          }
        }
      }
      // No copy may be under way when the CTA ends, and whoever waits for the last ones may give up: wait
      // (bounded) here too.
      for (int i = 0; i < kStages; ++i)
        if (used >> i & 1u) mbar_wait_bounded(&s.full[i], last >> i & 1u);
    }
  } else {
    // ---- x: a warp quantizes eight blocks of 128 at a time, four lanes each, 32 elements a lane ----
    const int blocks = p.m * p.kb, c4 = lane & 3;
    for (int first = 8 * warp; first < blocks; first += 8 * kWarps) {
      const int i = first + (lane >> 2) < blocks ? first + (lane >> 2) : blocks - 1;  // block kb of token m
      const int m = i / p.kb, kb = i - m * p.kb;
      Vec<T, kUnit<T>> v[kUnits<T>];
      load32<T, VEC>(static_cast<const T*>(p.x) + m * p.ldx + static_cast<long long>(kb) * kBlock, c4,
                     p.k - static_cast<long long>(kb) * kBlock, v);
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < kUnits<T>; ++j)
#pragma unroll
        for (int e = 0; e < kUnit<T>; ++e) top = max_magnitude(top, to_f32(v[j].e[e]));
      if (!(top <= 3.402823466e38f)) {  // an infinity or a NaN: the others' maximum
        top = 0.0f;
#pragma unroll
        for (int j = 0; j < kUnits<T>; ++j)
#pragma unroll
          for (int e = 0; e < kUnit<T>; ++e) {
            const float f = finite_or_nan(to_f32(v[j].e[e]));
            v[j].e[e] = from_f32<T>(f);
            top = fmaxf(top, fabsf(f));
          }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = scale_exponent(__float_as_uint(top), fmt_top(kE4M3));
      const float inv = pow2f(-ex);
      uint8_t* dst = codes + i * kBlock;
      const int flip = (m & 1) << 6;
#pragma unroll
      for (int j = 0; j < kUnits<T>; ++j) {
        const int at = ((4 * j + c4) * kUnit<T>) ^ flip;
#pragma unroll
        for (int e = 0; e < kUnit<T>; e += 4)
          *reinterpret_cast<uint32_t*>(dst + at + e) =
              codes4<kE4M3>(to_f32(v[j].e[e]) * inv, to_f32(v[j].e[e + 1]) * inv, to_f32(v[j].e[e + 2]) * inv,
                            to_f32(v[j].e[e + 3]) * inv);
      }
      if (c4 == 0) scales[i] = pow2f(ex);
    }
    named_sync(1, 32 * kWarps);

    // ---- products ----
    const int group = warp >> 2, w4 = warp & 3, g = lane >> 2, c = lane & 3;
    bool ok = true;
    int at = 0;
    uint32_t phase = 0;
    for (int first = 0; ok && first + group < own; first += kGroups) {
      float sum[TILES][4];
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[t][e] = 0.0f;
      for (int q = 0; q < quads; ++q) {
        const int slot = group * ring + at, kb = kQuad * q + w4;
        ok = __all_sync(0xffffffffu, wait_bounded<false>(&s.dead, &s.full[slot], phase, p.fault));
        if (!ok) break;
        // unit u of row r is at u ^ (r & 7)
        const uint8_t* w0 = s.w[slot][w4][g];
        const uint8_t* w1 = s.w[slot][w4][g + 8];
        const uint4 x00 = *reinterpret_cast<const uint4*>(w0 + ((c ^ g) << 4));
        const uint4 x01 = *reinterpret_cast<const uint4*>(w0 + (((c + 4) ^ g) << 4));
        const uint4 x10 = *reinterpret_cast<const uint4*>(w1 + ((c ^ g) << 4));
        const uint4 x11 = *reinterpret_cast<const uint4*>(w1 + (((c + 4) ^ g) << 4));
        const float s0 = s.ws[slot][w4][g], s1 = s.ws[slot][w4][g + 8];
        // what the products' sums start from: NaN under a scale that is no power of two
        const float nan = __uint_as_float(0x7fc00000u);
        const float z0 = scale_byte(s0) == kScaleNaN ? nan : 0.0f, z1 = scale_byte(s1) == kScaleNaN ? nan : 0.0f;
        if (kb < p.kb) {
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            const int m = 8 * t + g, m0 = 8 * t + 2 * c;
            uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
            if (m < p.m) {
              const uint8_t* x = codes + m * kp + kb * kBlock + 16 * c;
              b0 = *reinterpret_cast<const uint4*>(x + ((g & 1) << 6));
              b1 = *reinterpret_cast<const uint4*>(x + ((~g & 1) << 6));
            }
            // this lane's results are rows g, g + 8 and tokens 2 c, 2 c + 1
            const float u0 = m0 < p.m ? scales[m0 * p.kb + kb] : 0.0f;
            const float u1 = m0 + 1 < p.m ? scales[(m0 + 1) * p.kb + kb] : 0.0f;
            float d[4] = {z0, z0, z1, z1};
            mma_f8<WFMT>(d, x00.x, x10.x, x00.y, x10.y, b0.x, b0.y);
            mma_f8<WFMT>(d, x00.z, x10.z, x00.w, x10.w, b0.z, b0.w);
            mma_f8<WFMT>(d, x01.x, x11.x, x01.y, x11.y, b1.x, b1.y);
            mma_f8<WFMT>(d, x01.z, x11.z, x01.w, x11.w, b1.z, b1.w);
            sum[t][0] = add_scaled(sum[t][0], d[0], s0, u0);
            sum[t][1] = add_scaled(sum[t][1], d[1], s0, u1);
            sum[t][2] = add_scaled(sum[t][2], d[2], s1, u0);
            sum[t][3] = add_scaled(sum[t][3], d[3], s1, u1);
          }
        }
        __syncwarp();
        if (lane == 0) arrive_here(&s.empty[slot]);
        if (++at == ring) {
          at = 0;
          phase ^= 1u;
        }
      }
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const int m = 8 * t + 2 * c;
        float* q = part + (warp * p.m + m) * kRows + g;
        if (m < p.m) {
          q[0] = sum[t][0];
          q[8] = sum[t][2];
        }
        if (m + 1 < p.m) {
          q[kRows] = sum[t][1];
          q[kRows + 8] = sum[t][3];
        }
      }
      // The group goes on or stops as one: a warp that gave up must not leave the others at a barrier, and
      // they may have found the stage it gave up on complete.
      ok = named_all(2 + group, 32 * kQuad, ok);
      const long long n0 = static_cast<long long>(blockIdx.x + static_cast<long long>(first + group) * gridDim.x) * kRows;
      for (int i = 32 * w4 + lane; ok && i < p.m * kRows; i += 32 * kQuad) {
        const int m = i / kRows, r = i % kRows;
        const long long n = n0 + r;
        if (n >= p.n) continue;
        const float* q = part + 4 * group * kRows * p.m + i;
        float v = q[0];
#pragma unroll
        for (int j = 1; j < kQuad; ++j) v += q[j * kRows * p.m];
        const long long at = m * p.ldo + n;
        if (p.out_dtype == kF32)
          static_cast<float*>(p.out)[at] = v;
        else if (p.out_dtype == kBF16)
          static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
        else
          static_cast<__half*>(p.out)[at] = __float2half_rn(v);
      }
      named_sync(2 + group, 32 * kQuad);  // the sums are read before the next rows' are written
    }
  }
}

template <typename T, bool VEC, int WFMT>
auto* pick_tiles(int m) {
  return m <= 8    ? linear_kernel<T, VEC, WFMT, 1>
         : m <= 16 ? linear_kernel<T, VEC, WFMT, 2>
         : m <= 32 ? linear_kernel<T, VEC, WFMT, 4>
                   : linear_kernel<T, VEC, WFMT, 5>;
}
template <typename T, bool VEC>
auto* pick_format(int w_fmt, int m) {
  return w_fmt == kE4M3 ? pick_tiles<T, VEC, kE4M3>(m) : pick_tiles<T, VEC, kE5M2>(m);
}
template <typename T>
auto* pick_vec(bool vec, int w_fmt, int m) {
  return vec ? pick_format<T, true>(w_fmt, m) : pick_format<T, false>(w_fmt, m);
}
auto* pick(int dtype, bool vec, int w_fmt, int m) {
  return dtype == kF32    ? pick_vec<float>(vec, w_fmt, m)
         : dtype == kBF16 ? pick_vec<__nv_bfloat16>(vec, w_fmt, m)
                          : pick_vec<__half>(vec, w_fmt, m);
}

}  // namespace

cudaError_t launch_linear(const LinearParams& p, int dtype, int w_fmt, int sms, cudaStream_t st) {
  const size_t size = dtype == kF32 ? 4 : 2;
  // 16-byte units of x: every row starts on one
  const bool vec = (reinterpret_cast<uintptr_t>(p.x) & 15) == 0 &&
                   (p.m == 1 || static_cast<size_t>(p.ldx) * size % 16 == 0);
  const long long row_blocks = (p.n + kRows - 1) / kRows;
  const size_t smem = sizeof(LinearShared) + 1024 + static_cast<size_t>(linear_bytes(p.m, p.kb));
  return launch_overlapped(pick(dtype, vec, w_fmt, p.m), static_cast<unsigned>(row_blocks < sms ? row_blocks : sms),
                           kThreads, smem, st, p);
}

cudaError_t prepare_linear_kernels() {
  for (int dtype : {kF32, kBF16, kF16})
    for (int i = 0; i < 16; ++i) {
      const cudaError_t e =
          cudaFuncSetAttribute(pick(dtype, i & 1, i & 2 ? kE5M2 : kE4M3, 8 << (i >> 2)),
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(sizeof(LinearShared) + 1024 + kLinearSmem));
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace demo
