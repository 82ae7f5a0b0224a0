// Product of two matrices in 8-bit floating point with a scale for each block of 128 along k:
//
//   out[m][n] (+)= sum over blocks b of sa[b][m] sb[b][n] * (sum over k in block b of a[m][k] b[n][k])
//
// A CTA computes a 128 x 256 tile.  TMA brings 128 codes of k of both operands into a ring of
// shared-memory stages; one thread issues four K = 32 tensor-core instructions per block into one
// of two halves of tensor memory; eight warps meanwhile read the other half, apply the block's
// scales and add it to float32 accumulators in registers.  So every sum that passes a block is an
// IEEE float32 multiply-add, and the tensor core's own accumulator only ever holds 128 products.
// Scales travel through a ring of their own, so that a stage of codes is free as soon as the tensor
// core has read it.
#include "train_common.cuh"
#include "train_tensor.cuh"

namespace demo {

namespace {

constexpr int kBM = 128, kBN = 256;
constexpr int kStages = 4, kScaleSlots = 8;
constexpr int kPromoteWarps = 8;
// Two groups of four warps that add up, and one whose first two warps load and multiply.  Launched
// with 168 registers a thread; the last group gives up what the others' accumulators need:
// 256 * 216 + 128 * 72 = 384 * 168.
constexpr int kThreads = 32 * (kPromoteWarps + 4);
constexpr int kPromoteRegs = 216, kFeedRegs = 72;
static_assert(256 * kPromoteRegs + 128 * kFeedRegs == kThreads * 168, "the launch's registers");
constexpr uint32_t kTmemCols = 2 * kBN;
constexpr uint32_t kABytes = kBM * kBlock, kBBytes = kBN * kBlock;

struct Shared {
  uint8_t a[kStages][kABytes];  // 1024-byte aligned (swizzle atoms)
  uint8_t b[kStages][kBBytes];
  float sa[kScaleSlots][kBM];
  float sb[kScaleSlots][kBN];
  uint4 out[kPromoteWarps][128];  // a warp's 32 rows x 64 bytes on their way out
  uint64_t full[kStages], empty[kStages];
  uint64_t sfull[kScaleSlots], sempty[kScaleSlots];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem;
  volatile uint32_t dead;  // a wait gave up: everyone stops
};
constexpr size_t kSmem = sizeof(Shared) + 1024;

// Phase `parity` of `bar`, or false once any wait of the CTA has given up.
__device__ __forceinline__ bool wait_or_dead(Shared& s, uint64_t* bar, uint32_t parity, unsigned int* fault) {
  uint64_t t0 = 0;  // read late: the timer itself is slow to read, and most waits are short
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 0u) {
      if (s.dead) return false;
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        s.dead = 1;
        atomicOr(fault, kFaultLoadTimeout);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// A position in a ring of N slots: the slot, and the parity of its current phase.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

struct Tile {
  int m0, n0;
};

// Tiles in bands of 16 along m, along n within a band: the tiles that run at one time then cover
// about as many rows of a as of b, and share both in the L2 cache.
constexpr int kBand = 16;
__device__ __forceinline__ Tile tile_at(long long t, int tiles_m, int tiles_n) {
  const long long per = static_cast<long long>(kBand) * tiles_n;
  const int band = static_cast<int>(t / per), i = static_cast<int>(t - band * per);
  const int height = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
  return Tile{(band * kBand + i % height) * kBM, i / height * kBN};
}

// Units of 16 bytes of a result row: E elements, converted from float32.
template <typename T>
__device__ __forceinline__ uint4 to_unit(const float* v) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  } else {
    Vec<T, 8> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.e[e] = from_f32<T>(v[e]);
    return *reinterpret_cast<uint4*>(&o);
  }
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// A warp's 32 rows (lane l holds row l) x 128 columns to out[m0 ..][n0 ..], 64 bytes of every row at
// a time through 2 KB of shared memory: written a row per lane, read back as 8 rows x 4 units, so
// that every store covers whole 32-byte sectors.  Unit u of row r is stored at u ^ ((r >> 1) & 3):
// two rows span the banks once, so eight lanes of either access reach different ones.
template <typename T, bool ADD>
__device__ __forceinline__ void store_rows(uint4* buf, int lane, const uint64_t (&sum)[64], const MatmulParams& p,
                                           long long m0, long long n0) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const bool vec = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && p.ldo % E == 0;
#pragma unroll
  for (int c = 0; c < 128; c += 4 * E) {
    if (n0 + c >= p.n) break;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 q = unpack2(sum[(c + u * E + e) / 2]);
        v[e] = q.x;
        v[e + 1] = q.y;
      }
      buf[lane * 4 + (u ^ ((lane >> 1) & 3))] = to_unit<T>(v);
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 8 * q + (lane >> 2), u = lane & 3;
      uint4 w = buf[r * 4 + (u ^ ((r >> 1) & 3))];
      const long long m = m0 + r, n = n0 + c + u * E;
      if (m < p.m && n < p.n) {
        T* o = static_cast<T*>(p.out) + m * p.ldo + n;
        if (vec && n + E <= p.n) {
          if constexpr (ADD) {
            const float4 s = add4(*reinterpret_cast<const float4*>(o), *reinterpret_cast<const float4*>(&w));
            w = *reinterpret_cast<const uint4*>(&s);
          }
          *reinterpret_cast<uint4*>(o) = w;
        } else {
          const T* x = reinterpret_cast<const T*>(&w);
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (n + e < p.n) o[e] = ADD ? from_f32<T>(to_f32(o[e]) + to_f32(x[e])) : x[e];
        }
      }
    }
    __syncwarp();
  }
}

}  // namespace

// TILES: b's scales are equal within each 128 rows, that is for all columns of a promoting warp.
template <bool TILES>
__global__ void __launch_bounds__(kThreads, 1) matmul_kernel(const __grid_constant__ MatmulParams p) {
  extern __shared__ uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_m = static_cast<int>((p.m + kBM - 1) / kBM);
  const int tiles_n = static_cast<int>((p.n + kBN - 1) / kBN);
  const long long tiles = static_cast<long long>(tiles_m) * tiles_n;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(&s.sfull[i], 1);
      mbar_init(&s.sempty[i], kPromoteWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], kPromoteWarps);
    }
    mbar_init(&s.drain, 1);
    s.dead = 0;
    fence_mbar_init();
  }
  if (warp == kPromoteWarps + 1) tmem_alloc(&s.tmem, kTmemCols);
  tensor_fence_before();
  __syncthreads();
  tensor_fence_after();
  const uint32_t tmem = s.tmem;
  const uint32_t idesc = f8_instruction(p.a_fmt, p.b_fmt, kBM, kBN);

  if (warp >= kPromoteWarps) {
    registers_down<kFeedRegs>();
    if (warp == kPromoteWarps && lane == 0) {
      // ---- loads ----
      const long long lda = (p.m + 3) / 4 * 4, ldb = (p.n + 3) / 4 * 4;  // strides of the scales
      Ring<kStages> st;
      Ring<kScaleSlots> sc;
      uint32_t used = 0;  // stages that have been loaded at least once
      bool ok = true;
      for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile tl = tile_at(t, tiles_m, tiles_n);
        const uint32_t na = static_cast<uint32_t>(lda - tl.m0 < kBM ? lda - tl.m0 : kBM) * 4;
        const uint32_t nb = static_cast<uint32_t>(ldb - tl.n0 < kBN ? ldb - tl.n0 : kBN) * 4;
        for (int kb = 0; kb < p.kb; ++kb) {
          if (!(ok = wait_or_dead(s, &s.empty[st.slot], st.phase ^ 1u, p.fault))) break;
          mbar_expect_tx(&s.full[st.slot], kABytes + kBBytes);
          tma_load_2d(s.a[st.slot], &p.a, &s.full[st.slot], kb * kBlock, tl.m0);
          tma_load_2d(s.b[st.slot], &p.b, &s.full[st.slot], kb * kBlock, tl.n0);
          used |= 1u << st.slot;
          st.next();
          if (!(ok = wait_or_dead(s, &s.sempty[sc.slot], sc.phase ^ 1u, p.fault))) break;
          mbar_expect_tx(&s.sfull[sc.slot], na + nb);
          bulk_load(s.sa[sc.slot], p.a_scales + kb * lda + tl.m0, na, &s.sfull[sc.slot]);
          bulk_load(s.sb[sc.slot], p.b_scales + kb * ldb + tl.n0, nb, &s.sfull[sc.slot]);
          used |= 1u << (kStages + sc.slot);
          sc.next();
        }
      }
      // Stopped early: copies may be in flight into this CTA's shared memory.  Wait (bounded) for
      // the last load of every slot: the slots before the ring's position are in its current phase,
      // the others in the one before.
      if (!ok) {
        for (int i = 0; i < kStages; ++i)
          if (used >> i & 1u) mbar_wait_bounded(&s.full[i], i < st.slot ? st.phase : st.phase ^ 1u);
        for (int i = 0; i < kScaleSlots; ++i)
          if (used >> (kStages + i) & 1u) mbar_wait_bounded(&s.sfull[i], i < sc.slot ? sc.phase : sc.phase ^ 1u);
      }
    }
    if (warp == kPromoteWarps + 1 && lane == 0) {
      // ---- tensor-core instructions ----
      Ring<kStages> st;
      Ring<2> acc;
      bool ok = true;
      for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        for (int kb = 0; kb < p.kb; ++kb) {
          if (!(ok = wait_or_dead(s, &s.tempty[acc.slot], acc.phase ^ 1u, p.fault))) break;
          if (!(ok = wait_or_dead(s, &s.full[st.slot], st.phase, p.fault))) break;
          tensor_fence_after();
          const uint64_t da = operand_desc(smem_addr(s.a[st.slot])), db = operand_desc(smem_addr(s.b[st.slot]));
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k)  // 32 bytes along the swizzled row: 2 units of 16
            tensor_mma_f8(tmem + acc.slot * kBN, da + 2 * k, db + 2 * k, idesc, k > 0);
          tensor_commit(&s.empty[st.slot]);
          tensor_commit(&s.tfull[acc.slot]);
          st.next();
          acc.next();
        }
      }
    }
  } else {
    registers_up<kPromoteRegs>();
    // ---- scales and float32 sums: warp w holds rows 32 (w & 3) .., columns 128 (w >> 2) .. ----
    const int row = 32 * (warp & 3) + lane;
    const int col0 = kBN / 2 * (warp >> 2);
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + col0;
    Ring<kScaleSlots> sc;
    Ring<2> acc;
    bool ok = true;
    for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const Tile tl = tile_at(t, tiles_m, tiles_n);
      uint64_t sum[kBN / 4];  // pairs of columns
#pragma unroll
      for (int i = 0; i < kBN / 4; ++i) sum[i] = 0;
      for (int kb = 0; kb < p.kb; ++kb) {
        // every lane waits (each reads what the barrier guards); the warp goes on or stops as one
        if (!(ok = __all_sync(0xffffffffu, wait_or_dead(s, &s.sfull[sc.slot], sc.phase, p.fault)))) break;
        const float scale = TILES ? s.sa[sc.slot][row] * s.sb[sc.slot][col0] : s.sa[sc.slot][row];
        const uint64_t scale2 = pack2(scale, scale);
        if (!(ok = __all_sync(0xffffffffu, wait_or_dead(s, &s.tfull[acc.slot], acc.phase, p.fault)))) break;
        tensor_fence_after();
#pragma unroll
        for (int c = 0; c < kBN / 2; c += 32) {
          uint32_t v[32];
          tmem_load32(taddr + acc.slot * kBN + c, v);
          tensor_wait_load(v);
          if constexpr (TILES) {
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[c / 2 + j] = fma2(pack2(v[2 * j], v[2 * j + 1]), scale2, sum[c / 2 + j]);
          } else {
            const ulonglong2* sb = reinterpret_cast<const ulonglong2*>(&s.sb[sc.slot][col0 + c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const ulonglong2 q = sb[j];
              sum[c / 2 + 2 * j] = fma2(mul2(pack2(v[4 * j], v[4 * j + 1]), q.x), scale2, sum[c / 2 + 2 * j]);
              sum[c / 2 + 2 * j + 1] =
                  fma2(mul2(pack2(v[4 * j + 2], v[4 * j + 3]), q.y), scale2, sum[c / 2 + 2 * j + 1]);
            }
          }
        }
        tensor_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.tempty[acc.slot]);
          mbar_arrive(&s.sempty[sc.slot]);
        }
        sc.next();
        acc.next();
      }
      if (!ok) break;
      const long long m0 = tl.m0 + 32 * (warp & 3), n0 = tl.n0 + col0;
      if (m0 < p.m && n0 < p.n) {
        uint4* buf = s.out[warp];
        if (p.out_dtype == kBF16)
          store_rows<__nv_bfloat16, false>(buf, lane, sum, p, m0, n0);
        else if (p.out_dtype == kF16)
          store_rows<__half, false>(buf, lane, sum, p, m0, n0);
        else if (p.add)
          store_rows<float, true>(buf, lane, sum, p, m0, n0);
        else
          store_rows<float, false>(buf, lane, sum, p, m0, n0);
      }
    }
  }
  tensor_fence_before();
  __syncthreads();
  if (warp == kPromoteWarps + 1) {
    // A CTA that stopped early may have matrix instructions in flight: wait (bounded) for them.
    if (s.dead && lane == 0) {
      tensor_commit(&s.drain);
      mbar_wait_bounded(&s.drain, 0);
    }
    __syncwarp();
    tensor_fence_after();
    tmem_free(tmem, kTmemCols);
  }
}

cudaError_t launch_matmul(const MatmulParams& p, int sms, cudaStream_t st) {
  const long long tiles = ((p.m + kBM - 1) / kBM) * ((p.n + kBN - 1) / kBN);
  const unsigned grid = static_cast<unsigned>(tiles < sms ? tiles : sms);
  if (p.b_tiles)
    matmul_kernel<true><<<grid, kThreads, kSmem, st>>>(p);
  else
    matmul_kernel<false><<<grid, kThreads, kSmem, st>>>(p);
  return cudaGetLastError();
}

cudaError_t prepare_matmul_kernels() {
  const cudaError_t e = cudaFuncSetAttribute(matmul_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(matmul_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kSmem));
}

}  // namespace demo
