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
constexpr int kThreads = 32 * (kPromoteWarps + 2);  // + one warp that loads, one that multiplies
constexpr uint32_t kTmemCols = 2 * kBN;
constexpr uint32_t kABytes = kBM * kBlock, kBBytes = kBN * kBlock;

struct Shared {
  uint8_t a[kStages][kABytes];  // 1024-byte aligned (swizzle atoms)
  uint8_t b[kStages][kBBytes];
  float sa[kScaleSlots][kBM];
  float sb[kScaleSlots][kBN];
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
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0u) {
      if (s.dead) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
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

__device__ __forceinline__ Tile tile_at(long long t, int tiles_m) {
  return Tile{static_cast<int>(t % tiles_m) * kBM, static_cast<int>(t / tiles_m) * kBN};
}

__device__ __forceinline__ void store_one(const MatmulParams& p, long long m, long long n, float v) {
  const long long i = m * p.ldo + n;
  if (p.out_dtype == kF32) {
    float* o = static_cast<float*>(p.out) + i;
    *o = p.add ? *o + v : v;
  } else if (p.out_dtype == kBF16) {
    static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
  } else {
    static_cast<__half*>(p.out)[i] = __float2half_rn(v);
  }
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1) matmul_kernel(const __grid_constant__ MatmulParams p) {
  extern __shared__ uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_m = static_cast<int>((p.m + kBM - 1) / kBM);
  const long long tiles = static_cast<long long>(tiles_m) * ((p.n + kBN - 1) / kBN);

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

  if (warp == kPromoteWarps) {
    // ---- loads ----
    if (lane == 0) {
      const long long lda = (p.m + 3) / 4 * 4, ldb = (p.n + 3) / 4 * 4;  // strides of the scales
      Ring<kStages> st;
      Ring<kScaleSlots> sc;
      uint32_t used = 0;  // stages that have been loaded at least once
      bool ok = true;
      for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile tl = tile_at(t, tiles_m);
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
  } else if (warp == kPromoteWarps + 1) {
    // ---- tensor-core instructions ----
    if (lane == 0) {
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
    // ---- scales and float32 sums: warp w holds rows 32 (w & 3) .., columns 128 (w >> 2) .. ----
    const int row = 32 * (warp & 3) + lane;
    const int col0 = kBN / 2 * (warp >> 2);
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + col0;
    Ring<kScaleSlots> sc;
    Ring<2> acc;
    bool ok = true;
    for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const Tile tl = tile_at(t, tiles_m);
      float sum[kBN / 2];
#pragma unroll
      for (int i = 0; i < kBN / 2; ++i) sum[i] = 0.0f;
      for (int kb = 0; kb < p.kb; ++kb) {
        // every lane waits (each reads what the barrier guards); the warp goes on or stops as one
        if (!(ok = __all_sync(0xffffffffu, wait_or_dead(s, &s.sfull[sc.slot], sc.phase, p.fault)))) break;
        const float sa = s.sa[sc.slot][row];
        if (!(ok = __all_sync(0xffffffffu, wait_or_dead(s, &s.tfull[acc.slot], acc.phase, p.fault)))) break;
        tensor_fence_after();
#pragma unroll
        for (int c = 0; c < kBN / 2; c += 32) {
          uint32_t v[32];
          tmem_load32(taddr + acc.slot * kBN + c, v);
          tensor_wait_load(v);
          const float4* sb = reinterpret_cast<const float4*>(&s.sb[sc.slot][col0 + c]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 q = sb[j];
            sum[c + 4 * j + 0] = fmaf(__uint_as_float(v[4 * j + 0]) * q.x, sa, sum[c + 4 * j + 0]);
            sum[c + 4 * j + 1] = fmaf(__uint_as_float(v[4 * j + 1]) * q.y, sa, sum[c + 4 * j + 1]);
            sum[c + 4 * j + 2] = fmaf(__uint_as_float(v[4 * j + 2]) * q.z, sa, sum[c + 4 * j + 2]);
            sum[c + 4 * j + 3] = fmaf(__uint_as_float(v[4 * j + 3]) * q.w, sa, sum[c + 4 * j + 3]);
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
      const long long m = tl.m0 + row;
      if (m < p.m) {
#pragma unroll
        for (int i = 0; i < kBN / 2; ++i) {
          const long long n = tl.n0 + col0 + i;
          if (n < p.n) store_one(p, m, n, sum[i]);
        }
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
  matmul_kernel<<<static_cast<unsigned>(tiles < sms ? tiles : sms), kThreads, kSmem, st>>>(p);
  return cudaGetLastError();
}

cudaError_t prepare_matmul_kernels() {
  return cudaFuncSetAttribute(matmul_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
}

}  // namespace demo
