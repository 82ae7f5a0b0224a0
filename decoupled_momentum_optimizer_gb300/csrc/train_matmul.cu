// Product of two matrices in 8-bit floating point with a power-of-two scale for each block of 128
// along k:
//
//   out[m][n] (+)= sum over blocks b of sa[b][m] sb[b][n] * (sum over k in block b of a[m][k] b[n][k])
//
// A CTA computes a 128 x 224 tile.  TMA brings 128 codes of k of both operands into a ring of
// shared-memory stages; four warps pack the scales of four blocks into a 32-bit word per row (UE8M0
// bytes), which the tensor core copies to tensor memory; one thread issues four K = 32 block-scaled
// tensor-core instructions per block.  Four blocks run into one of two halves of tensor memory, and eight warps meanwhile add the other half to float32 sums in
// registers, so the tensor core's accumulator holds 512 products at most and every longer sum is an
// IEEE float32 addition: its own additions drop low bits, and over a whole k of thousands that
// showed.  (Scales in the instruction instead of in the sums: with a multiply-add per element and
// block in the eight warps, 8192 x 2048 x 8192 took 170 us, and 250 us with a scale per row of b.)
// 224 columns leave room in tensor memory for two halves and their scales.
#include "train_common.cuh"
#include "train_tensor.cuh"

namespace demo {

namespace {

constexpr int kBM = 128, kBN = 224;
constexpr int kChain = 4;  // blocks of 128 that one half of tensor memory sums
constexpr int kSumWarps = 8, kScaleWarps = 4;
constexpr int kLoadWarp = kSumWarps + kScaleWarps, kMmaWarp = kLoadWarp + 1, kScaleLoadWarp = kLoadWarp + 2;
// Whole groups of four warps, launched with 128 registers a thread: the summing ones take 192, the
// others keep 64.
constexpr int kThreads = 512;
constexpr int kSumRegs = 192, kFeedRegs = 64;
static_assert(256 * kSumRegs + 256 * kFeedRegs == kThreads * 128, "the launch's registers");
constexpr uint32_t kTmemCols = 512;
// Scale words of a half: 4 columns of a's (one for 32 rows) and 8 of b's (7 used).
constexpr uint32_t kScaleCol = 2 * kBN, kScaleCols = 12;
static_assert(kScaleCol + 2 * kScaleCols <= kTmemCols, "tensor memory");
constexpr int kScaleSlots = kScaleWarps;  // chains whose words are ready in shared memory
static_assert(kChain == 4, "a word holds the scales of a chain");
constexpr int kCols = kBN / 2;  // columns of a summing warp

// G CTAs (1, or a cluster of 2) share a tile of G * 128 x 224: each loads its 128 rows of a and
// 224 / G of b, and the rest of the shared memory is stages.
template <int G>
struct Shared {
  static constexpr int kStages = G == 1 ? 4 : 6;
  static constexpr uint32_t kABytes = kBM * kBlock, kBBytes = kBN / G * kBlock;
  uint8_t a[kStages][kABytes];  // 1024-byte aligned (swizzle atoms)
  uint8_t b[kStages][kBBytes];
  uint4 out[kSumWarps][128];  // a warp's 32 rows x 64 bytes on their way out
  // Scale words: row 32 c + l of an operand at [l][c] of its 512-byte unit of 128 rows (a's, then
  // b's two), as the tensor core's copy wants them.
  uint32_t words[kScaleSlots][3][32][4];
  // a chain's scales as they arrive
  float sa[kScaleSlots][kChain][kBM];
  float sb[kScaleSlots][kChain][kBN];
  uint64_t full[kStages], empty[kStages];
  uint64_t sfull[kScaleSlots], sempty[kScaleSlots];  // scales
  uint64_t scaled[kScaleSlots], sfree[kScaleSlots];  // words
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem;
  volatile uint32_t dead;  // a wait gave up: everyone stops
};
template <int G>
constexpr size_t kSmem = sizeof(Shared<G>) + 1024;
static_assert(kSmem<1> <= 227 * 1024 && kSmem<2> <= 227 * 1024, "shared memory");

// Phase `parity` of `bar`, or false once any wait of the CTA has given up.
template <int G>
__device__ __forceinline__ bool wait_or_dead(Shared<G>& s, uint64_t* bar, uint32_t parity, unsigned int* fault) {
  uint64_t t0 = 0;  // read late: the timer itself is slow to read, and most waits are short
  for (uint32_t it = 1;; ++it) {
    if (G == 1 ? mbar_try_wait(bar, parity) : mbar_try_wait_cluster(bar, parity)) return true;
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

__device__ __forceinline__ void arrive_here(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// An arrival on the barrier of the CTA whose thread issues the matrix instructions.  RELEASE: it
// publishes writes to shared memory; reads of tensor memory are ordered by the tensor-core fences
// alone, and a release to the cluster would hold the warp up.
template <int G, bool RELEASE>
__device__ __forceinline__ void arrive_at_issuer(uint64_t* bar) {
  if constexpr (G == 1)
    arrive_here(bar);
  else
    mbar_arrive_at<RELEASE>(bar, 0);
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

// Tiles in bands of 2048 rows of m, along n within a band: the tiles that run at one time then cover
// about as many rows of a as of b, and share both in the L2 cache.  m0 is the CTA's own first row.
template <int G>
__device__ __forceinline__ Tile tile_at(int t, int tiles_m, int tiles_n, int rank) {
  constexpr int kBand = 16 / G;
  const int per = kBand * tiles_n;
  const int band = t / per, i = t - band * per;
  const int height = tiles_m - band * kBand < kBand ? tiles_m - band * kBand : kBand;
  const int col = i / height;
  return Tile{((band * kBand + i - col * height) * G + rank) * kBM, col * kBN};
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

// A warp's 32 rows (lane l holds row l) x kCols columns to out[m0 ..][n0 ..], 64 bytes of every row at
// a time through 2 KB of shared memory: written a row per lane, read back as 8 rows x 4 units, so
// that every store covers whole 32-byte sectors.  Unit u of row r is stored at u ^ ((r >> 1) & 3):
// two rows span the banks once, so eight lanes of either access reach different ones.
template <typename T, bool ADD>
__device__ __forceinline__ void store_rows(uint4* buf, int lane, const uint64_t (&sum)[kCols / 2],
                                           const MatmulParams& p, long long m0, long long n0) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const bool vec = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && p.ldo % E == 0;
#pragma unroll
  for (int c = 0; c < kCols; c += 4 * E) {
    if (n0 + c >= p.n) break;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (c + u * E >= kCols) break;
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
      if (m < p.m && n < p.n && c + u * E < kCols) {
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

// A CTA's chains (up to kChain blocks of a tile) in order, tile after tile.
struct Chains {
  int t, tiles, stride;
  int c = 0, per_tile;
  __device__ __forceinline__ Chains(int first, int n, int step, int kb)
      : t(kb > 0 ? first : n), tiles(n), stride(step), per_tile((kb + kChain - 1) / kChain) {}
  __device__ __forceinline__ bool more() const { return t < tiles; }
  __device__ __forceinline__ void next(int by = 1) {
    for (c += by; c >= per_tile && t < tiles; c -= per_tile) t += stride;
  }
};

// Up to 128 rows' scales of a chain (LD floats from block to block) as exponent bytes: word i is row
// 32 i + lane's.
template <int ROWS, int LD>
__device__ __forceinline__ uint4 scale_words(const float* v, int lane) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < ROWS / 32; ++i)
#pragma unroll
    for (int j = 0; j < kChain; ++j)
      w[i] |= ((__float_as_uint(v[j * LD + 32 * i + lane]) >> 23) & 0xffu) << (8 * j);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1) matmul_kernel(const __grid_constant__ MatmulParams p) {
  extern __shared__ uint8_t raw[];
  using S = Shared<G>;
  constexpr int kStages = S::kStages;
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  // the warp's number from one lane: the roles below are branches of whole warps
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = G == 1 ? 0 : static_cast<int>(cluster_rank());
  const int tiles_m = static_cast<int>((p.m + G * kBM - 1) / (G * kBM));
  const int tiles_n = static_cast<int>((p.n + kBN - 1) / kBN);
  const int tiles = tiles_m * tiles_n;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(&s.scaled[i], G);
      mbar_init(&s.sfree[i], 1);
      mbar_init(&s.sfull[i], 1);
      mbar_init(&s.sempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], G * kSumWarps);
    }
    mbar_init(&s.drain, 1);
    s.dead = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc<G>(&s.tmem, kTmemCols);
  tensor_fence_before();
  __syncthreads();
  if constexpr (G > 1) cluster_sync();  // the other CTA's barriers are there
  tensor_fence_after();
  const uint32_t tmem = s.tmem;

  if (warp >= kSumWarps) {
    registers_down<kFeedRegs>();
    if (warp < kLoadWarp) {
      // ---- scale words: warp w makes those of every fourth chain, in slot w ----
      const int w = warp - kSumWarps;
      Chains in(blockIdx.x / G, tiles, gridDim.x / G, p.kb);
      uint32_t phase = 0;
      for (in.next(w); in.more(); in.next(kScaleWarps)) {
        if (!__all_sync(0xffffffffu, wait_or_dead(s, &s.sfull[w], phase, p.fault))) break;
        const uint4 wa = scale_words<128, kBM>(s.sa[w][0], lane), wb = scale_words<128, kBN>(s.sb[w][0], lane),
                    wc = scale_words<kBN - 128, kBN>(s.sb[w][0] + 128, lane);
        __syncwarp();
        if (lane == 0) arrive_here(&s.sempty[w]);
        if (!__all_sync(0xffffffffu, wait_or_dead(s, &s.sfree[w], phase ^ 1u, p.fault))) break;
        phase ^= 1u;
        *reinterpret_cast<uint4*>(s.words[w][0][lane]) = wa;
        *reinterpret_cast<uint4*>(s.words[w][1][lane]) = wb;
        *reinterpret_cast<uint4*>(s.words[w][2][lane]) = wc;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_at_issuer<G, true>(&s.scaled[w]);
      }
    } else if (warp == kLoadWarp && elect_one()) {
      // ---- loads of codes ----
      Ring<kStages> st;
      uint32_t used = 0;  // stages that have been loaded at least once
      bool ok = true;
      for (int t = blockIdx.x / G; ok && t < tiles; t += gridDim.x / G) {
        const Tile tl = tile_at<G>(t, tiles_m, tiles_n, rank);
        for (int kb = 0; kb < p.kb; ++kb) {
          if (!(ok = wait_or_dead(s, &s.empty[st.slot], st.phase ^ 1u, p.fault))) break;
          // a pair's loads all complete on the even CTA's barrier
          if (rank == 0) mbar_expect_tx(&s.full[st.slot], G * (S::kABytes + S::kBBytes));
          if constexpr (G == 1) {
            tma_load_2d(s.a[st.slot], &p.a, &s.full[st.slot], kb * kBlock, tl.m0);
            tma_load_2d(s.b[st.slot], &p.b, &s.full[st.slot], kb * kBlock, tl.n0);
          } else {
            tma_load_2d_pair(s.a[st.slot], &p.a, &s.full[st.slot], kb * kBlock, tl.m0);
            tma_load_2d_pair(s.b[st.slot], &p.b, &s.full[st.slot], kb * kBlock, tl.n0 + rank * (kBN / G));
          }
          used |= 1u << st.slot;
          st.next();
        }
      }
      // Stopped early: copies may be in flight into this CTA's shared memory.  Wait (bounded) for
      // the last load of every stage: those before the ring's position are in its current phase,
      // the others in the one before.  (A pair's stages complete on the even CTA's barriers; the odd
      // one waits for it at the end.)
      if (!ok) {
        for (int i = 0; i < kStages; ++i)
          if (rank == 0 && (used >> i & 1u)) mbar_wait_bounded(&s.full[i], i < st.slot ? st.phase : st.phase ^ 1u);
      }
    } else if (warp == kScaleLoadWarp && elect_one()) {
      // ---- loads of scales, in the same queue as the codes': a plain load would wait behind every
      // stage that is under way.  (From the codes' thread they cost it half of its time.) ----
      Chains in(blockIdx.x / G, tiles, gridDim.x / G, p.kb);
      Ring<kScaleSlots> sc;
      uint32_t used = 0;
      bool ok = true;
      for (; in.more(); in.next()) {
        if (!(ok = wait_or_dead(s, &s.sempty[sc.slot], sc.phase ^ 1u, p.fault))) break;
        const Tile tl = tile_at<G>(in.t, tiles_m, tiles_n, rank);
        mbar_expect_tx(&s.sfull[sc.slot], kChain * (kBM + kBN) * 4);
        tma_load_2d(s.sa[sc.slot], &p.sa, &s.sfull[sc.slot], tl.m0, kChain * in.c);
        tma_load_2d(s.sb[sc.slot], &p.sb, &s.sfull[sc.slot], tl.n0, kChain * in.c);
        used |= 1u << sc.slot;
        sc.next();
      }
      if (!ok) {
        for (int i = 0; i < kScaleSlots; ++i)
          if (used >> i & 1u) mbar_wait_bounded(&s.sfull[i], i < sc.slot ? sc.phase : sc.phase ^ 1u);
      }
    } else if (warp == kMmaWarp && rank == 0 && elect_one()) {
      // ---- tensor-core instructions ----
      const uint32_t idesc = mxf8_instruction(p.a_fmt, p.b_fmt, G * kBM, kBN);
      Ring<kStages> st;
      Ring<kScaleSlots> sc;
      Ring<2> acc;
      bool ok = true;
      for (int t = blockIdx.x / G; ok && t < tiles; t += gridDim.x / G) {
        for (int kb = 0; ok && kb < p.kb; kb += kChain) {
          if (!(ok = wait_or_dead(s, &s.tempty[acc.slot], acc.phase ^ 1u, p.fault))) break;
          if (!(ok = wait_or_dead(s, &s.scaled[sc.slot], sc.phase, p.fault))) break;
          tensor_fence_after();
          const uint32_t sf = tmem + kScaleCol + acc.slot * kScaleCols;
#pragma unroll
          for (int i = 0; i < 3; ++i) tensor_copy_scales<G>(sf + 4 * i, smem_addr(s.words[sc.slot][i]));
#pragma unroll
          for (int j = 0; j < kChain; ++j) {
            if (kb + j >= p.kb) break;
            if (!(ok = wait_or_dead(s, &s.full[st.slot], st.phase, p.fault))) break;
            tensor_fence_after();
            const uint64_t da = operand_desc(smem_addr(s.a[st.slot])), db = operand_desc(smem_addr(s.b[st.slot]));
#pragma unroll
            for (int k = 0; k < kBlock / 32; ++k)  // 32 bytes along the swizzled row: 2 units of 16
              tensor_mma_mxf8<G>(tmem + acc.slot * kBN, da + 2 * k, db + 2 * k, idesc | mxf8_scale_byte(j), sf, sf + 4,
                              j > 0 || k > 0);
            tensor_commit<G>(&s.empty[st.slot]);
            st.next();
          }
          if (!ok) break;
          tensor_commit<G>(&s.sfree[sc.slot]);
          tensor_commit<G>(&s.tfull[acc.slot]);
          sc.next();
          acc.next();
        }
      }
    }
  } else {
    registers_up<kSumRegs>();
    // ---- float32 sums: warp w holds rows 32 (w & 3) .., columns kCols (w >> 2) .. ----
    const int col0 = kCols * (warp >> 2);
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + col0;
    Ring<2> acc;
    bool ok = true;
    for (int t = blockIdx.x / G; ok && t < tiles; t += gridDim.x / G) {
      const Tile tl = tile_at<G>(t, tiles_m, tiles_n, rank);
      uint64_t sum[kCols / 2];  // pairs of columns
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) sum[i] = 0;
      for (int kb = 0; kb < p.kb; kb += kChain) {
        // every lane waits (each reads what the barrier guards); the warp goes on or stops as one
        ok = __all_sync(0xffffffffu, wait_or_dead(s, &s.tfull[acc.slot], acc.phase, p.fault));
        if (!ok) break;
        tensor_fence_after();
        // 16 columns at a time, the next ones on their way while these are added
        uint32_t v[2][16];
        tmem_load16(taddr + acc.slot * kBN, v[0]);
#pragma unroll
        for (int c = 0; c < kCols / 16; ++c) {
          tensor_wait_load(v[c & 1]);
          if (c + 1 < kCols / 16) {
            tmem_load16(taddr + acc.slot * kBN + 16 * (c + 1), v[(c + 1) & 1]);
          } else {
            tensor_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at_issuer<G, false>(&s.tempty[acc.slot]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sum[8 * c + j] = add2(sum[8 * c + j], pack2(v[c & 1][2 * j], v[c & 1][2 * j + 1]));
        }
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
  // A CTA that stopped early may have matrix instructions in flight: wait (bounded) for them.
  if (warp == kMmaWarp && rank == 0 && s.dead && elect_one()) {
    tensor_commit<G>(&s.drain);
    mbar_wait_bounded(&s.drain, 0);
  }
  __syncthreads();
  if constexpr (G > 1) cluster_sync();  // neither CTA leaves while the other may still reach its memory
  if (warp == kMmaWarp) {
    tensor_fence_after();
    tmem_free<G>(tmem, kTmemCols);
  }
}

template <int G>
static cudaError_t launch_matmul_t(const MatmulParams& p, long long tiles, int sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  const long long groups = tiles < sms / G ? tiles : sms / G;
  cfg.gridDim = dim3(static_cast<unsigned>(groups * G));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem<G>;
  cfg.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = G;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = G > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, matmul_kernel<G>, p);
}

MatmulPlan plan_matmul(long long m, long long n, int sms) {
  const int group = m > kBM ? 2 : 1;
  return MatmulPlan{group, kBM, kBN / group, kBN, kChain, ((m + group * kBM - 1) / (group * kBM)) * ((n + kBN - 1) / kBN)};
}

cudaError_t launch_matmul(const MatmulParams& p, const MatmulPlan& plan, int sms, cudaStream_t st) {
  return plan.group == 1 ? launch_matmul_t<1>(p, plan.tiles, sms, st) : launch_matmul_t<2>(p, plan.tiles, sms, st);
}

cudaError_t prepare_matmul_kernels() {
  const cudaError_t e = cudaFuncSetAttribute(matmul_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kSmem<1>));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(matmul_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kSmem<2>));
}

}  // namespace demo
