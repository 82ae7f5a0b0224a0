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
constexpr int kStages = 4;
constexpr int kChain = 4;  // blocks of 128 that one half of tensor memory sums
constexpr int kSumWarps = 8, kScaleWarps = 4;
constexpr int kLoadWarp = kSumWarps + kScaleWarps, kMmaWarp = kLoadWarp + 1;
// Whole groups of four warps, launched with 128 registers a thread: the summing ones take 192, the
// others keep 64.
constexpr int kThreads = 512;
constexpr int kSumRegs = 192, kFeedRegs = 64;
static_assert(256 * kSumRegs + 256 * kFeedRegs == kThreads * 128, "the launch's registers");
constexpr uint32_t kTmemCols = 512;
// Scale words of a half: 4 columns of a's (one for 32 rows) and 8 of b's (7 used).
constexpr uint32_t kScaleCol = 2 * kBN, kScaleCols = 12;
static_assert(kScaleCol + 2 * kScaleCols <= kTmemCols, "tensor memory");
constexpr int kScaleSlots = 4;  // chains whose words are ready in shared memory
static_assert(kChain == 4, "a word holds the scales of a chain");
constexpr uint32_t kABytes = kBM * kBlock, kBBytes = kBN * kBlock;
constexpr int kCols = kBN / 2;  // columns of a summing warp

struct Shared {
  uint8_t a[kStages][kABytes];  // 1024-byte aligned (swizzle atoms)
  uint8_t b[kStages][kBBytes];
  uint4 out[kSumWarps][128];  // a warp's 32 rows x 64 bytes on their way out
  // Scale words: row 32 c + l of an operand at [l][c] of its 512-byte unit of 128 rows (a's, then
  // b's two), as the tensor core's copy wants them.
  uint32_t words[kScaleSlots][3][32][4];
  uint64_t full[kStages], empty[kStages];
  uint64_t scaled[kScaleSlots], sfree[kScaleSlots];
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

// A CTA's chains in order, tile after tile: the scales of up to four blocks of three rows, row
// 32 w + l of a's tile (warp w, lane l) and rows 32 w + l and 128 + 32 w + l of b's.
struct ScaleStream {
  const MatmulParams& p;
  long long lda, ldb, t, tiles;
  int row, tiles_m, tiles_n, kb = 0;
  const float *pa, *pb;
  bool in_a, in_b0, in_b1;  // whether the rows exist

  __device__ __forceinline__ ScaleStream(const MatmulParams& q, int r, int tm, int tn)
      : p(q), lda((q.m + 3) / 4 * 4), ldb((q.n + 3) / 4 * 4), t(blockIdx.x), tiles(static_cast<long long>(tm) * tn),
        row(r), tiles_m(tm), tiles_n(tn) {
    if (p.kb == 0) t = tiles;
    start();
  }
  __device__ __forceinline__ void start() {
    if (t >= tiles) return;
    const Tile tl = tile_at(t, tiles_m, tiles_n);
    pa = p.a_scales + tl.m0 + row;
    pb = p.b_scales + tl.n0 + row;
    in_a = tl.m0 + row < p.m;
    in_b0 = tl.n0 + row < p.n;
    in_b1 = 128 + row < kBN && tl.n0 + 128 + row < p.n;
  }
  // Returns false past the last chain.
  __device__ __forceinline__ bool fetch(float (&v)[3][4]) {
    if (t >= tiles) return false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = kb + j < p.kb;
      v[0][j] = in && in_a ? pa[j * lda] : 1.0f;
      v[1][j] = in && in_b0 ? pb[j * ldb] : 1.0f;
      v[2][j] = in && in_b1 ? pb[j * ldb + 128] : 1.0f;
    }
    pa += 4 * lda;
    pb += 4 * ldb;
    kb += 4;
    if (kb >= p.kb) {
      kb = 0;
      t += gridDim.x;
      start();
    }
    return true;
  }
};

// The exponent bytes of four powers of two.
__device__ __forceinline__ uint32_t scale_word(const float (&v)[4]) {
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) w |= ((__float_as_uint(v[j]) >> 23) & 0xffu) << (8 * j);
  return w;
}

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
      mbar_init(&s.scaled[i], kScaleWarps);
      mbar_init(&s.sfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tfull[i], 1);
      mbar_init(&s.tempty[i], kSumWarps);
    }
    mbar_init(&s.drain, 1);
    s.dead = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&s.tmem, kTmemCols);
  tensor_fence_before();
  __syncthreads();
  tensor_fence_after();
  const uint32_t tmem = s.tmem;

  if (warp >= kSumWarps) {
    registers_down<kFeedRegs>();
    if (warp < kLoadWarp) {
      // ---- scales, a chain ahead of the slot that waits to be free ----
      const int w = warp - kSumWarps;
      ScaleStream in(p, 32 * w + lane, tiles_m, tiles_n);
      Ring<kScaleSlots> sc;
      float v[3][4];
      while (in.fetch(v)) {
        if (!__all_sync(0xffffffffu, wait_or_dead(s, &s.sfree[sc.slot], sc.phase ^ 1u, p.fault))) break;
#pragma unroll
        for (int i = 0; i < 3; ++i) s.words[sc.slot][i][lane][w] = scale_word(v[i]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.scaled[sc.slot]);
        sc.next();
      }
    } else if (warp == kLoadWarp && lane == 0) {
      // ---- loads ----
      Ring<kStages> st;
      uint32_t used = 0;  // stages that have been loaded at least once
      bool ok = true;
      for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile tl = tile_at(t, tiles_m, tiles_n);
        for (int kb = 0; kb < p.kb; ++kb) {
          if (!(ok = wait_or_dead(s, &s.empty[st.slot], st.phase ^ 1u, p.fault))) break;
          mbar_expect_tx(&s.full[st.slot], kABytes + kBBytes);
          tma_load_2d(s.a[st.slot], &p.a, &s.full[st.slot], kb * kBlock, tl.m0);
          tma_load_2d(s.b[st.slot], &p.b, &s.full[st.slot], kb * kBlock, tl.n0);
          used |= 1u << st.slot;
          st.next();
        }
      }
      // Stopped early: copies may be in flight into this CTA's shared memory.  Wait (bounded) for
      // the last load of every stage: the stages before the ring's position are in its current
      // phase, the others in the one before.
      if (!ok) {
        for (int i = 0; i < kStages; ++i)
          if (used >> i & 1u) mbar_wait_bounded(&s.full[i], i < st.slot ? st.phase : st.phase ^ 1u);
      }
    } else if (warp == kMmaWarp && lane == 0) {
      // ---- tensor-core instructions ----
      const uint32_t idesc = mxf8_instruction(p.a_fmt, p.b_fmt, kBM, kBN);
      Ring<kStages> st;
      Ring<kScaleSlots> sc;
      Ring<2> acc;
      bool ok = true;
      for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        for (int kb = 0; ok && kb < p.kb; kb += kChain) {
          if (!(ok = wait_or_dead(s, &s.tempty[acc.slot], acc.phase ^ 1u, p.fault))) break;
          if (!(ok = wait_or_dead(s, &s.scaled[sc.slot], sc.phase, p.fault))) break;
          tensor_fence_after();
          const uint32_t sf = tmem + kScaleCol + acc.slot * kScaleCols;
#pragma unroll
          for (int i = 0; i < 3; ++i) tensor_copy_scales(sf + 4 * i, smem_addr(s.words[sc.slot][i]));
#pragma unroll
          for (int j = 0; j < kChain; ++j) {
            if (kb + j >= p.kb) break;
            if (!(ok = wait_or_dead(s, &s.full[st.slot], st.phase, p.fault))) break;
            tensor_fence_after();
            const uint64_t da = operand_desc(smem_addr(s.a[st.slot])), db = operand_desc(smem_addr(s.b[st.slot]));
#pragma unroll
            for (int k = 0; k < kBlock / 32; ++k)  // 32 bytes along the swizzled row: 2 units of 16
              tensor_mma_mxf8(tmem + acc.slot * kBN, da + 2 * k, db + 2 * k, idesc | mxf8_scale_byte(j), sf, sf + 4,
                              j > 0 || k > 0);
            tensor_commit(&s.empty[st.slot]);
            st.next();
          }
          if (!ok) break;
          tensor_commit(&s.sfree[sc.slot]);
          tensor_commit(&s.tfull[acc.slot]);
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
    for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const Tile tl = tile_at(t, tiles_m, tiles_n);
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
            if (lane == 0) mbar_arrive(&s.tempty[acc.slot]);
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
  if (warp == kMmaWarp) {
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

int matmul_box_rows(bool b) { return b ? kBN : kBM; }

cudaError_t launch_matmul(const MatmulParams& p, int sms, cudaStream_t st) {
  const long long tiles = ((p.m + kBM - 1) / kBM) * ((p.n + kBN - 1) / kBN);
  matmul_kernel<<<static_cast<unsigned>(tiles < sms ? tiles : sms), kThreads, kSmem, st>>>(p);
  return cudaGetLastError();
}

cudaError_t prepare_matmul_kernels() {
  return cudaFuncSetAttribute(matmul_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
}

}  // namespace demo
