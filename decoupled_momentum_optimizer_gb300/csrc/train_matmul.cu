// Product of two matrices in 8-bit floating point with a power-of-two scale for each block of 128
// along k:
//
//   out[m][n] (+)= sum over blocks b of sa[b][m] sb[b][n] * (sum over k in block b of a[m][k] b[n][k])
//
// A pair of CTAs computes a 256 x bn tile (bn up to 224), or one CTA 128 x bn.  TMA brings 128 codes of
// k of both operands into a ring of shared-memory stages, and the scales by a thread and a ring of
// their own; two warps pack the scales of four blocks into a 32-bit word per row (UE8M0 bytes), which
// the tensor core copies to tensor memory; one thread issues four K = 32 block-scaled tensor-core
// instructions per block.  Four blocks run into one of two halves of tensor memory, and eight warps
// meanwhile add the other half to float32 sums in registers: the tensor core's accumulator holds 512
// products at most, and every longer sum is an IEEE float32 addition.  (The scales in the instruction
// instead of in the sums: with a multiply-add per element and block in the eight warps, 8192 x 2048 x
// 8192 took 170 us, and 250 us with a scale per row of b.)  224 columns leave room in tensor memory for
// two halves and their scales.
//
// What bounds it: power, at n = 8192.  8192 x 8192 x 2048 takes 102 us (2.7 PFLOP/s) over a second, at 1.37 kW
// with the SM clock down to 1.67 GHz, and 91 in the first milliseconds.  At n = 2048 the layout takes a share
// as well: 8192 x 2048 x 8192 takes 105 to 110 us (2.5 to 2.6 PFLOP/s) at 1.8 GHz and 98 at first; its 352
// tiles of 256 x 192 on 76 pairs are 4.6 rounds run as 5, over 2112 columns for 2048, 90% useful work where
// n = 8192 has 96%.  At full clock the stages' arrival would be next: a block of a 256 x 224 tile is 448 cycles of tensor core and 30 KB for either CTA, and takes
// about 600; half of b per CTA of a pair is what keeps that near the tensor cores' pace (one CTA per
// 128 x 224 tile reads 44 KB a block).
#include "train_common.cuh"
#include "train_tensor.cuh"

namespace demo {

namespace {

constexpr int kSumWarps = 8, kScaleWarps = 2;
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
constexpr int kCols = kBN / 2;  // most columns of a summing warp
constexpr int kOutBytes = 32 * kBN;  // a warp's rows on their way out, bn bytes each

// G CTAs (1, or a cluster of 2) share a tile: each loads its 128 rows of a and bn / G of b, and the
// rest of the shared memory is stages.
template <int G>
struct Shared {
  // Stages: a's rows, then b's, whole units of 1024 bytes (swizzle atoms).  A pair has five; single CTAs
  // have as many as fit (at most kMaxStages), with only the rows of a that exist.
  static constexpr int kRingBytes = G == 1 ? kRingBytesSingle : kPairStages * (kBM + kBN / 2) * kBlock;
  uint8_t ring[kRingBytes];  // 1024-byte aligned
  uint8_t out[kSumWarps][kOutBytes];
  // Scale words: row 32 c + l of an operand at [l][c] of its 512-byte unit of 128 rows (a's, then
  // b's two), as the tensor core's copy wants them.
  uint32_t words[kScaleSlots][3][32][4];
  // a chain's scales as they arrive: rows of kBM, and of bn
  float sa[kScaleSlots][kChain * kBM];
  float sb[kScaleSlots][kChain * kBN];
  uint64_t full[kMaxStages], empty[kMaxStages];
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
// A split tile's float32 sums go where the stages were.
static_assert(kBM * kBN * 4 <= Shared<1>::kRingBytes, "a tile of sums");

template <int G>
__device__ __forceinline__ bool wait_or_dead(Shared<G>& s, uint64_t* bar, uint32_t parity, unsigned int* fault) {
  return wait_bounded<G != 1>(&s.dead, bar, parity, fault);
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

struct Tile {
  int m0, n0;
};

// The tiles and blocks of a CTA (or pair).  Tiles go in bands of 1024 rows of m, along n within a
// band: those that run at one time then cover about as many rows of a as of b, and share both in
// the L2 cache.
struct Work {
  int tiles_m, tiles_n, tiles, bn;
  int first, stride;  // tiles first, first + stride, ...
  int kb0, blocks;    // blocks of k, from kb0
  int group, rank;    // CTAs of a tile's rows, and this one's number

  // m0 is the CTA's own first row.
  __device__ __forceinline__ Tile tile(int t) const {
    const int band_tiles = 8 / group;
    const int per = band_tiles * tiles_n;
    const int band = t / per, i = t - band * per;
    const int height = tiles_m - band * band_tiles < band_tiles ? tiles_m - band * band_tiles : band_tiles;
    const int col = i / height;
    return Tile{((band * band_tiles + i - col * height) * group + rank) * kBM, col * bn};
  }
};

// A CTA's chains (up to kChain blocks of a tile) in order, tile after tile.
struct Chains {
  const Work& w;
  int t, c = 0, per_tile;
  __device__ __forceinline__ explicit Chains(const Work& work)
      : w(work), t(work.blocks > 0 ? work.first : work.tiles), per_tile((work.blocks + kChain - 1) / kChain) {}
  __device__ __forceinline__ bool more() const { return t < w.tiles; }
  __device__ __forceinline__ void next(int by = 1) {
    for (c += by; c >= per_tile && t < w.tiles; c -= per_tile) t += w.stride;
  }
};

// The scales of 128 rows and a chain's blocks (`ld` floats from block to block) as exponent bytes:
// word i is row 32 i + lane's.  Rows past `rows` have scale 1.
__device__ __forceinline__ uint4 scale_words(const float* v, int ld, int rows, int lane) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 0x7f7f7f7fu;
    if (32 * i < rows) {
      w[i] = 0;
#pragma unroll
      for (int j = 0; j < kChain; ++j) w[i] |= scale_byte(v[j * ld + 32 * i + lane]) << (8 * j);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ void store_elem(const MatmulParams& p, long long i, T v) {
  T* o = static_cast<T*>(p.out) + i;
  if constexpr (sizeof(T) == 4) {
    *o = p.add ? *o + v : v;
  } else {
    *o = v;
  }
}

// Results that no bulk store can write (rows or addresses off 16 bytes): a warp's `cols` columns,
// staged as below, one row after another.
template <typename T>
__device__ __noinline__ void store_plain(const MatmulParams& p, const uint8_t* buf, int cols, int lane, long long m0,
                                         long long n0) {
  for (int r = 0; r < 32 && m0 + r < p.m; ++r)
    for (int c = lane; c < cols && n0 + c < p.n; c += 32)
      store_elem<T>(p, (m0 + r) * p.ldo + n0 + c, reinterpret_cast<const T*>(buf + r * p.bn)[c]);
}

// What a warp has staged (32 rows of bn bytes, `cols` columns) to out[m0 ..][n0 ..]: one bulk store,
// which cuts off what is past the matrix, adds where asked, and runs on behind the warp's next work.
template <typename T>
__device__ __forceinline__ void store_staged(const MatmulParams& p, const uint8_t* buf, int cols, int lane,
                                             long long m0, long long n0) {
  if (p.bulk_out) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && m0 < p.m && n0 < p.n) {
      if (p.add)
        tma_add_2d(&p.o, buf, static_cast<int>(n0), static_cast<int>(m0));
      else
        tma_store_2d(&p.o, buf, static_cast<int>(n0), static_cast<int>(m0));
      bulk_commit();
    }
  } else {
    __syncwarp();
    store_plain<T>(p, buf, cols, lane, m0, n0);
  }
}

// The staging buffer may be written again: its last bulk store has read it.
__device__ __forceinline__ void staging_free(int lane) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
}

// A warp's 32 rows (lane l holds row l) x bn / 2 columns to out[m0 ..][n0 ..], through rows of bn bytes
// in shared memory: all columns at once in 16 bits, half of them at a time in 32.
template <typename T>
__device__ __forceinline__ void store_sums(const MatmulParams& p, uint8_t* buf, int lane,
                                           const uint64_t (&sum)[kCols / 2], long long m0, long long n0) {
  if constexpr (sizeof(T) == 2) {
    staging_free(lane);
#pragma unroll
    for (int u = 0; u < kCols / 8; ++u) {
      if (16 * u < p.bn) {
        Vec<T, 8> o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 q = unpack2(sum[4 * u + e]);
          o.e[2 * e] = from_f32<T>(q.x);
          o.e[2 * e + 1] = from_f32<T>(q.y);
        }
        *reinterpret_cast<Vec<T, 8>*>(buf + lane * p.bn + 16 * u) = o;
      }
    }
    store_staged<T>(p, buf, p.bn / 2, lane, m0, n0);
  } else {
    const int units = p.bn / 16;  // of four columns, a half
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      staging_free(lane);
#pragma unroll
      for (int u = 0; u < kCols / 4; ++u) {
        if (u >= h * units && u < (h + 1) * units) {
          const float2 x = unpack2(sum[2 * u]), y = unpack2(sum[2 * u + 1]);
          *reinterpret_cast<float4*>(buf + lane * p.bn + 16 * (u - h * units)) = make_float4(x.x, x.y, y.x, y.y);
        }
      }
      store_staged<T>(p, buf, p.bn / 4, lane, m0, n0 + h * (p.bn / 4));
    }
  }
}

// Four columns of a row from a split tile's joined sums.
template <typename T>
__device__ __forceinline__ void store_four(const MatmulParams& p, long long m, long long n, float4 v) {
  if (m >= p.m || n >= p.n) return;
  const long long i = m * p.ldo + n;
  const float x[4] = {v.x, v.y, v.z, v.w};
  if (p.bulk_out && n + 4 <= p.n) {  // rows are multiples of 16 bytes from an aligned start
    if constexpr (sizeof(T) == 4) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + i);
      if (p.add) {
        const float4 w = *o;
        v = make_float4(w.x + v.x, w.y + v.y, w.z + v.z, w.w + v.w);
      }
      *o = v;
    } else {
      Vec<T, 4> o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o.e[e] = from_f32<T>(x[e]);
      *reinterpret_cast<Vec<T, 4>*>(static_cast<T*>(p.out) + i) = o;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.n) store_elem<T>(p, i + e, from_f32<T>(x[e]));
  }
}

}  // namespace

// G = 2: pairs of CTAs, each pair walks its tiles.  G = 1: a cluster of p.split CTAs for a tile, each
// sums its share of k; the shares are joined in the order of k through distributed shared memory.
template <int G>
__global__ void __launch_bounds__(kThreads, 1) matmul_kernel(const __grid_constant__ MatmulParams p) {
  extern __shared__ uint8_t raw[];
  using S = Shared<G>;
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  // the warp's number from one lane: the roles below are branches of whole warps
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = G == 1 ? 0 : static_cast<int>(cluster_rank());  // in the pair
  const int part = G == 1 ? static_cast<int>(cluster_rank()) : 0;  // of k
  // A stage: the rows of a that are loaded (the tensor core reads 128, past fewer into what follows: those
  // results are not used), and b's.
  const int a_bytes = (G == 1 ? p.rows_a : kBM) * kBlock;
  const int stage_bytes = a_bytes + (G == 1 ? p.bn : kBN / 2) * kBlock;
  const int stages = G == 1 ? p.stages : kPairStages;
  Work work;
  work.tiles_m = static_cast<int>((p.m + G * kBM - 1) / (G * kBM));
  work.tiles_n = static_cast<int>((p.n + p.bn - 1) / p.bn);
  work.tiles = work.tiles_m * work.tiles_n;
  work.bn = p.bn;
  work.group = G;
  work.rank = rank;
  if constexpr (G == 1) {
    const int q = p.kb / p.split, r = p.kb - q * p.split;
    work.first = blockIdx.x / p.split;
    work.stride = work.tiles;
    work.kb0 = part * q + (part < r ? part : r);
    work.blocks = q + (part < r ? 1 : 0);
  } else {
    work.first = blockIdx.x / G;
    work.stride = gridDim.x / G;
    work.kb0 = 0;
    work.blocks = p.kb;
  }

  if (threadIdx.x == 32 * kLoadWarp && p.kb > 0) {
    prefetch_tmap(&p.a);
    prefetch_tmap(&p.b);
    prefetch_tmap(&p.sa);
    prefetch_tmap(&p.sb);
    if (p.bulk_out) prefetch_tmap(&p.o);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
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
  griddep_launch_dependents();
  griddep_wait();  // the operands, and the result that was there, are complete from here on
  const uint32_t tmem = s.tmem;

  if (warp >= kSumWarps) {
    registers_down<kFeedRegs>();
    if (warp < kLoadWarp) {
      // ---- scale words: warp w makes those of every second chain, in slot w ----
      const int w = warp - kSumWarps;
      Chains in(work);
      uint32_t phase = 0;
      for (in.next(w); in.more(); in.next(kScaleWarps)) {
        if (!__all_sync(0xffffffffu, wait_or_dead(s, &s.sfull[w], phase, p.fault))) break;
        const uint4 wa = scale_words(s.sa[w], kBM, kBM, lane), wb = scale_words(s.sb[w], p.bn, p.bn, lane),
                    wc = scale_words(s.sb[w] + 128, p.bn, p.bn - 128, lane);
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
      Ring st(stages);
      uint32_t used = 0;  // stages that have been loaded at least once
      bool ok = true;
      const uint32_t bytes = G * a_bytes + p.bn * kBlock;  // of a stage, of the pair together
      long long loads = 0;
      for (int t = work.first; ok && t < work.tiles; t += work.stride) {
        const Tile tl = work.tile(t);
        for (int kb = work.kb0; kb < work.kb0 + work.blocks; ++kb) {
          if (!(ok = wait_or_dead(s, &s.empty[st.slot], st.phase ^ 1u, p.fault))) break;
          // a pair's loads all complete on the even CTA's barrier
          if (rank == 0) mbar_expect_tx(&s.full[st.slot], bytes + stall_extra(p.stall_at, blockIdx.x, loads++));
          uint8_t* a = s.ring + st.slot * stage_bytes;
          if constexpr (G == 1) {
            tma_load_2d(a, &p.a, &s.full[st.slot], kb * kBlock, tl.m0);
            tma_load_2d(a + a_bytes, &p.b, &s.full[st.slot], kb * kBlock, tl.n0);
          } else {
            tma_load_2d_pair(a, &p.a, &s.full[st.slot], kb * kBlock, tl.m0);
            tma_load_2d_pair(a + a_bytes, &p.b, &s.full[st.slot], kb * kBlock, tl.n0 + rank * (p.bn / G));
          }
          used |= 1u << st.slot;
          st.next();
        }
      }
      // No copy may be in flight into this CTA's shared memory when it ends, and whoever stopped early,
      // here or among those who use the stages, waits for none.  Wait (bounded) for the last load of
      // every stage: those before the ring's position are in its current phase, the others in the one
      // before.  (A pair's stages complete on the even CTA's barriers; the odd one waits for it at the
      // end.)
      for (int i = 0; i < stages; ++i)
        if (rank == 0 && (used >> i & 1u)) mbar_wait_bounded(&s.full[i], i < st.slot ? st.phase : st.phase ^ 1u);
    } else if (warp == kScaleLoadWarp && elect_one()) {
      // ---- loads of scales, in the same queue as the codes': a plain load would wait behind every
      // stage that is under way.  (From the codes' thread they cost it half of its time.) ----
      Chains in(work);
      Ring sc(kScaleSlots);
      uint32_t used = 0;
      for (; in.more(); in.next()) {
        if (!wait_or_dead(s, &s.sempty[sc.slot], sc.phase ^ 1u, p.fault)) break;
        const Tile tl = work.tile(in.t);
        const int kb = work.kb0 + kChain * in.c;  // rows past the last block are filled, or not used
        mbar_expect_tx(&s.sfull[sc.slot], kChain * (kBM + p.bn) * 4);
        tma_load_2d(s.sa[sc.slot], &p.sa, &s.sfull[sc.slot], tl.m0, kb);
        tma_load_2d(s.sb[sc.slot], &p.sb, &s.sfull[sc.slot], tl.n0, kb);
        used |= 1u << sc.slot;
        sc.next();
      }
      for (int i = 0; i < kScaleSlots; ++i)
        if (used >> i & 1u) mbar_wait_bounded(&s.sfull[i], i < sc.slot ? sc.phase : sc.phase ^ 1u);
    } else if (warp == kMmaWarp && rank == 0 && elect_one()) {
      // ---- tensor-core instructions ----
      const uint32_t idesc = mxf8_instruction(p.a_fmt, p.b_fmt, G * kBM, p.bn);
      Ring st(stages);
      Ring sc(kScaleSlots);
      Ring acc(2);
      bool ok = true;
      for (int t = work.first; ok && t < work.tiles; t += work.stride) {
        for (int kb = 0; ok && kb < work.blocks; kb += kChain) {
          if (!(ok = wait_or_dead(s, &s.tempty[acc.slot], acc.phase ^ 1u, p.fault))) break;
          if (!(ok = wait_or_dead(s, &s.scaled[sc.slot], sc.phase, p.fault))) break;
          tensor_fence_after();
          const uint32_t sf = tmem + kScaleCol + acc.slot * kScaleCols;
#pragma unroll
          for (int i = 0; i < 3; ++i) tensor_copy_scales<G>(sf + 4 * i, smem_addr(s.words[sc.slot][i]));
#pragma unroll
          for (int j = 0; j < kChain; ++j) {
            if (kb + j >= work.blocks) break;
            if (!(ok = wait_or_dead(s, &s.full[st.slot], st.phase, p.fault))) break;
            tensor_fence_after();
            const uint32_t a = smem_addr(s.ring) + st.slot * stage_bytes;
            const uint64_t da = operand_desc(a), db = operand_desc(a + a_bytes);
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
    // ---- float32 sums: warp w holds rows 32 (w & 3) .., columns bn / 2 (w >> 2) .. ----
    const int cols = p.bn / 2, col0 = cols * (warp >> 2);
    const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + col0;
    Ring acc(2);
    bool ok = true;
    for (int t = work.first; ok && t < work.tiles; t += work.stride) {
      const Tile tl = work.tile(t);
      uint64_t sum[kCols / 2];  // pairs of columns
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) sum[i] = 0;
      for (int kb = 0; kb < work.blocks; kb += kChain) {
        // every lane waits (each reads what the barrier guards); the warp goes on or stops as one
        ok = __all_sync(0xffffffffu, wait_or_dead(s, &s.tfull[acc.slot], acc.phase, p.fault));
        if (!ok) break;
        tensor_fence_after();
        // 16 columns at a time, the next ones on their way while these are added
        uint32_t v[2][16];
        tmem_load16(taddr + acc.slot * kBN, v[0]);
#pragma unroll
        for (int c = 0; c < kCols / 16; ++c) {
          if (16 * c < cols) {
            tensor_wait_load(v[c & 1]);
            if (16 * (c + 1) < cols) {
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
        }
        acc.next();
      }
      if (!ok) break;
      if (G == 1 && p.split > 1) {
        // to shared memory, unit u (four columns) of row r at [u][r]
        float4* red = reinterpret_cast<float4*>(s.ring);
#pragma unroll
        for (int u = 0; u < kCols / 4; ++u) {
          if (4 * u < cols) {
            const float2 x = unpack2(sum[2 * u]), y = unpack2(sum[2 * u + 1]);
            red[(col0 / 4 + u) * kBM + 32 * (warp & 3) + lane] = make_float4(x.x, x.y, y.x, y.y);
          }
        }
      } else {
        const long long m0 = tl.m0 + 32 * (warp & 3), n0 = tl.n0 + col0;
        if (p.out_dtype == kBF16)
          store_sums<__nv_bfloat16>(p, s.out[warp], lane, sum, m0, n0);
        else if (p.out_dtype == kF16)
          store_sums<__half>(p, s.out[warp], lane, sum, m0, n0);
        else
          store_sums<float>(p, s.out[warp], lane, sum, m0, n0);
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tensor_fence_before();
  __syncthreads();
  // A CTA that stopped early may have matrix instructions in flight: wait (bounded) for them.
  if (warp == kMmaWarp && rank == 0 && s.dead && elect_one()) {
    tensor_commit<G>(&s.drain);
    mbar_wait_bounded(&s.drain, 0);
  }
  __syncthreads();
  if (G > 1 || p.split > 1) cluster_sync();  // a pair: neither CTA leaves while the other may reach its memory
  if (G == 1 && p.split > 1) {
    // each CTA joins its share of the columns, always from the first part of k to the last
    const Tile tl = work.tile(work.first);
    const int units = p.bn / 4, row = threadIdx.x & (kBM - 1);
    const int hi = units * (part + 1) / p.split;
    const uint32_t red = smem_addr(s.ring);
    for (int u = units * part / p.split + (threadIdx.x >> 7); u < hi && tl.m0 + row < p.m; u += kThreads / kBM) {
      float4 v[kMaxSplit];
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q)
        if (q < p.split) v[q] = load_cluster(red + (u * kBM + row) * 16, q);
#pragma unroll
      for (int q = 1; q < kMaxSplit; ++q)
        if (q < p.split) v[0] = make_float4(v[0].x + v[q].x, v[0].y + v[q].y, v[0].z + v[q].z, v[0].w + v[q].w);
      if (p.out_dtype == kBF16)
        store_four<__nv_bfloat16>(p, tl.m0 + row, tl.n0 + 4 * u, v[0]);
      else if (p.out_dtype == kF16)
        store_four<__half>(p, tl.m0 + row, tl.n0 + 4 * u, v[0]);
      else
        store_four<float>(p, tl.m0 + row, tl.n0 + 4 * u, v[0]);
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its sums
  }
  if (warp == kMmaWarp) {
    tensor_fence_after();
    tmem_free<G>(tmem, kTmemCols);
  }
}

template <int G>
struct MatmulLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2] = {};
  MatmulLaunch(unsigned grid, int cluster, cudaStream_t st) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem<G>;
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
  }
};

cudaError_t launch_matmul(const MatmulParams& p, const MatmulPlan& plan, cudaStream_t st) {
  if (plan.group == 1) {
    MatmulLaunch<1> l(plan.grid, plan.split, st);
    return cudaLaunchKernelEx(&l.cfg, matmul_kernel<1>, p);
  }
  MatmulLaunch<2> l(plan.grid, 2, st);
  return cudaLaunchKernelEx(&l.cfg, matmul_kernel<2>, p);
}

// A count of 0 where the device has no place for such a cluster (a part of one, with few SMs or none that
// are together): plan_matmul goes without it, and whatever else the library does is not concerned.
template <int G>
static int clusters_of(int sms, int size) {
  if (sms < size) return 0;
  MatmulLaunch<G> l(static_cast<unsigned>(sms / size * size), size, nullptr);
  l.cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, matmul_kernel<G>, &l.cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

cudaError_t prepare_matmul_kernels(int sms, Clusters* clusters) {
  cudaError_t e = cudaFuncSetAttribute(matmul_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmem<1>));
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(matmul_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem<2>));
  if (e != cudaSuccess) return e;
  for (int size = 1; size <= kMaxSplit; ++size) clusters->of[size] = clusters_of<1>(sms, size);
  clusters->of[0] = clusters_of<2>(sms, 2);
  return cudaSuccess;
}

}  // namespace demo
