// Rows of a table by token, scaled, and the gradient of the table:
//
//   out[i]    = scale table[t_i], zeros where t_i is outside [0, vocab)
//   dtable[v] = scale sum_{i: t_i = v} dy[i]   (added to what it holds, or 0 for rows without a token)
//
// The lookup is bound by HBM and, for a few tokens, by two dependent loads.
//
// The gradient sums in a fixed order without atomics.  Tokens are sorted by value, equal ones by position, in
// the shared memory of one cluster; the sorted list is cut into pieces of kPiece positions, and a warp sums
// the rows of one piece over 32 accesses of columns, writing each token's sum as it ends.  A token that goes
// on past its piece leaves its part in the workspace (at most one at either end of a piece), and a second
// kernel adds a token's parts in the order of the pieces.  Words are spread as 1 / rank, so one row of the
// table may take a tenth of all positions: cutting by position, not by token, keeps the warps' work equal.
#include <cooperative_groups.h>

#include "train_common.cuh"

namespace demo {

namespace cg = cooperative_groups;

// Token of flat position i; positions lie in rows of `per` tokens, `ld` apart.
__device__ __forceinline__ long long token_at(const Tokens& t, long long i) {
  long long at = i;
  if (t.ld != t.per) {
    const long long row = i < (1ll << 32) && t.per < (1ll << 32)
                              ? static_cast<long long>(static_cast<uint32_t>(i) / static_cast<uint32_t>(t.per))
                              : i / t.per;
    at = row * t.ld + (i - row * t.per);
  }
  return t.wide ? static_cast<const long long*>(t.p)[at] : static_cast<const int*>(t.p)[at];
}

// N consecutive elements as float32, by 16-byte accesses (N * sizeof(T) a multiple of 16).
template <typename T, int N>
__device__ __forceinline__ void load_wide(const T* p, float (&v)[N]) {
  constexpr int P = 16 / static_cast<int>(sizeof(T));
#pragma unroll
  for (int i = 0; i < N / P; ++i) {
    const Vec<T, P> q = reinterpret_cast<const Vec<T, P>*>(p)[i];
#pragma unroll
    for (int e = 0; e < P; ++e) v[P * i + e] = to_f32(q.e[e]);
  }
}

template <typename T, int N>
__device__ __forceinline__ void store_wide(T* p, const float (&v)[N]) {
  constexpr int P = 16 / static_cast<int>(sizeof(T));
#pragma unroll
  for (int i = 0; i < N / P; ++i) {
    Vec<T, P> q;
#pragma unroll
    for (int e = 0; e < P; ++e) q.e[e] = from_f32<T>(v[P * i + e]);
    reinterpret_cast<Vec<T, P>*>(p)[i] = q;
  }
}

// ----------------------------------------------------------------------------
// Lookup
// ----------------------------------------------------------------------------

constexpr int kLookThreads = 256, kLookUnroll = 2;

// Eight columns a thread as 16-byte accesses, or (rows off 16 bytes) warps of 128 columns, four a lane.
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kLookThreads) lookup_kernel(const __grid_constant__ LookupParams p, long long per_row) {
  kernel_begin();
  const T* table = static_cast<const T*>(p.table);
  O* out = static_cast<O*>(p.out);
  const long long units = p.n * per_row;
  const auto row_of = [&](long long u) {
    return u < (1ll << 32) ? static_cast<long long>(static_cast<uint32_t>(u) / static_cast<uint32_t>(per_row)) : u / per_row;
  };
  if constexpr (VEC) {
    const long long first = static_cast<long long>(blockIdx.x) * (kLookThreads * kLookUnroll) + threadIdx.x;
    float v[kLookUnroll][8];
    long long row[kLookUnroll], col[kLookUnroll];
#pragma unroll
    for (int j = 0; j < kLookUnroll; ++j) {
      const long long u = first + j * kLookThreads;
      row[j] = -1;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
      if (u < units) {
        row[j] = row_of(u);
        col[j] = (u - row[j] * per_row) * 8;
        const long long t = token_at(p.tokens, row[j]);
        if (t >= 0 && t < p.vocab) load_wide<T, 8>(table + t * p.ldt + col[j], v[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kLookUnroll; ++j) {
      if (row[j] < 0) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] *= p.scale;
      store_wide<O, 8>(out + row[j] * p.ldo + col[j], v[j]);
    }
  } else {
    const long long u = static_cast<long long>(blockIdx.x) * (kLookThreads / 32) + (threadIdx.x >> 5);
    if (u >= units) return;
    const int lane = threadIdx.x & 31;
    const long long row = row_of(u), col = (u - row * per_row) * 128 + lane;
    const long long t = token_at(p.tokens, row);
    const bool live = t >= 0 && t < p.vocab;
    T v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (live && col + 32 * e < p.cols) v[e] = table[t * p.ldt + col + 32 * e];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + 32 * e < p.cols) out[row * p.ldo + col + 32 * e] = from_f32<O>(live ? to_f32(v[e]) * p.scale : 0.0f);
  }
}

namespace {

template <typename T, typename O>
cudaError_t launch_lookup_t(const LookupParams& p, cudaStream_t st) {
  const auto at = [](const void* q, long long ld, size_t size) {
    return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld * static_cast<long long>(size) % 16 == 0;
  };
  if (p.cols % 8 == 0 && at(p.table, p.ldt, sizeof(T)) && at(p.out, p.ldo, sizeof(O))) {
    const long long per = p.cols / 8, each = kLookThreads * kLookUnroll;
    return launch_overlapped(lookup_kernel<T, O, true>, static_cast<unsigned>((p.n * per + each - 1) / each), kLookThreads, 0,
                             st, p, per);
  }
  const long long per = (p.cols + 127) / 128, each = kLookThreads / 32;
  return launch_overlapped(lookup_kernel<T, O, false>, static_cast<unsigned>((p.n * per + each - 1) / each), kLookThreads, 0,
                           st, p, per);
}

template <typename T>
cudaError_t launch_lookup_o(const LookupParams& p, int out_dtype, cudaStream_t st) {
  if (out_dtype == kF32) return launch_lookup_t<T, float>(p, st);
  return out_dtype == kBF16 ? launch_lookup_t<T, __nv_bfloat16>(p, st) : launch_lookup_t<T, __half>(p, st);
}

}  // namespace

cudaError_t launch_lookup(const LookupParams& p, int table_dtype, int out_dtype, cudaStream_t st) {
  if (table_dtype == kF32) return launch_lookup_o<float>(p, out_dtype, st);
  return table_dtype == kBF16 ? launch_lookup_o<__nv_bfloat16>(p, out_dtype, st) : launch_lookup_o<__half>(p, out_dtype, st);
}

// ----------------------------------------------------------------------------
// Tokens sorted by value, equal ones by position
// ----------------------------------------------------------------------------

// A radix sort, least digit first, within one cluster: CTA r holds a run of positions, a warp a run of
// those, 32 at a time, so that (CTA, warp, round, lane) is their order.  In each pass a warp counts its
// digits (lanes with the same digit find each other by match and take consecutive ranks), the warps' counts
// become offsets within the CTA, the CTAs exchange their totals through distributed shared memory, and every
// item goes straight to its place in the CTA that will hold it.  Up to 2^16 tokens: 8 CTAs x 1024 threads x 8.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortRounds = 8;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
static_assert(kMaxSorted == 8 * kSortThreads * kSortRounds, "capacity of the largest cluster");
static_assert(kMaxSorted <= 65536, "positions are 16 bits");
static_assert(kDigits <= kSortThreads, "a thread for each digit");

struct SortShared {
  uint32_t key[2][kSortThreads * kSortRounds];
  uint16_t pos[2][kSortThreads * kSortRounds];
  uint16_t count[kSortWarps][kDigits];  // of a warp's items, then the warps' before it
  uint32_t total[kDigits];              // of the CTA
  uint32_t base[kDigits];               // where the CTA's items of a digit begin
  uint32_t scan[kSortWarps];
};

__global__ void __launch_bounds__(kSortThreads, 1) sort_tokens_kernel(const __grid_constant__ SortParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  SortShared& sh = *reinterpret_cast<SortShared*>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), me = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // items of a CTA (a multiple of 32), of a warp (a multiple of 32)
  const int per_cta = ((p.n + ctas - 1) / ctas + 31) / 32 * 32;
  const int begin = me * per_cta;
  const int mine = p.n - begin < per_cta ? (p.n > begin ? p.n - begin : 0) : per_cta;
  const int per_warp = (per_cta / 32 + kSortWarps - 1) / kSortWarps * 32;  // at most 32 * kSortRounds
  kernel_begin();
  for (int i = tid; i < mine; i += kSortThreads) {
    const long long t = token_at(p.tokens, p.first + begin + i);
    sh.key[0][i] = t >= 0 && t < p.vocab ? static_cast<uint32_t>(t) : static_cast<uint32_t>(p.vocab);  // others last
    sh.pos[0][i] = static_cast<uint16_t>(begin + i);
  }
  int from = 0;
  for (int pass = 0; pass < p.passes; ++pass, from ^= 1) {
    const int shift = pass * p.bits, digits = 1 << p.bits;
    for (int i = tid; i < kSortWarps * kDigits / 2; i += kSortThreads) reinterpret_cast<uint32_t*>(sh.count)[i] = 0;
    __syncthreads();  // counts cleared; and, in the first pass, the items are there
    uint32_t key[kSortRounds];
    int rank[kSortRounds];
    uint16_t* count = sh.count[warp];
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
      const int in_warp = 32 * j + lane, i = warp * per_warp + in_warp;
      const bool live = in_warp < per_warp && i < mine;
      rank[j] = -1;
      const unsigned there = __ballot_sync(0xffffffffu, live);
      if (live) {
        key[j] = sh.key[from][i];
        const uint32_t d = (key[j] >> shift) & (digits - 1);
        const unsigned same = __match_any_sync(there, d);
        const int before = __popc(same & ((1u << lane) - 1));
        rank[j] = count[d] + before;
        __syncwarp(there);
        if (before == 0) count[d] = static_cast<uint16_t>(rank[j] + __popc(same));
        __syncwarp(there);
      }
    }
    __syncthreads();
    if (tid < digits) {
      uint32_t sum = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = sh.count[w][tid];
        sh.count[w][tid] = static_cast<uint16_t>(sum);
        sum += c;
      }
      sh.total[tid] = sum;
    }
    cluster.sync();
    // Where digit d begins: all items of smaller digits, then the earlier CTAs' of d.
    uint32_t before = 0, all = 0;
    if (tid < digits) {
      for (int r = 0; r < ctas; ++r) {
        const uint32_t c = cluster.map_shared_rank(sh.total, r)[tid];
        if (r < me) before += c;
        all += c;
      }
    }
    uint32_t sum = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += v;
    }
    if (lane == 31) sh.scan[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      uint32_t v = sh.scan[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
      }
      sh.scan[lane] = v;
    }
    __syncthreads();
    if (tid < digits) sh.base[tid] = sum - all + (warp > 0 ? sh.scan[warp - 1] : 0) + before;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
      if (rank[j] >= 0) {
        const uint32_t d = (key[j] >> shift) & (digits - 1);
        const uint32_t to = sh.base[d] + sh.count[warp][d] + static_cast<uint32_t>(rank[j]);
        const uint32_t r = to / static_cast<uint32_t>(per_cta), i = to - r * static_cast<uint32_t>(per_cta);
        cluster.map_shared_rank(sh.key[from ^ 1], r)[i] = key[j];
        cluster.map_shared_rank(sh.pos[from ^ 1], r)[i] = sh.pos[from][warp * per_warp + 32 * j + lane];
      }
    }
    cluster.sync();  // every item has arrived, and nobody reads this CTA's totals any more
  }
  for (int i = tid; i < mine; i += kSortThreads) {
    p.keys[begin + i] = static_cast<int>(sh.key[from][i]);
    p.positions[begin + i] = sh.pos[from][i];
  }
}

cudaError_t prepare_embedding_kernels() {
  return cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortShared));
}

// ----------------------------------------------------------------------------
// Sums over equal tokens
// ----------------------------------------------------------------------------

constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;
constexpr int kAhead = 8;  // rows of dy in flight a warp

// A lane's columns of one row of dy: eight consecutive ones, or four 32 apart.
template <typename T, bool VEC>
struct Slab {
  static constexpr int N = VEC ? 8 : 4, kCols = 32 * N;
  __device__ static __forceinline__ int column(int slab, int lane, int e) {
    return VEC ? slab * kCols + lane * N + e : slab * kCols + 32 * e + lane;
  }
  __device__ static __forceinline__ void load(const T* row, int slab, int lane, int cols, float (&v)[N]) {
    if constexpr (VEC) {
      const int c = column(slab, lane, 0);
      if (c < cols) {
        load_wide<T, N>(row + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int c = column(slab, lane, e);
        v[e] = c < cols ? to_f32(row[c]) : 0.0f;
      }
    }
  }
};

// Adds scale * v to, or writes it to, a row of the gradient (16-byte accesses where VEC).
template <bool VEC, int N>
__device__ __forceinline__ void put_row(float* row, int slab, int lane, int cols, bool add, float scale, const float (&v)[N]) {
  if constexpr (VEC) {
    const int c = slab * 32 * N + lane * N;
    if (c >= cols) return;
    float o[N];
    if (add) load_wide<float, N>(row + c, o);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = add ? o[e] + v[e] * scale : v[e] * scale;
    store_wide<float, N>(row + c, o);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int c = slab * 32 * N + 32 * e + lane;
      if (c < cols) row[c] = add ? row[c] + v[e] * scale : v[e] * scale;
    }
  }
}

// Parts of tokens that cross pieces: [piece][0: goes on from the piece before, 1: starts here][padded columns].
template <int N>
__device__ __forceinline__ float* part_of(const EmbedGradParams& p, long long piece, int which, int slab, int lane) {
  return p.parts + (2 * piece + which) * p.ldparts + static_cast<long long>(slab) * 32 * N + lane * N;
}

// The first of `zero_blocks` blocks write the rows of the table that no token names; the others sum.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const __grid_constant__ EmbedGradParams p) {
  using S = Slab<T, VEC>;
  constexpr int N = S::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cols = static_cast<int>(p.cols);
  kernel_begin();
  if (blockIdx.x < p.zero_blocks) {
    // 32 rows a warp: each lane looks its row up in the sorted keys, then the warp writes the absent ones.
    const long long r0 = (static_cast<long long>(blockIdx.x) * kSumWarps + warp) * 32, r = r0 + lane;
    int lo = 0, hi = p.n;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.keys[mid] < r)
        lo = mid + 1;
      else
        hi = mid;
    }
    unsigned absent = __ballot_sync(0xffffffffu, r < p.vocab && !(lo < p.n && p.keys[lo] == r));
    while (absent != 0) {
      const int i = __ffs(static_cast<int>(absent)) - 1;
      absent &= absent - 1;
      float* row = p.grad + (r0 + i) * p.ldg;
      if constexpr (VEC) {
        for (int c = 4 * lane; c < cols; c += 128) *reinterpret_cast<float4*>(row + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      } else {
        for (int c = lane; c < cols; c += 32) row[c] = 0.0f;
      }
    }
    return;
  }
  const long long item = static_cast<long long>(blockIdx.x - p.zero_blocks) * kSumWarps + warp;
  const int piece = static_cast<int>(item / p.slabs), slab = static_cast<int>(item - static_cast<long long>(piece) * p.slabs);
  const int at = piece * p.piece;
  if (at >= p.n) return;
  const int here = p.n - at < p.piece ? p.n - at : p.piece;  // at most 32
  const int key = lane < here ? p.keys[at + lane] : -1;
  const int pos = lane < here ? p.positions[at + lane] : 0;
  const int before = at > 0 ? p.keys[at - 1] : -1, after = at + here < p.n ? p.keys[at + here] : -1;
  const T* dy = static_cast<const T*>(p.dy);
  float sum[N];
#pragma unroll
  for (int e = 0; e < N; ++e) sum[e] = 0.0f;
  const int vocab = static_cast<int>(p.vocab);
  bool whole = __shfl_sync(0xffffffffu, key, 0) != before;  // the token's rows began in this piece
  for (int i0 = 0; i0 < here; i0 += kAhead) {
    float v[kAhead][N];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = __shfl_sync(0xffffffffu, key, i0 + j);
      const long long q = __shfl_sync(0xffffffffu, pos, i0 + j);
      if (i0 + j < here && k < vocab) S::load(dy + (p.first + q) * p.lddy, slab, lane, cols, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = __shfl_sync(0xffffffffu, key, i0 + j);
      const int next = __shfl_sync(0xffffffffu, key, (i0 + j + 1) & 31);
      if (i0 + j < here && k < vocab) {
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] += v[j][e];
        const bool end_of_piece = i0 + j + 1 == here;
        if (!end_of_piece && next == k) continue;
        const bool goes_on = end_of_piece && after == k;
        if (whole && !goes_on) {
          put_row<VEC, N>(p.grad + static_cast<long long>(k) * p.ldg, slab, lane, cols, p.add != 0, p.scale, sum);
        } else {
          float* part = part_of<N>(p, piece, whole ? 1 : 0, slab, lane);
#pragma unroll
          for (int e = 0; e < N; e += 4) *reinterpret_cast<float4*>(part + e) = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
        }
        whole = true;
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] = 0.0f;
      }
    }
  }
}

// A token that starts in a piece and goes on: its part there, then the following pieces', in their order.
template <bool VEC>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const __grid_constant__ EmbedGradParams p) {
  constexpr int N = VEC ? 8 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  kernel_begin();
  const long long item = static_cast<long long>(blockIdx.x) * kSumWarps + warp;
  const int piece = static_cast<int>(item / p.slabs), slab = static_cast<int>(item - static_cast<long long>(piece) * p.slabs);
  const int at = piece * p.piece, end = at + p.piece;
  if (end >= p.n) return;  // the last piece goes nowhere
  const int key = p.keys[end - 1];
  if (key >= p.vocab || p.keys[end] != key) return;
  if (at > 0 && p.keys[at - 1] == key) return;  // a later part, joined from where the token starts
  // Pieces that the token reaches: 32 piece ends at a time.
  int last = piece + 1;
  for (;;) {
    const int q = last + lane, e = (q + 1) * p.piece;  // does the token fill piece q and go on?
    const unsigned on = __ballot_sync(0xffffffffu, e < p.n && p.keys[e] == key);
    const int run = on == 0xffffffffu ? 32 : __ffs(static_cast<int>(~on)) - 1;
    last += run;
    if (run < 32) break;
  }
  float sum[N];
  load_wide<float, N>(part_of<N>(p, piece, 1, slab, lane), sum);
  for (int q0 = piece + 1; q0 <= last; q0 += kAhead) {
    float v[kAhead][N];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (q0 + j <= last) load_wide<float, N>(part_of<N>(p, q0 + j, 0, slab, lane), v[j]);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (q0 + j <= last) {
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] += v[j][e];
      }
    }
  }
  put_row<VEC, N>(p.grad + static_cast<long long>(key) * p.ldg, slab, lane, static_cast<int>(p.cols), p.add != 0, p.scale, sum);
}

namespace {

template <typename T, bool VEC>
cudaError_t launch_sums(EmbedGradParams& p, cudaStream_t st) {
  constexpr int cols = Slab<T, VEC>::kCols;
  p.slabs = static_cast<int>((p.cols + cols - 1) / cols);
  p.ldparts = static_cast<long long>(p.slabs) * cols;
  const long long pieces = (p.n + p.piece - 1) / p.piece, items = pieces * p.slabs;
  const unsigned blocks = static_cast<unsigned>((items + kSumWarps - 1) / kSumWarps);
  p.zero_blocks = p.add ? 0 : static_cast<unsigned>((p.vocab + 32 * kSumWarps - 1) / (32 * kSumWarps));
  cudaError_t e = launch_overlapped(embed_sum_kernel<T, VEC>, p.zero_blocks + blocks, kSumThreads, 0, st, p);
  if (e != cudaSuccess || pieces <= 1) return e;
  return launch_overlapped(embed_join_kernel<VEC>, blocks, kSumThreads, 0, st, p);
}

template <typename T>
cudaError_t launch_sums_t(EmbedGradParams& p, cudaStream_t st) {
  const auto at = [](const void* q, long long ld, size_t size) {
    return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld * static_cast<long long>(size) % 16 == 0;
  };
  const bool vec = p.cols % 8 == 0 && at(p.dy, p.lddy, sizeof(T)) && at(p.grad, p.ldg, sizeof(float));
  return vec ? launch_sums<T, true>(p, st) : launch_sums<T, false>(p, st);
}

}  // namespace

cudaError_t launch_sort_tokens(const SortParams& p, cudaStream_t st) {
  SortParams q = p;
  int bits = 1;
  while ((p.vocab >> bits) != 0) ++bits;  // vocab itself is the key of tokens outside the table
  q.passes = (bits + kDigitBits - 1) / kDigitBits;
  q.bits = (bits + q.passes - 1) / q.passes;
  const int ctas = p.n <= kSortThreads ? 1 : p.n <= 2 * kSortThreads ? 2 : p.n <= 4 * kSortThreads ? 4 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = sizeof(SortShared);
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sort_tokens_kernel, q);
}

cudaError_t launch_embed_grad(EmbedGradParams& p, int dtype, cudaStream_t st) {
  if (dtype == kF32) return launch_sums_t<float>(p, st);
  return dtype == kBF16 ? launch_sums_t<__nv_bfloat16>(p, st) : launch_sums_t<__half>(p, st);
}

}  // namespace demo
