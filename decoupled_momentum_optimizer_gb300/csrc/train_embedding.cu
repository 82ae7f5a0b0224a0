// Rows of a table by token, scaled, and the gradient of the table:
//
//   out[i]    = scale table[t_i], zeros where t_i is outside [0, vocab)
//   dtable[v] = scale sum_{i: t_i = v} dy[i]   (added to what it holds, or 0 for rows without a token)
//
// The lookup is bound by HBM and, for a few tokens, by two dependent loads.
//
// The gradient sums in a fixed order without atomics.  Tokens are sorted by value, equal ones by position, in
// the shared memory of one cluster; the sorted list is cut into pieces of 8, 16 or 32 positions, and a warp sums
// the rows of one piece over 256 columns, writing each token's sum as it ends.  A token that goes
// on past its piece leaves its part in the workspace (at most one at either end of a piece), and a second
// kernel adds a token's parts in the order of the pieces.  Words are spread as 1 / rank, so one row of the
// table may take a tenth of all positions: cutting by position, not by token, keeps the warps' work equal.
//
// 16384 positions of bfloat16 added to 100352 x 2048: 51 us, 13 of them the sort (its launch, and two passes of
// barriers and remote stores on eight SMs, with the others idle) and 38 the sums, 177 MB that cannot be done
// without (26 us).  Written anew 138 us, 889 MB (131 us): zeros beside the sort, and beside the sums where no token
// is.  4096 positions into 32128 x 768 anew 26 us, 105 MB (15).  (L2 asked for dy by the idle SMs during the sort: no
// difference.)
#include <cooperative_groups.h>

#include "train_norm.cuh"

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

// 16384 x 2048 into bfloat16 20.5 us (122 MB that cannot be done without: 17.9), two accesses of one row 22.9; 65536 x
// 768 25.2 us and 31.  Rows off 16 bytes, by accesses of one element: 16384 x 2051 71 us, 65536 x 765 100 (floors 17.9, 21.9).
constexpr int kLookThreads = 128, kLookRows = 4;

// A thread takes eight columns of kLookRows rows as 16-byte accesses, or (rows off 16 bytes) a warp 128 columns of
// one row, four a lane.
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kLookThreads) lookup_kernel(const __grid_constant__ LookupParams p, long long per_row) {
  kernel_begin();
  const T* table = static_cast<const T*>(p.table);
  O* out = static_cast<O*>(p.out);
  const auto row_of = [&](long long u) {
    return u < (1ll << 32) ? static_cast<long long>(static_cast<uint32_t>(u) / static_cast<uint32_t>(per_row)) : u / per_row;
  };
  if constexpr (VEC) {
    const long long u = static_cast<long long>(blockIdx.x) * kLookThreads + threadIdx.x;
    const long long group = row_of(u), row0 = group * kLookRows, col = (u - group * per_row) * 8;
    float v[kLookRows][8];
    long long t[kLookRows];
#pragma unroll
    for (int j = 0; j < kLookRows; ++j) t[j] = row0 + j < p.n ? token_at(p.tokens, row0 + j) : -1;
#pragma unroll
    for (int j = 0; j < kLookRows; ++j) {
      if (t[j] >= 0 && t[j] < p.vocab) {
        load_wide<T, 8>(table + t[j] * p.ldt + col, v[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < kLookRows; ++j) {
      if (row0 + j >= p.n) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] *= p.scale;
      store_wide<O, 8>(out + (row0 + j) * p.ldo + col, v[j]);
    }
  } else {
    const long long u = static_cast<long long>(blockIdx.x) * (kLookThreads / 32) + (threadIdx.x >> 5);
    if (u >= p.n * per_row) return;
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
    const long long per = p.cols / 8, units = (p.n + kLookRows - 1) / kLookRows * per;
    return launch_overlapped(lookup_kernel<T, O, true>, static_cast<unsigned>((units + kLookThreads - 1) / kLookThreads),
                             kLookThreads, 0, st, p, per);
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
// digits (lanes with the same digit find each other by a ballot for each of its bits and take consecutive
// ranks; a match instruction takes a step for each different digit: 8 us for 16384 tokens), the warps' counts
// become offsets within the CTA, the CTAs exchange their totals through distributed shared memory, and every
// item goes straight to its place in the CTA that will hold it.  Up to 2^16 tokens: 8 CTAs x 1024 threads x 8.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortRounds = 8;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
static_assert(kMaxSorted == 8 * kSortThreads * kSortRounds, "capacity of the largest cluster");
static_assert(kMaxSorted <= 65536, "positions are 16 bits");
static_assert(kDigits <= kSortThreads, "a thread for each digit");

struct SortShared {
  uint64_t item[2][kSortThreads * kSortRounds];  // token << 16 | position
  uint16_t count[kSortWarps][kDigits];  // of a warp's items, then the warps' before it
  uint32_t total[kDigits];              // of the CTA
  uint32_t base[kDigits];               // where the CTA's items of a digit begin
  uint32_t scan[kSortWarps];
};

// Writes 0 to the first `filled` rows of the table, `part` of `parts`.
__device__ __forceinline__ void fill_rows(const SortParams& p, long long part, long long parts) {
  if (p.ldg == p.cols) {  // one run of floats: whole 16-byte accesses, and what is off them at either end
    float* base = p.grad;
    const long long total = p.filled * p.cols, head = (4 - (reinterpret_cast<uintptr_t>(base) / 4 & 3)) & 3;
    const long long first = head < total ? head : total, units = (total - first) / 4;
    for (long long u = part * kSortThreads + threadIdx.x; u < units; u += parts * kSortThreads)
      reinterpret_cast<float4*>(base + first)[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (part == 0) {
      if (threadIdx.x < first) base[threadIdx.x] = 0.0f;
      const long long tail = first + 4 * units + threadIdx.x;
      if (tail < total && threadIdx.x < 4) base[tail] = 0.0f;
    }
    return;
  }
  const int lane = threadIdx.x & 31;
  const bool wide = p.cols % 4 == 0 && p.ldg % 4 == 0 && (reinterpret_cast<uintptr_t>(p.grad) & 15) == 0;
  for (long long r = part * kSortWarps + (threadIdx.x >> 5); r < p.filled; r += parts * kSortWarps) {
    float* row = p.grad + r * p.ldg;
    if (wide) {
      for (long long c = 4 * lane; c < p.cols; c += 128) *reinterpret_cast<float4*>(row + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    } else {
      for (long long c = lane; c < p.cols; c += 32) row[c] = 0.0f;
    }
  }
}

// The first cluster sorts.  Where the table's gradient is written anew, the other SMs fill its first rows with
// zeros meanwhile, as many as the sort takes time for (the sums then overwrite those that have tokens).
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
  if (blockIdx.x >= static_cast<unsigned>(ctas)) {
    fill_rows(p, blockIdx.x - ctas, gridDim.x - ctas);
    return;
  }
  for (int i = tid; i < mine; i += kSortThreads) {
    const long long t = token_at(p.tokens, p.first + begin + i);
    sh.item[0][i] = static_cast<uint64_t>(t >= 0 && t < p.vocab ? t : p.vocab) << 16 | (begin + i);  // others last
  }
  int from = 0;
  for (int pass = 0; pass < p.passes; ++pass, from ^= 1) {
    const int shift = 16 + pass * p.bits, digits = 1 << p.bits;
    for (int i = tid; i < kSortWarps * kDigits / 2; i += kSortThreads) reinterpret_cast<uint32_t*>(sh.count)[i] = 0;
    __syncthreads();  // counts cleared; and, in the first pass, the items are there
    uint64_t item[kSortRounds];
    int rank[kSortRounds];
    uint16_t* count = sh.count[warp];
#pragma unroll
    for (int j = 0; j < kSortRounds; ++j) {
      const int in_warp = 32 * j + lane, i = warp * per_warp + in_warp;
      const bool live = in_warp < per_warp && i < mine;
      rank[j] = -1;
      const unsigned there = __ballot_sync(0xffffffffu, live);
      if (there == 0) continue;
      item[j] = live ? sh.item[from][i] : 0;
      const uint32_t d = static_cast<uint32_t>(item[j] >> shift) & (digits - 1);
      unsigned same = there;
      for (int b = 0; b < p.bits; ++b) {
        const bool one = d >> b & 1;
        const unsigned ones = __ballot_sync(0xffffffffu, one);
        same &= one ? ones : ~ones;
      }
      const int before = __popc(same & ((1u << lane) - 1));
      if (live) rank[j] = count[d] + before;
      __syncwarp();
      if (live && before == 0) count[d] = static_cast<uint16_t>(rank[j] + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    if (tid < digits) {
      uint32_t c[kSortWarps], sum = 0;  // all read before any is written
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = sh.count[w][tid];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        sh.count[w][tid] = static_cast<uint16_t>(sum);
        sum += c[w];
      }
      sh.total[tid] = sum;
    }
    cluster.sync();
    // Where digit d begins: all items of smaller digits, then the earlier CTAs' of d.
    uint32_t before = 0, all = 0;
    if (tid < digits) {
      uint32_t c[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) c[r] = r < ctas ? cluster.map_shared_rank(sh.total, r)[tid] : 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (r < me) before += c[r];
        all += c[r];
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
        const uint32_t d = static_cast<uint32_t>(item[j] >> shift) & (digits - 1);
        const uint32_t to = sh.base[d] + sh.count[warp][d] + static_cast<uint32_t>(rank[j]);
        const uint32_t r = to / static_cast<uint32_t>(per_cta), i = to - r * static_cast<uint32_t>(per_cta);
        cluster.map_shared_rank(sh.item[from ^ 1], r)[i] = item[j];
      }
    }
    cluster.sync();  // every item has arrived, and nobody reads this CTA's totals any more
  }
  for (int i = tid; i < mine; i += kSortThreads) {
    const uint64_t v = sh.item[from][i];
    p.keys[begin + i] = static_cast<int>(v >> 16);
    p.positions[begin + i] = static_cast<unsigned short>(v);
  }
}

cudaError_t prepare_embedding_kernels() {
  return cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SortShared));
}

// ----------------------------------------------------------------------------
// Sums over equal tokens
// ----------------------------------------------------------------------------

constexpr int kSumThreads = 128, kSumWarps = kSumThreads / 32;
constexpr int kAhead = 4;     // rows of dy, and of the gradient that is added to, in flight a warp
constexpr int kAheadFew = 8;  // the same where few warps run: 26 positions 6.6 us, with four 7.2

// A warp's columns of a row: eight a lane as 16-byte accesses, or four a lane 32 apart.
template <bool VEC>
constexpr int kSlabN = VEC ? 8 : 4;

template <bool VEC, int N>
__device__ __forceinline__ void put_row(float* row, const Place& at, const F2 (&v)[N / 2]) {
  if constexpr (VEC) {
    if (at.reach > 0) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i)
        reinterpret_cast<float4*>(row)[i] = make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (at.has<VEC, N>(0, e)) row[32 * e] = e % 2 ? v[e / 2].y : v[e / 2].x;
  }
}

// Parts of tokens that cross pieces: [piece][0: goes on from the piece before, 1: starts here][padded columns],
// a lane's N side by side.
template <int N>
__device__ __forceinline__ float* part_of(const EmbedGradParams& p, long long piece, int which, int slab, int lane) {
  return p.parts + (2 * piece + which) * p.ldparts + static_cast<long long>(slab) * 32 * N + lane * N;
}
template <int N>
__device__ __forceinline__ void add_part(const float4 (&v)[N / 4], F2 (&sum)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    sum[2 * i] = add2(sum[2 * i], f2(v[i].x, v[i].y));
    sum[2 * i + 1] = add2(sum[2 * i + 1], f2(v[i].z, v[i].w));
  }
}
template <int N>
__device__ __forceinline__ void read_part(const float* part, float4 (&v)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) v[i] = reinterpret_cast<const float4*>(part)[i];
}

// scale * sum, added to what the row holds if asked.
template <bool VEC, int N>
__device__ __forceinline__ void finish_row(const EmbedGradParams& p, long long token, const Place& at, F2 (&sum)[N / 2]) {
  float* row = p.grad + token * p.ldg + at.first;
  Unit<float, VEC, N> old;
  if (p.add) old.load(row, at, 0);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    sum[i] = mul2(sum[i], f2(p.scale, p.scale));
    if (p.add) sum[i] = add2(old.get2(i), sum[i]);
  }
  put_row<VEC, N>(row, at, sum);
}

enum : int { kEnds = 1 << 16, kFinal = 1 << 17, kStarts = 1 << 18, kLive = 1 << 19 };

constexpr int kZeroCols = 1024;  // columns of a warp's rows that it zeroes

// Writes 0 to columns c0 .. c0 + kZeroCols - 1 of a warp's rows r0 + (the set bits).
template <bool VEC>
__device__ __forceinline__ void zero_rows(const EmbedGradParams& p, long long r0, unsigned rows, int c0, int lane) {
  const int end = p.cols - c0 < kZeroCols ? static_cast<int>(p.cols) : c0 + kZeroCols;
  // all of them, end to end from a 16-byte boundary: whole accesses whatever the width
  float* run = p.grad + r0 * p.ldg;
  if (rows == 0xffffffffu >> (32 - p.zero_rows) && p.cols <= kZeroCols && p.ldg == p.cols &&
      (reinterpret_cast<uintptr_t>(run) & 15) == 0) {
    for (long long u = lane; u < p.zero_rows * p.cols / 4; u += 32) reinterpret_cast<float4*>(run)[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    return;
  }
  while (rows != 0) {
    const int i = __ffs(static_cast<int>(rows)) - 1;
    rows &= rows - 1;
    float* row = p.grad + (r0 + i) * p.ldg;
    if constexpr (VEC) {
      for (int c = c0 + 4 * lane; c < end; c += 128) *reinterpret_cast<float4*>(row + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    } else {
      for (int c = c0 + lane; c < end; c += 32) row[c] = 0.0f;
    }
  }
}

// The sums of up to 32 sorted positions: lane i holds entry i's token and position; `before` and `after` are the
// tokens around them.
template <typename T, bool VEC, int AHEAD>
__device__ __forceinline__ void sum_entries(const EmbedGradParams& p, int key, int info, int here, int before, int after,
                                            int piece, int slab, int lane) {
  constexpr int N = kSlabN<VEC>;
  const Place at = Place::of<VEC, N>(slab, 1, lane, 32, static_cast<int>(p.cols));
  const int next = __shfl_down_sync(0xffffffffu, key, 1);
  if (lane < here && key < p.vocab) {
    info |= kLive;
    const bool ends = lane == here - 1 || next != key;
    if (key != before) info |= kStarts;
    if (ends) info |= kEnds;
    if (ends && key != before && key != after) info |= kFinal;
  }
  const T* dy = static_cast<const T*>(p.dy) + at.first;
  F2 sum[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) sum[i] = f2(0.0f, 0.0f);
  for (int i0 = 0; i0 < here; i0 += AHEAD) {
    Unit<T, VEC, N> v[AHEAD];
    Unit<float, VEC, N> old[AHEAD];
    int what[AHEAD];
    float* row[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      what[j] = __shfl_sync(0xffffffffu, info, i0 + j);
      row[j] = p.grad + static_cast<long long>(__shfl_sync(0xffffffffu, key, i0 + j)) * p.ldg + at.first;
      if (what[j] & kLive) v[j].load(dy + (p.first + (what[j] & 0xffff)) * p.lddy, at, 0);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (p.add && (what[j] & kFinal)) old[j].load(row[j], at, 0);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (!(what[j] & kLive)) continue;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) sum[i] = add2(sum[i], v[j].get2(i));
      if (!(what[j] & kEnds)) continue;
      if (what[j] & kFinal) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          sum[i] = mul2(sum[i], f2(p.scale, p.scale));
          if (p.add) sum[i] = add2(old[j].get2(i), sum[i]);
        }
        put_row<VEC, N>(row[j], at, sum);
      } else {
        float4* part = reinterpret_cast<float4*>(part_of<N>(p, piece, what[j] & kStarts ? 1 : 0, slab, lane));
#pragma unroll
        for (int i = 0; i < N / 4; ++i) part[i] = make_float4(sum[2 * i].x, sum[2 * i].y, sum[2 * i + 1].x, sum[2 * i + 1].y);
      }
#pragma unroll
      for (int i = 0; i < N / 2; ++i) sum[i] = f2(0.0f, 0.0f);
    }
  }
}

// The first of the sorted keys lo .. hi - 1 that is not below `row`, hi if none: a warp looks at 32 at a time.
__device__ __forceinline__ int first_key(const int* keys, int lo, int hi, long long row, int lane) {
  while (lo < hi) {
    const int step = (hi - lo + 32) / 33, at = lo + (lane + 1) * step - 1;  // the last of 32 runs of `step`
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && keys[at] < row);
    const int runs = __popc(below);
    lo += runs * step;
    if (step == 1 && runs < 32) break;
    if (runs < 32 && lo + step - 1 < hi) hi = lo + step - 1;
  }
  return lo;
}

// A warp sums one piece over one slab of columns.  What becomes of an entry follows from its key and those around
// the piece, so every row that a batch needs is asked for at once: the rows of dy, and those of the gradient
// that a token's sum is added to.  Blocks behind those write 0 to the rows that no token names, from `zero_from` on.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kSumThreads, 4) embed_sum_kernel(const __grid_constant__ EmbedGradParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  kernel_begin();
  if (blockIdx.x >= p.sum_blocks) {
    // A few rows a warp: it finds their part of the sorted keys, each lane its row there; then it writes the absent ones.
    const long long z = static_cast<long long>(blockIdx.x - p.sum_blocks) * kSumWarps + warp, group = z / p.zero_slabs;
    const long long r0 = p.zero_from + group * p.zero_rows, r = r0 + lane;
    int lo = first_key(p.keys, 0, p.n, r0, lane);
    const int end = first_key(p.keys, lo, p.n, r0 + p.zero_rows, lane);
    for (int hi = end; lo < hi;) {
      const int mid = (lo + hi) / 2;
      if (p.keys[mid] < r)
        lo = mid + 1;
      else
        hi = mid;
    }
    zero_rows<VEC>(p, r0, __ballot_sync(0xffffffffu, lane < p.zero_rows && r < p.vocab && !(lo < end && p.keys[lo] == r)),
                   static_cast<int>(z - group * p.zero_slabs) * kZeroCols, lane);
    return;
  }
  const long long item = static_cast<long long>(blockIdx.x) * kSumWarps + warp;
  const int piece = static_cast<int>(item / p.slabs), slab = static_cast<int>(item - static_cast<long long>(piece) * p.slabs);
  const int begin = piece * p.piece;
  if (begin >= p.n) return;
  const int here = p.n - begin < p.piece ? p.n - begin : p.piece;  // at most 32
  const int key = lane < here ? p.keys[begin + lane] : -1;
  const int pos = lane < here ? p.positions[begin + lane] : 0;
  const int before = begin > 0 ? p.keys[begin - 1] : -1, after = begin + here < p.n ? p.keys[begin + here] : -1;
  sum_entries<T, VEC, kAhead>(p, key, pos, here, before, after, piece, slab, lane);
}

// Up to 32 positions in one kernel: every warp sorts them itself (a token's place is the number of those before it),
// and finds the rows that none names by comparing.  A call of 26 positions: two launches and a workspace less.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kSumThreads) embed_few_kernel(const __grid_constant__ EmbedGradParams p,
                                                                const __grid_constant__ Tokens tokens) {
  __shared__ int keys[kSumWarps][32], positions[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  kernel_begin();
  const long long t = lane < p.n ? token_at(tokens, lane) : -1;
  const int key = t >= 0 && t < p.vocab ? static_cast<int>(t) : static_cast<int>(p.vocab);  // others last
  if (blockIdx.x >= p.sum_blocks) {
    const long long z = static_cast<long long>(blockIdx.x - p.sum_blocks) * kSumWarps + warp, group = z / p.zero_slabs;
    const long long r0 = group * p.zero_rows, r = r0 + lane;
    bool named = false;
    for (int j = 0; j < p.n; ++j) named |= __shfl_sync(0xffffffffu, key, j) == r;
    zero_rows<VEC>(p, r0, __ballot_sync(0xffffffffu, lane < p.zero_rows && r < p.vocab && !named),
                   static_cast<int>(z - group * p.zero_slabs) * kZeroCols, lane);
    return;
  }
  const int slab = static_cast<int>(blockIdx.x) * kSumWarps + warp;
  if (slab >= p.slabs) return;
  int place = 0;
  for (int j = 0; j < p.n; ++j) {
    const int other = __shfl_sync(0xffffffffu, key, j);
    place += other < key || (other == key && j < lane);
  }
  if (lane < p.n) {
    keys[warp][place] = key;
    positions[warp][place] = lane;
  }
  __syncwarp();
  sum_entries<T, VEC, kAheadFew>(p, lane < p.n ? keys[warp][lane] : -1, lane < p.n ? positions[warp][lane] : 0, p.n, -1, -1, 0, slab, lane);
}

// A token that starts in a piece and goes on: its part there, then the following pieces', in their order.  A
// warp finds where a piece's last token ends; few parts it adds alone, of many every warp of the CTA takes
// every sixteenth (one token in 5461 of 16384 positions took 68 us with one warp).
constexpr int kJoinWarps = 16, kAlone = 16;
constexpr int kJoinAhead = 4;

template <bool VEC>
__global__ void __launch_bounds__(32 * kJoinWarps) embed_join_kernel(const __grid_constant__ EmbedGradParams p) {
  constexpr int N = kSlabN<VEC>;
  __shared__ __align__(16) float sums[kJoinWarps][32 * N];
  __shared__ int2 run[kJoinWarps];  // token and last piece of a long run
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  kernel_begin();
  const int group = static_cast<int>(blockIdx.x / p.slabs), slab = static_cast<int>(blockIdx.x - static_cast<unsigned>(group) * p.slabs);
  const Place at = Place::of<VEC, N>(slab, 1, lane, 32, static_cast<int>(p.cols));
  // Parts q0, q0 + step, ... of a token, up to the last.
  const auto add_parts = [&](int q0, int step, int last, F2(&sum)[N / 2]) {
    for (int q = q0; q <= last; q += kJoinAhead * step) {
      float4 v[kJoinAhead][N / 4];
#pragma unroll
      for (int j = 0; j < kJoinAhead; ++j)
        if (q + j * step <= last) read_part<N>(part_of<N>(p, q + j * step, 0, slab, lane), v[j]);
#pragma unroll
      for (int j = 0; j < kJoinAhead; ++j)
        if (q + j * step <= last) add_part<N>(v[j], sum);
    }
  };
  const int mine = group * kJoinWarps + warp, begin = mine * p.piece, end = begin + p.piece;
  int last = -1, key = -1;
  if (end < p.n) {  // the last piece goes nowhere
    key = p.keys[end - 1];
    // A token outside the table has no sum; one that began before is joined from where it did.
    if (key < p.vocab && p.keys[end] == key && (begin == 0 || p.keys[begin - 1] != key)) {
      last = mine + 1;
      for (;;) {  // pieces that the token reaches, 32 piece ends at a time
        const int e = (last + lane + 1) * p.piece;  // does the token fill this piece and go on?
        const unsigned on = __ballot_sync(0xffffffffu, e < p.n && p.keys[e] == key);
        const int filled = on == 0xffffffffu ? 32 : __ffs(static_cast<int>(~on)) - 1;
        last += filled;
        if (filled < 32) break;
      }
    }
  }
  const bool alone = last >= 0 && last - mine <= kAlone;
  if (lane == 0) run[warp] = alone ? make_int2(-1, -1) : make_int2(key, last);
  if (alone) {
    F2 sum[N / 2];
    float4 v[N / 4];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) sum[i] = f2(0.0f, 0.0f);
    read_part<N>(part_of<N>(p, mine, 1, slab, lane), v);
    add_part<N>(v, sum);
    add_parts(mine + 1, 1, last, sum);
    finish_row<VEC, N>(p, key, at, sum);
  }
  __syncthreads();
  for (int w = 0; w < kJoinWarps; ++w) {
    if (run[w].y < 0) continue;  // the same for the CTA
    const int from = group * kJoinWarps + w;
    F2 sum[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) sum[i] = f2(0.0f, 0.0f);
    if (warp == 0) {
      float4 v[N / 4];
      read_part<N>(part_of<N>(p, from, 1, slab, lane), v);
      add_part<N>(v, sum);
    }
    add_parts(from + 1 + warp, kJoinWarps, run[w].y, sum);
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4*>(&sums[warp][lane * N])[i] = make_float4(sum[2 * i].x, sum[2 * i].y, sum[2 * i + 1].x, sum[2 * i + 1].y);
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 1; k < kJoinWarps; ++k) {
        float4 v[N / 4];
        read_part<N>(&sums[k][lane * N], v);
        add_part<N>(v, sum);
      }
      finish_row<VEC, N>(p, run[w].x, at, sum);
    }
    __syncthreads();
  }
}

namespace {

// Blocks that zero rows from `from` on; sets what their warps take: 4, 8, 16 or 32 rows of up to 1024 columns, 16 to 32 KB
// from 128 columns on, less where rows are narrower or a wide row's last columns are few.  4096 positions into 32128 x
// 768 25.6 us, 16384 into 100352 x 2048 138; warps with 1024 columns of 32 rows 42 and 146 (a few long ones are left at the
// end), with 128 columns of them 27 and 155 (pieces of 512 bytes).
unsigned zero_blocks(EmbedGradParams& p, long long from) {
  p.zero_rows = p.cols >= 1024 ? 4 : p.cols >= 512 ? 8 : p.cols >= 256 ? 16 : 32;
  p.zero_slabs = static_cast<int>((p.cols + kZeroCols - 1) / kZeroCols);
  const long long warps = from < p.vocab ? (p.vocab - from + p.zero_rows - 1) / p.zero_rows * p.zero_slabs : 0;
  return static_cast<unsigned>((warps + kSumWarps - 1) / kSumWarps);
}

template <typename T, bool VEC>
cudaError_t launch_sums(EmbedGradParams& p, const Tokens& tokens, cudaStream_t st) {
  constexpr int cols = 32 * kSlabN<VEC>;
  p.slabs = static_cast<int>((p.cols + cols - 1) / cols);
  if (p.keys == nullptr) {  // few positions, not sorted
    p.sum_blocks = static_cast<unsigned>((p.slabs + kSumWarps - 1) / kSumWarps);
    return launch_overlapped(embed_few_kernel<T, VEC>, p.sum_blocks + zero_blocks(p, p.add ? p.vocab : 0), kSumThreads,
                             0, st, p, tokens);
  }
  p.ldparts = static_cast<long long>(p.slabs) * cols;
  const long long pieces = (p.n + p.piece - 1) / p.piece, items = pieces * p.slabs;
  p.sum_blocks = static_cast<unsigned>((items + kSumWarps - 1) / kSumWarps);
  const unsigned zero = zero_blocks(p, p.zero_from);
  const cudaError_t e = launch_overlapped(embed_sum_kernel<T, VEC>, p.sum_blocks + zero, kSumThreads, 0, st, p);
  if (e != cudaSuccess || pieces <= 1) return e;
  return launch_overlapped(embed_join_kernel<VEC>, static_cast<unsigned>((pieces + kJoinWarps - 1) / kJoinWarps * p.slabs),
                           32 * kJoinWarps, 0, st, p);
}

template <typename T>
cudaError_t launch_sums_t(EmbedGradParams& p, const Tokens& tokens, cudaStream_t st) {
  const auto at = [](const void* q, long long ld, size_t size) {
    return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld * static_cast<long long>(size) % 16 == 0;
  };
  const bool vec = p.cols % 8 == 0 && at(p.dy, p.lddy, sizeof(T)) && at(p.grad, p.ldg, sizeof(float));
  return vec ? launch_sums<T, true>(p, tokens, st) : launch_sums<T, false>(p, tokens, st);
}

}  // namespace

cudaError_t launch_sort_tokens(const SortParams& p, int sms, cudaStream_t st) {
  SortParams q = p;
  int bits = 1;
  while ((p.vocab >> bits) != 0) ++bits;  // vocab itself is the key of tokens outside the table
  q.passes = (bits + kDigitBits - 1) / kDigitBits;
  q.bits = (bits + q.passes - 1) / q.passes;
  // Two rounds of 32 a warp (16384 tokens: 13 us; with eight rounds, in two CTAs, 22).
  const int each = 2 * kSortThreads;
  const int ctas = p.n <= each ? 1 : p.n <= 2 * each ? 2 : p.n <= 4 * each ? 4 : 8;
  cudaLaunchConfig_t cfg = {};
  // Three quarters of the SMs fill (clusters of eight do not fit on all of them at one time), 64 KB each at least.
  long long fill = 0;
  if (p.filled > 0) {
    const long long worth = (p.filled * p.cols + 16383) / 16384, most = sms * 3 / 4 / ctas - 1;
    fill = (worth + ctas - 1) / ctas;
    fill = fill < 1 || most < 1 ? 1 : fill < most ? fill : most;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(ctas * (1 + fill)));
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

cudaError_t launch_embed_grad(EmbedGradParams& p, const Tokens& tokens, int dtype, cudaStream_t st) {
  if (dtype == kF32) return launch_sums_t<float>(p, tokens, st);
  return dtype == kBF16 ? launch_sums_t<__nv_bfloat16>(p, tokens, st) : launch_sums_t<__half>(p, tokens, st);
}

}  // namespace demo
