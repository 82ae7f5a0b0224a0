// Parameter blocks and launchers of the training operators' kernels (dropout, block-scaled 8-bit
// quantization, products of quantized matrices, norms), and what their C entry points need of the
// library's per-device state.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "train_embed_plan.h"
#include "train_plan.h"

namespace demo {

enum { kF32 = 0, kBF16 = 1, kF16 = 2 };
enum { kE4M3 = 0, kE5M2 = 1 };

// Exponent of each format's largest finite code, 1.75 * 2^top (448 and 57344).
__host__ __device__ constexpr int fmt_top(int fmt) { return fmt == kE4M3 ? 8 : 15; }

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The initialised current device; returns a status of include/demo.h.
struct DeviceInfo {
  int sms;
  unsigned int* fault;
  EncodeTiledFn encode;
  const Clusters* clusters;
};
int device_info(DeviceInfo* out);
// Test hook of the bounded waits (demo_test_stall_next_launch): 1 + the load of the next launch's first
// CTA that shall never complete, 0 for none; taken (and cleared) by the launch.
long long take_stall();

struct DropParams {
  unsigned long long key;  // sm(sm(sm(seed) ^ step) ^ site)
  unsigned int threshold;
  float scale;
};

struct DropoutParams {
  const void* x;
  const void* residual;  // may be NULL
  void* out;
  long long rows, cols, ldx, ldr, ldo;
  DropParams drop;
};

cudaError_t launch_dropout(const DropoutParams& p, int dtype, cudaStream_t st);

struct QuantParams {
  const void* x;
  const void* gate;  // may be NULL
  long long rows, cols, ldx, ldg;
  unsigned int row_blocks, col_blocks;  // of 128; their product is the grid
  int relu, tiles;
  DropParams drop;
  void* codes_rows;    // [rows][cols up to 128], may be NULL
  float* scales_rows;  // [column blocks][rows up to 4]
  void* codes_cols;    // [cols][rows up to 128], may be NULL
  float* scales_cols;  // [row blocks][cols up to 4]
  const float* rstd;   // NULL, or x is (x rstd[row]) weight[column] first (see train_norm.cu)
  const void* weight;
  int weight_dtype;
};

cudaError_t launch_quantize(const QuantParams& p, int dtype, int fmt, cudaStream_t st);

// Root-mean-square norm of rows (see train_norm.cu).  inv = 1 / cols; it and eps also as pairs of floats.
constexpr long long kNormCols = 32768;  // 32 warps of 32 elements a lane
struct NormParams {
  const void* x;
  const void* residual;  // may be NULL
  const void* weight;
  void* total;  // x + residual, may be NULL
  void* out;    // may be NULL
  float* rstd;  // may be NULL
  void* codes;  // by rows, may be NULL
  float* scales;
  long long rows, cols, ldx, ldr, ldt, ldo;
  unsigned int col_blocks;
  int fmt, warps, per, lanes;  // warps of a row, units of a warp, lanes of a short row: set by the launcher
  float inv_hi, inv_lo, eps_hi, eps_lo;
  double inv, eps;
};
cudaError_t launch_norm(NormParams& p, int dtype, int weight_dtype, int sms, cudaStream_t st);

constexpr int kNormParts = 256;  // most CTAs of the gradient's kernel, whose sums over rows a second one joins
struct NormGradParams {
  const void* dy;
  const void* total;
  const void* weight;
  const float* rstd;
  const void* past;  // may be NULL
  void* dx;
  float* dw;        // may be NULL
  float* partials;  // [CTAs][cols], unused with one CTA
  long long rows, cols, lddy, ldt, ldp, lddx;
  int add, warps, per, lanes;  // warps of a row, units of a warp, lanes of a short row: set by the launcher
  float inv;
};
cudaError_t launch_norm_grad(NormGradParams& p, int dtype, int weight_dtype, int sms, cudaStream_t st);

// Token tables (see train_embedding.cu).  Tokens are `per` consecutive ones in rows `ld` apart, 4 or 8 bytes each.
struct Tokens {
  const void* p;
  long long per, ld;
  int wide;
};
struct LookupParams {
  Tokens tokens;
  const void* table;
  void* out;
  long long n, vocab, cols, ldt, ldo;
  float scale;
};
cudaError_t launch_lookup(const LookupParams& p, int table_dtype, int out_dtype, cudaStream_t st);

constexpr int kMaxSorted = 65536;  // tokens that one cluster sorts
struct SortParams {
  Tokens tokens;
  long long first, vocab;  // the first token's flat position
  int n, passes, bits;     // passes over digits of `bits`: set by the launcher
  int* keys;               // [n] sorted; vocab stands for tokens outside the table
  unsigned short* positions;  // [n], from the first token on
  float* grad;                // the table's gradient, whose first `filled` rows are filled with zeros meanwhile
  long long cols, ldg, filled;
};
cudaError_t launch_sort_tokens(const SortParams& p, int sms, cudaStream_t st);
constexpr int kFewTokens = 32;  // positions that need no sort before the sums
struct EmbedGradParams {
  const int* keys;  // NULL: few positions, taken from the tokens themselves
  const unsigned short* positions;
  const void* dy;
  float* grad;
  float* parts;  // [pieces][2][ldparts]
  long long first, vocab, cols, lddy, ldg, ldparts;
  long long zero_from;  // rows from here on that no token names are written 0; vocab for none
  unsigned int sum_blocks;
  int zero_rows, zero_slabs;  // rows that warps share (4 to 32), and those warps
  int n, piece, slabs, add;  // piece: 8, 16 or 32
  float scale;
};
cudaError_t launch_embed_grad(EmbedGradParams& p, const Tokens& tokens, int dtype, cudaStream_t st);
cudaError_t prepare_embedding_kernels();

// The gradients' norm and their scaling (see train_clip.cu): a launch takes up to CAP tensors.  The block is copied
// with every launch (14 KB for 512 tensors), so short lists have a smaller one.
template <int CAP>
struct ClipParams {
  const void* g[CAP];
  void* out[CAP];
  long long n[CAP];
  unsigned int start[CAP];  // the tensor's first chunk; empty tensors are left out
  int count, part_count;
  unsigned int chunks;
  int given, first_launch, in_place, only_norm;
  double max_norm;
  double* parts;            // this launch's sums
  const double* all_parts;  // every launch's
  float* norm;
};
constexpr int kClipTensors = 512, kClipFew = 64;
constexpr int kClipParts = 640;  // most CTAs of a launch, each of which leaves a sum
long long clip_chunks(uintptr_t address, long long n, int size);  // chunks of a tensor
int clip_parts(unsigned chunks, int dtype, int sms);              // CTAs of a launch
// Norm and scaling of at most kSmallChunks chunks in one launch (the norm alone: `only_norm`).  us with one launch / with
// two, float32 from L2; "clipped": into other tensors, "unclipped": in place, nothing to scale:
//                             norm, called   from a graph  clipped, called  from a graph  unclipped, called  from a graph
//   1 chunk, 1 tensor         4.1 / 6.2      3.9 / 4.3     5.6 / 6.7        5.4 / 6.4     4.2 / 6.5          4.0 / 5.0
//   16 chunks, 1 tensor       4.8 / 6.1      4.5 / 4.2     6.9 / 7.1        6.6 / 6.4     4.9 / 6.4          4.6 / 5.0
//   17 chunks, 17 tensors     6.0 / 7.0      5.5 / 4.4     9.3 / 8.0        8.9 / 7.0     6.1 / 7.4          5.6 / 5.3
//   32 chunks, 1 tensor       5.5 / 6.0      5.2 / 4.2     8.9 / 7.4        8.6 / 6.5     5.6 / 6.4          5.3 / 5.3
//   57 chunks, 57 tensors     8.0 / 7.8      7.6 / 4.6     13.4 / 10.5      13.0 / 7.0    8.1 / 9.6          7.7 / 5.6
//   64 chunks, 1 tensor       6.7 / 6.1      6.4 / 4.2     12.6 / 8.5       12.7 / 7.0    6.8 / 6.4          6.6 / 5.8
// So the limit suits calls whose gradients need no scaling.  What it gives up: calls that scale 17 chunks or more take 16 to
// 50% longer than with two launches, graphs of them up to 86%; which of them a list meets is not known at its launch.
constexpr unsigned kSmallChunks = 64;
static_assert(kSmallChunks <= kClipFew, "a chunk for each tensor at least");
cudaError_t launch_small_clip(const ClipParams<kClipFew>& p, int dtype, int out_dtype, cudaStream_t st);
// CAP kClipFew or kClipTensors
template <int CAP>
cudaError_t launch_squares(const ClipParams<CAP>& p, int dtype, int sms, cudaStream_t st);
template <int CAP>
cudaError_t launch_scale(const ClipParams<CAP>& p, int dtype, int out_dtype, int sms, cudaStream_t st);
cudaError_t launch_norm_of_parts(const double* parts, int count, float* norm, cudaStream_t st);

// out = a b^T (+ out): a [m][k], b [n][k] quantized by rows.
struct MatmulParams {
  CUtensorMap a, b;    // codes, unused without blocks
  CUtensorMap sa, sb;  // scales
  CUtensorMap o;       // the result, where bulk_out
  long long m, n, ldo;
  void* out;
  int kb;         // blocks of 128 along k, may be 0
  int bn, split, rows_a, stages;  // see MatmulPlan
  int out_dtype, add, a_fmt, b_fmt;
  long long stall_at;  // see take_stall
  int bulk_out;  // the result's start, rows and row stride are multiples of 16 bytes
  unsigned int* fault;
};

cudaError_t launch_matmul(const MatmulParams& p, const MatmulPlan& plan, cudaStream_t st);
cudaError_t prepare_matmul_kernels(int sms, Clusters* clusters);

// out = Q(x) w^T for few rows of x, whose codes and scales fit in shared memory: see train_linear.cu.
// One launch and no workspace: from Python a call takes 12 to 13 us, where quantize and product take 18 to 19,
// as long as the device is not the longer of the two.  On the device, of the two kernels' time (us):
//   rows           1            8            16           24           40
//   1000 x 768     2.9 of 6.5   3.0 of 6.7   3.5 of 6.7   5.4 of 6.7   6.4 of 6.6
//   4096 x 1024    3.2 of 6.6   3.4 of 6.8   4.2 of 6.9   6.3 of 7.0   8.5 of 6.8
//   8192 x 2048    6.0 of 8.8   7.0 of 9.0   9.4 of 9.1   13.2 of 9.0
//   4096 x 4096    6.3 of 11.2  8.4 of 11.3  12.4 of 11.3
//   512 x 8192     6.4 of 8.2   11.2 of 8.5
//   32128 x 768    9.2 of 10.1  9.8 of 10.3  12.1 of 10.4  17.9 of 10.4  22.0 of 10.5
// So the limit is right for calls and small w; with many rows and a large w (and in a captured graph from 8
// to 16 rows on) the two kernels would be faster, up to twice at 40 x 32128 x 768.
constexpr int kLinearRows = 40, kLinearSmem = 90 * 1024;
// Its sums (1024 bytes a row), codes and scales.
constexpr long long linear_bytes(long long m, long long blocks) { return m * (1024 + blocks * (kBlock + 4)); }
constexpr bool few_rows(long long m, long long k) {
  return m <= kLinearRows && linear_bytes(m, (k + kBlock - 1) / kBlock) <= kLinearSmem;
}
struct LinearParams {
  CUtensorMap w;   // codes as [block][row][128], boxes of 4 x 16 x 128; unused without blocks
  CUtensorMap ws;  // scales, boxes of 4 blocks x 16 rows
  const void* x;
  void* out;
  long long ldx, ldo, n, k;
  int m, kb, out_dtype;
  long long stall_at;  // see take_stall
  unsigned int* fault;
};
cudaError_t prepare_linear_kernels();
cudaError_t launch_linear(const LinearParams& p, int dtype, int w_fmt, int sms, cudaStream_t st);

}  // namespace demo
