// Parameter blocks and launchers of the training operators' kernels (dropout, block-scaled 8-bit
// quantization, products of quantized matrices), and what their C entry points need of the
// library's per-device state.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

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
};

cudaError_t launch_quantize(const QuantParams& p, int dtype, int fmt, cudaStream_t st);

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
