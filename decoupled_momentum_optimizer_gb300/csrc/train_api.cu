// C ABI of the training operators: argument checks, tensor maps, launches.  What each call
// computes is described in include/demo.h.
#include <cmath>
#include <cstring>

#include "../../include/demo.h"
#include "train_launch.h"

namespace {

using namespace demo;

constexpr int64_t kMaxElems = int64_t(1) << 38;  // keeps every grid within its limits
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 512;  // tensor-map coordinates are int32

uint64_t splitmix64_host(uint64_t z) {
  z += 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

bool valid_dtype(int dtype) { return dtype >= DEMO_F32 && dtype <= DEMO_F16; }
bool valid_fmt(int fmt) { return fmt == DEMO_E4M3 || fmt == DEMO_E5M2; }
int64_t elem_size(int dtype) { return dtype == DEMO_F32 ? 4 : 2; }
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
bool at(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int to_status(cudaError_t e) { return e == cudaSuccess ? DEMO_OK : DEMO_ECUDA; }

// A matrix in memory: `rows` rows of `width` bytes, `stride` bytes apart.
struct Region {
  const void* p;
  int64_t rows, width, stride;
};

Region matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  return Region{p, rows, cols * size, rows == 1 ? cols * size : ld * size};
}
Region flat(const void* p, int64_t bytes) { return Region{p, 1, bytes, bytes}; }

// Whether two regions share a byte.  Column slices of one buffer (equal strides) are told apart;
// otherwise the rows' whole span counts.
bool overlap(const Region& a, const Region& b) {
  if (a.p == nullptr || b.p == nullptr || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t ax = x + static_cast<uintptr_t>((a.rows - 1) * a.stride + a.width);
  const uintptr_t by = y + static_cast<uintptr_t>((b.rows - 1) * b.stride + b.width);
  if (!(x < by && y < ax)) return false;
  if (a.rows > 1 && b.rows > 1 && a.stride == b.stride && a.width <= a.stride && b.width <= b.stride) {
    const uintptr_t s = static_cast<uintptr_t>(a.stride);
    const uintptr_t d = x < y ? (y - x) % s : (s - (x - y) % s) % s;  // b's columns start d bytes into a's rows
    return d < static_cast<uintptr_t>(a.width) || d + static_cast<uintptr_t>(b.width) > s;
  }
  return true;
}

bool same(const Region& a, const Region& b) { return a.p == b.p && (a.rows == 1 || a.stride == b.stride); }

// A matrix argument of `rows` x `cols` elements; `written` ones may not have rows that overlap.
int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype, bool written) {
  if (p == nullptr) return DEMO_EINVAL;
  if (ld < 0 || ld > kMaxElems || (written && rows > 1 && ld < cols)) return DEMO_EINVAL;
  if (rows > 1 && ld > 0 && rows > (kMaxElems << 2) / ld) return DEMO_EINVAL;
  return at(p, static_cast<uintptr_t>(elem_size(dtype))) ? DEMO_OK : DEMO_EALIGN;
}

int drop_params(double p, uint64_t seed, uint64_t step, uint64_t site, DropParams* out) {
  if (!(p >= 0.0 && p <= 1.0)) return DEMO_EINVAL;
  const double t = std::nearbyint(65536.0 * p);
  out->key = splitmix64_host(splitmix64_host(splitmix64_host(seed) ^ step) ^ site);
  out->threshold = static_cast<unsigned int>(t);
  out->scale = t < 65536.0 ? static_cast<float>(65536.0 / (65536.0 - t)) : 0.0f;
  return DEMO_OK;
}

bool code_map(EncodeTiledFn encode, CUtensorMap* map, const void* codes, int64_t rows, int64_t kp, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kp), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kp)};
  const cuuint32_t box[2] = {kBlock, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Codes as [block][row][128]: boxes of 4 blocks x 16 rows.
bool block_map(EncodeTiledFn encode, CUtensorMap* map, const void* codes, int64_t rows, int64_t blocks) {
  const cuuint64_t dims[3] = {kBlock, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(blocks)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(blocks) * kBlock, kBlock};
  const cuuint32_t box[3] = {kBlock, 16, 4};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales: [blocks][ld] float32, boxes of `box_rows` columns and `box_blocks` rows.
bool scale_map(EncodeTiledFn encode, CUtensorMap* map, const float* scales, int64_t rows, int64_t blocks, int box_rows,
               int box_blocks) {
  const cuuint64_t ld = static_cast<cuuint64_t>(up(rows, 4));
  const cuuint64_t dims[2] = {ld, static_cast<cuuint64_t>(blocks)};
  const cuuint64_t strides[1] = {ld * 4};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_blocks)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(scales), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The result [m][n], boxes of 32 rows of `bytes` bytes.
bool out_map(EncodeTiledFn encode, CUtensorMap* map, void* out, int64_t m, int64_t n, int64_t ldo, int dtype, int bytes) {
  const int64_t size = elem_size(dtype);
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(m)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(m == 1 ? n * size : ldo * size)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(bytes / size), 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType type = dtype == DEMO_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : dtype == DEMO_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encode(map, type, 2, out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_quantized(const void* codes, const float* scales, int fmt) {
  if (!valid_fmt(fmt) || codes == nullptr || scales == nullptr) return DEMO_EINVAL;
  return at(codes, 16) && at(scales, 16) ? DEMO_OK : DEMO_EALIGN;
}

int64_t code_bytes(int64_t rows, int64_t k) { return rows * up(k, kBlock); }
int64_t scale_bytes(int64_t rows, int64_t k) { return up(k, kBlock) / kBlock * up(rows, 4) * 4; }

}  // namespace

extern "C" {

int demo_dropout(const void* x, int64_t ldx, const void* residual, int64_t ldr, void* out, int64_t ldo, int dtype,
                 int64_t rows, int64_t cols, double p, uint64_t seed, uint64_t step, uint64_t site, void* stream) {
  if (!valid_dtype(dtype) || rows < 0 || cols < 0) return DEMO_EINVAL;
  DropoutParams q;
  std::memset(&q, 0, sizeof(q));
  int s = drop_params(p, seed, step, site, &q.drop);
  if (s != DEMO_OK) return s;
  if (rows == 0 || cols == 0) return DEMO_OK;
  if (cols > kMaxElems || rows > kMaxElems / ((cols + 3) / 4)) return DEMO_EINVAL;
  if ((s = check_matrix(x, rows, cols, ldx, dtype, false)) != DEMO_OK) return s;
  if (residual != nullptr && (s = check_matrix(residual, rows, cols, ldr, dtype, false)) != DEMO_OK) return s;
  if ((s = check_matrix(out, rows, cols, ldo, dtype, true)) != DEMO_OK) return s;
  const int64_t size = elem_size(dtype);
  const Region rx = matrix(x, rows, cols, ldx, size), rr = matrix(residual, rows, cols, ldr, size),
               ro = matrix(out, rows, cols, ldo, size);
  if (!same(rx, ro) && overlap(rx, ro)) return DEMO_EINVAL;
  if (residual != nullptr && !same(rr, ro) && overlap(rr, ro)) return DEMO_EINVAL;
  DeviceInfo dev;
  if ((s = device_info(&dev)) != DEMO_OK) return s;
  q.x = x;
  q.residual = residual;
  q.out = out;
  q.rows = rows;
  q.cols = cols;
  q.ldx = ldx;
  q.ldr = ldr;
  q.ldo = ldo;
  return to_status(launch_dropout(q, dtype, static_cast<cudaStream_t>(stream)));
}

size_t demo_fp8_bytes(int64_t rows, int64_t k, size_t* scale_bytes_out) {
  if (scale_bytes_out) *scale_bytes_out = 0;
  if (rows < 0 || k < 0 || rows > kMaxDim || k > kMaxDim) return 0;
  if (scale_bytes_out) *scale_bytes_out = static_cast<size_t>(scale_bytes(rows, k));
  return static_cast<size_t>(code_bytes(rows, k));
}

int demo_fp8_quantize(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols, int relu, const void* gate,
                      int64_t ldg, double p, uint64_t seed, uint64_t step, uint64_t site, int fmt, int tiles,
                      void* codes_rows, float* scales_rows, void* codes_cols, float* scales_cols, void* stream) {
  if (!valid_dtype(dtype) || !valid_fmt(fmt) || rows < 0 || cols < 0) return DEMO_EINVAL;
  if (relu < 0 || relu > 1 || tiles < 0 || tiles > 1) return DEMO_EINVAL;
  QuantParams q;
  std::memset(&q, 0, sizeof(q));
  int s = drop_params(p, seed, step, site, &q.drop);
  if (s != DEMO_OK) return s;
  if (rows == 0 || cols == 0) return DEMO_OK;
  if (rows > kMaxDim || cols > kMaxDim || up(rows, kBlock) > kMaxElems / up(cols, kBlock)) return DEMO_EINVAL;
  if (codes_rows == nullptr && codes_cols == nullptr) return DEMO_EINVAL;
  if ((codes_rows == nullptr) != (scales_rows == nullptr) || (codes_cols == nullptr) != (scales_cols == nullptr))
    return DEMO_EINVAL;
  if ((s = check_matrix(x, rows, cols, ldx, dtype, false)) != DEMO_OK) return s;
  if (gate != nullptr && (s = check_matrix(gate, rows, cols, ldg, dtype, false)) != DEMO_OK) return s;
  if (codes_rows != nullptr && (s = check_quantized(codes_rows, scales_rows, fmt)) != DEMO_OK) return s;
  if (codes_cols != nullptr && (s = check_quantized(codes_cols, scales_cols, fmt)) != DEMO_OK) return s;
  const int64_t size = elem_size(dtype);
  const Region in[2] = {matrix(x, rows, cols, ldx, size), matrix(gate, rows, cols, ldg, size)};
  const Region out[4] = {flat(codes_rows, code_bytes(rows, cols)), flat(scales_rows, scale_bytes(rows, cols)),
                         flat(codes_cols, code_bytes(cols, rows)), flat(scales_cols, scale_bytes(cols, rows))};
  for (int i = 0; i < 4; ++i) {
    if (overlap(out[i], in[0]) || overlap(out[i], in[1])) return DEMO_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return DEMO_EINVAL;
  }
  DeviceInfo dev;
  if ((s = device_info(&dev)) != DEMO_OK) return s;
  q.x = x;
  q.gate = gate;
  q.rows = rows;
  q.cols = cols;
  q.ldx = ldx;
  q.ldg = ldg;
  q.row_blocks = static_cast<unsigned int>(up(rows, kBlock) / kBlock);
  q.col_blocks = static_cast<unsigned int>(up(cols, kBlock) / kBlock);
  q.relu = relu;
  q.tiles = tiles;
  q.codes_rows = codes_rows;
  q.scales_rows = scales_rows;
  q.codes_cols = codes_cols;
  q.scales_cols = scales_cols;
  return to_status(launch_quantize(q, dtype, fmt, static_cast<cudaStream_t>(stream)));
}

int demo_fp8_matmul(const void* a_codes, const float* a_scales, int a_fmt, const void* b_codes, const float* b_scales,
                    int b_fmt, int64_t m, int64_t n, int64_t k, void* out, int64_t ldo, int out_dtype,
                    int add, void* stream) {
  if (!valid_dtype(out_dtype) || !valid_fmt(a_fmt) || !valid_fmt(b_fmt)) return DEMO_EINVAL;
  if (m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return DEMO_EINVAL;
  if (add < 0 || add > 1 || (add && out_dtype != DEMO_F32)) return DEMO_EINVAL;
  if (m == 0 || n == 0) return DEMO_OK;
  if (m > kMaxElems / n) return DEMO_EINVAL;
  int s;
  if ((s = check_matrix(out, m, n, ldo, out_dtype, true)) != DEMO_OK) return s;
  if (k > 0) {
    if ((s = check_quantized(a_codes, a_scales, a_fmt)) != DEMO_OK) return s;
    if ((s = check_quantized(b_codes, b_scales, b_fmt)) != DEMO_OK) return s;
    const Region ro = matrix(out, m, n, ldo, elem_size(out_dtype));
    if (overlap(ro, flat(a_codes, code_bytes(m, k))) || overlap(ro, flat(b_codes, code_bytes(n, k))) ||
        overlap(ro, flat(a_scales, scale_bytes(m, k))) || overlap(ro, flat(b_scales, scale_bytes(n, k))))
      return DEMO_EINVAL;
  }
  DeviceInfo dev;
  if ((s = device_info(&dev)) != DEMO_OK) return s;
  if (k == 0 && add) return DEMO_OK;  // adding zeros would turn -0 into 0
  MatmulParams q;
  std::memset(&q, 0, sizeof(q));
  q.kb = static_cast<int>(up(k, kBlock) / kBlock);
  const MatmulPlan plan = plan_matmul(*dev.clusters, m, n, q.kb);
  if (plan.grid == 0) return DEMO_ECUDA;
  const int64_t size = elem_size(out_dtype);
  // a bulk store writes whole units of 16 bytes, past the end of a row that is not a multiple of them
  q.bulk_out = at(out, 16) && n * size % 16 == 0 && (m == 1 || ldo * size % 16 == 0);
  if ((q.kb > 0 && (!code_map(dev.encode, &q.a, a_codes, m, up(k, kBlock), plan.rows_a) ||
                    !code_map(dev.encode, &q.b, b_codes, n, up(k, kBlock), plan.rows_b) ||
                    !scale_map(dev.encode, &q.sa, a_scales, m, q.kb, kBlock, plan.chain) ||
                    !scale_map(dev.encode, &q.sb, b_scales, n, q.kb, plan.bn, plan.chain))) ||
      (q.bulk_out && !out_map(dev.encode, &q.o, out, m, n, ldo, out_dtype, plan.bn)))
    return DEMO_ECUDA;
  q.m = m;
  q.n = n;
  q.ldo = ldo;
  q.out = out;
  q.bn = plan.bn;
  q.split = plan.split;
  q.rows_a = plan.rows_a;
  q.stages = plan.stages;
  q.out_dtype = out_dtype;
  q.add = add;
  q.a_fmt = a_fmt;
  q.b_fmt = b_fmt;
  q.fault = dev.fault;
  q.stall_at = take_stall();
  return to_status(launch_matmul(q, plan, static_cast<cudaStream_t>(stream)));
}

size_t demo_fp8_linear_workspace(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0 || k <= 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim || few_rows(m, k)) return 0;
  return static_cast<size_t>(code_bytes(m, k) + scale_bytes(m, k));
}

int demo_fp8_linear(const void* x, int64_t ldx, int dtype, const void* w_codes, const float* w_scales, int w_fmt,
                    int64_t m, int64_t n, int64_t k, void* out, int64_t ldo, int out_dtype,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype) || !valid_fmt(w_fmt)) return DEMO_EINVAL;
  if (m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return DEMO_EINVAL;
  if (m == 0 || n == 0) return DEMO_OK;
  if (m > kMaxElems / n || (k > 0 && m > kMaxElems / up(k, kBlock))) return DEMO_EINVAL;
  int s;
  if ((s = check_matrix(out, m, n, ldo, out_dtype, true)) != DEMO_OK) return s;
  const size_t need = demo_fp8_linear_workspace(m, n, k);
  if (k > 0) {
    if ((s = check_matrix(x, m, k, ldx, dtype, false)) != DEMO_OK) return s;
    if ((s = check_quantized(w_codes, w_scales, w_fmt)) != DEMO_OK) return s;
    const Region ro = matrix(out, m, n, ldo, elem_size(out_dtype)), rx = matrix(x, m, k, ldx, elem_size(dtype)),
                 rc = flat(w_codes, code_bytes(n, k)), rs = flat(w_scales, scale_bytes(n, k));
    if (overlap(ro, rx) || overlap(ro, rc) || overlap(ro, rs)) return DEMO_EINVAL;
    if (need > 0) {
      if (workspace_bytes < need) return DEMO_ENOSPACE;
      if (workspace == nullptr) return DEMO_EINVAL;
      if (!at(workspace, 16)) return DEMO_EALIGN;
      const Region rw = flat(workspace, static_cast<int64_t>(need));
      if (overlap(rw, ro) || overlap(rw, rx) || overlap(rw, rc) || overlap(rw, rs)) return DEMO_EINVAL;
    }
  }
  if (few_rows(m, k)) {
    DeviceInfo dev;
    if ((s = device_info(&dev)) != DEMO_OK) return s;
    LinearParams q;
    std::memset(&q, 0, sizeof(q));
    q.kb = static_cast<int>(up(k, kBlock) / kBlock);
    if (q.kb > 0 && (!block_map(dev.encode, &q.w, w_codes, n, q.kb) || !scale_map(dev.encode, &q.ws, w_scales, n, q.kb, 16, 4)))
      return DEMO_ECUDA;
    q.fault = dev.fault;
    q.stall_at = take_stall();
    q.x = x;
    q.out = out;
    q.ldx = ldx;
    q.ldo = ldo;
    q.n = n;
    q.k = k;
    q.m = static_cast<int>(m);
    q.out_dtype = out_dtype;
    return to_status(launch_linear(q, dtype, w_fmt, dev.sms, static_cast<cudaStream_t>(stream)));
  }
  void* codes = workspace;
  float* scales = reinterpret_cast<float*>(static_cast<char*>(workspace) + code_bytes(m, k));
  if (k > 0 && (s = demo_fp8_quantize(x, ldx, dtype, m, k, 0, nullptr, 0, 0.0, 0, 0, 0, DEMO_E4M3, 0, codes, scales,
                                      nullptr, nullptr, stream)) != DEMO_OK)
    return s;
  return demo_fp8_matmul(codes, scales, DEMO_E4M3, w_codes, w_scales, w_fmt, m, n, k, out, ldo, out_dtype, 0,
                         stream);
}

}  // extern "C"
