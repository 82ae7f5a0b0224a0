// C ABI of the training operators: argument checks, tensor maps, launches.  What each call
// computes is described in include/demo.h.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>

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

int check_norm(int dtype, int weight_dtype, int64_t rows, int64_t cols) {
  if (!valid_dtype(dtype) || (weight_dtype != DEMO_F32 && weight_dtype != dtype)) return DEMO_EINVAL;
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kNormCols) return DEMO_EINVAL;
  return cols > 0 && up(rows, kBlock) > kMaxElems / up(cols, kBlock) ? DEMO_EINVAL : DEMO_OK;
}

// Tokens as rows of `per`: their region, and whether the arguments are in range.
int check_tokens(const void* tokens, int token_bytes, int64_t rows, int64_t per, int64_t ld) {
  if ((token_bytes != 4 && token_bytes != 8) || rows < 0 || per < 0 || rows > kMaxDim || per > kMaxDim) return DEMO_EINVAL;
  if (rows == 0 || per == 0) return DEMO_OK;
  if (tokens == nullptr || rows > kMaxDim / per || ld < 0 || ld > kMaxElems) return DEMO_EINVAL;
  if (rows > 1 && ld > 0 && rows > kMaxElems / ld) return DEMO_EINVAL;
  return at(tokens, static_cast<uintptr_t>(token_bytes)) ? DEMO_OK : DEMO_EALIGN;
}
Tokens tokens_of(const void* tokens, int token_bytes, int64_t rows, int64_t per, int64_t ld) {
  return Tokens{tokens, per, rows == 1 ? per : ld, token_bytes == 8};
}

// The gradient's workspace: sorted tokens, their positions, parts of tokens that cross pieces.
struct EmbedWorkspace {
  int64_t batch, keys, positions, parts;
  int piece;
  EmbedWorkspace(int64_t n, int64_t cols) {
    batch = n < kMaxSorted ? n : kMaxSorted;
    piece = embed_piece(batch, cols);
    keys = n > kFewTokens ? up(4 * batch, 16) : 0;
    positions = n > kFewTokens ? up(2 * batch, 16) : 0;
    const int64_t pieces = (batch + piece - 1) / piece;
    parts = n > kFewTokens ? pieces * 2 * up(cols, 256) * 4 : 0;
  }
};

// Whether a list of tensors may be read, and written, as one call does: a place that is written is apart from
// every other place.
struct Span {
  uintptr_t begin, end;
};
// `reads` spans that are read only, then `writes` that are written.  Lists usually come in ascending order, so
// nothing but two walks is left.
bool apart(Span* spans, int64_t reads, int64_t writes) {
  const auto before = [](const Span& a, const Span& b) { return a.begin < b.begin; };
  Span* const r = spans;
  Span* const w = spans + reads;
  if (!std::is_sorted(r, r + reads, before)) std::sort(r, r + reads, before);
  if (!std::is_sorted(w, w + writes, before)) std::sort(w, w + writes, before);
  uintptr_t read = 0, written = 0;  // the ends of those so far
  for (int64_t i = 0, j = 0; i < reads || j < writes;) {
    if (j == writes || (i < reads && r[i].begin < w[j].begin)) {
      if (r[i].begin < written) return false;
      read = std::max(read, r[i++].end);
    } else {
      if (w[j].begin < written || w[j].begin < read) return false;
      written = std::max(written, w[j++].end);
    }
  }
  return true;
}

int64_t clip_launches(int64_t count) { return count > 0 ? (count + kClipTensors - 1) / kClipTensors : 1; }

// The arguments that the norm and the clipping share.  `out` NULL: nothing but the norm is written.
int check_grads(int count, const void* const* g, const int64_t* n, int dtype, void* const* out, int out_dtype, const float* norm,
                bool needs_work, const void* workspace, size_t workspace_bytes) {
  if (count < 0 || !valid_dtype(dtype) || norm == nullptr || (count > 0 && (g == nullptr || n == nullptr))) return DEMO_EINVAL;
  const size_t need = needs_work ? demo_grad_workspace(count) : 0;
  if (workspace_bytes < need) return DEMO_ENOSPACE;
  if (need > 0 && workspace == nullptr) return DEMO_EINVAL;
  if (!at(norm, 4) || (need > 0 && !at(workspace, 16))) return DEMO_EALIGN;
  const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[2 * static_cast<size_t>(count) + 2]);
  if (spans == nullptr) return DEMO_ENOSPACE;
  int64_t reads = 0, writes = 0;  // reads from the front; writes from the middle on, moved behind the reads below
  Span* const written = spans.get() + count;
  const auto span = [](const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + static_cast<uintptr_t>(bytes)};
  };
  const int64_t size = elem_size(dtype), osize = elem_size(out_dtype);
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    if (n[i] < 0 || n[i] > kMaxElems) return DEMO_EINVAL;
    if (n[i] == 0) continue;
    total += n[i];
    if (g[i] == nullptr || total > kMaxElems) return DEMO_EINVAL;
    if (!at(g[i], static_cast<uintptr_t>(size))) return DEMO_EALIGN;
    if (out != nullptr) {
      if (out[i] == nullptr) return DEMO_EINVAL;
      if (!at(out[i], static_cast<uintptr_t>(osize))) return DEMO_EALIGN;
      written[writes++] = span(out[i], n[i] * osize);
    }
    if (out == nullptr || out[i] != g[i] || size != osize) spans[reads++] = span(g[i], n[i] * size);
  }
  written[writes++] = span(norm, 4);
  if (need > 0) written[writes++] = span(workspace, static_cast<int64_t>(need));
  std::copy(written, written + writes, spans.get() + reads);
  return apart(spans.get(), reads, writes) ? DEMO_OK : DEMO_EINVAL;
}

// The tensors of one launch, from `from` on; returns the next one's index.
template <int CAP>
int fill_clip(ClipParams<CAP>* q, int from, int count, const void* const* g, const int64_t* n, void* const* out, int64_t size) {
  q->count = 0;
  q->chunks = 0;
  for (; from < count && q->count < CAP; ++from) {
    if (n[from] == 0) continue;
    q->g[q->count] = g[from];
    q->out[q->count] = out != nullptr ? out[from] : nullptr;
    q->n[q->count] = n[from];
    q->start[q->count++] = q->chunks;
    q->chunks += static_cast<unsigned int>(clip_chunks(reinterpret_cast<uintptr_t>(g[from]), n[from], static_cast<int>(size)));
  }
  return from;
}

// Whether all tensors fit one launch of a few chunks; fills it if so.
bool fill_small(ClipParams<kClipFew>* q, int count, const void* const* g, const int64_t* n, void* const* out, int64_t size,
                float* norm) {
  int64_t left = (int64_t(kSmallChunks) << 15) / size;  // chunks are 32 KB
  if (count > kClipFew) return false;
  for (int i = 0; i < count; ++i)
    if ((left -= n[i]) < 0) return false;
  fill_clip(q, 0, count, g, n, out, size);
  q->given = 0;
  q->norm = norm;
  return q->count > 0 && q->chunks <= kSmallChunks;
}

template <int CAP>
bool all_in_place(const ClipParams<CAP>& q) {
  for (int i = 0; i < q.count; ++i)
    if (q.out[i] != q.g[i]) return false;
  return true;
}

// Launches the sums of squares of all tensors; *parts_used sums are left in `parts`.
template <int CAP>
int launch_all_squares(ClipParams<CAP>* q, int count, const void* const* g, const int64_t* n, int dtype, int sms, double* parts,
                       int* parts_used, cudaStream_t st) {
  *parts_used = 0;
  for (int from = 0; from < count;) {
    from = fill_clip(q, from, count, g, n, nullptr, elem_size(dtype));
    if (q->count == 0) break;
    q->parts = parts + *parts_used;
    *parts_used += clip_parts(q->chunks, dtype, sms);
    const int s = to_status(launch_squares(*q, dtype, sms, st));
    if (s != DEMO_OK) return s;
  }
  return DEMO_OK;
}

template <int CAP>
int norm_of_list(ClipParams<CAP>* q, int count, const void* const* g, const int64_t* n, int dtype, int sms, double* parts,
                 float* norm, cudaStream_t st) {
  int used = 0;
  const int s = launch_all_squares(q, count, g, n, dtype, sms, parts, &used, st);
  return s != DEMO_OK ? s : to_status(launch_norm_of_parts(parts, used, norm, st));
}

template <int CAP>
int clip_list(ClipParams<CAP>* q, int count, const void* const* g, const int64_t* n, int dtype, void* const* to, int out_dtype,
              double max_norm, int sms, double* parts, float* norm, int norm_given, cudaStream_t st) {
  int used = 0, s;
  if (!norm_given && (s = launch_all_squares(q, count, g, n, dtype, sms, parts, &used, st)) != DEMO_OK) return s;
  bool any = false;
  for (int from = 0; from < count;) {
    from = fill_clip(q, from, count, g, n, to, elem_size(dtype));
    if (q->count == 0) break;
    q->part_count = used;
    q->all_parts = parts;
    q->given = norm_given;
    q->first_launch = !any;
    q->in_place = all_in_place(*q);
    q->max_norm = max_norm;
    q->norm = norm;
    if ((s = to_status(launch_scale(*q, dtype, out_dtype, sms, st))) != DEMO_OK) return s;
    any = true;
  }
  // Nothing to scale: the norm over nothing.
  return any || norm_given ? DEMO_OK : to_status(launch_norm_of_parts(parts, 0, norm, st));
}

// One row has no stride (whatever is given must not decide how it is read).
int64_t row_stride(int64_t rows, int64_t ld) { return rows == 1 ? 0 : ld; }

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

int demo_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int dtype, const void* weight,
                  int weight_dtype, int64_t rows, int64_t cols, double eps, void* total, int64_t ldt, void* out,
                  int64_t ldo, float* rstd, int fmt, void* codes_rows, float* scales_rows, void* codes_cols,
                  float* scales_cols, void* stream) {
  int s = check_norm(dtype, weight_dtype, rows, cols);
  if (s != DEMO_OK) return s;
  if (!valid_fmt(fmt) || !(eps > 0.0) || !std::isfinite(eps)) return DEMO_EINVAL;
  if ((codes_rows == nullptr) != (scales_rows == nullptr) || (codes_cols == nullptr) != (scales_cols == nullptr))
    return DEMO_EINVAL;
  if (residual == nullptr && total != nullptr) return DEMO_EINVAL;
  if (codes_cols != nullptr && (rstd == nullptr || (residual != nullptr && total == nullptr))) return DEMO_EINVAL;
  if (rows == 0 || cols == 0) return DEMO_OK;
  if (total == nullptr && out == nullptr && rstd == nullptr && codes_rows == nullptr && codes_cols == nullptr)
    return DEMO_EINVAL;
  if ((s = check_matrix(x, rows, cols, ldx, dtype, false)) != DEMO_OK) return s;
  if ((s = check_matrix(weight, 1, cols, cols, weight_dtype, false)) != DEMO_OK) return s;
  if (residual != nullptr && (s = check_matrix(residual, rows, cols, ldr, dtype, false)) != DEMO_OK) return s;
  if (total != nullptr && (s = check_matrix(total, rows, cols, ldt, dtype, true)) != DEMO_OK) return s;
  if (out != nullptr && (s = check_matrix(out, rows, cols, ldo, dtype, true)) != DEMO_OK) return s;
  if (rstd != nullptr && !at(rstd, 4)) return DEMO_EALIGN;
  if (codes_rows != nullptr && (s = check_quantized(codes_rows, scales_rows, fmt)) != DEMO_OK) return s;
  if (codes_cols != nullptr && (s = check_quantized(codes_cols, scales_cols, fmt)) != DEMO_OK) return s;
  const int64_t size = elem_size(dtype);
  const Region rx = matrix(x, rows, cols, ldx, size), rr = matrix(residual, rows, cols, ldr, size),
               rw = flat(weight, cols * elem_size(weight_dtype)), rt = matrix(total, rows, cols, ldt, size),
               ro = matrix(out, rows, cols, ldo, size);
  // The sum, and the result of the fused kernel, may take an input's place; the column form reads x again.
  for (const Region& in : {rx, rr}) {
    if (!same(in, rt) && overlap(in, rt)) return DEMO_EINVAL;
    if ((codes_cols != nullptr || !same(in, ro)) && overlap(in, ro)) return DEMO_EINVAL;
  }
  const Region made[7] = {rt, ro, flat(rstd, 4 * rows), flat(codes_rows, code_bytes(rows, cols)),
                          flat(scales_rows, scale_bytes(rows, cols)), flat(codes_cols, code_bytes(cols, rows)),
                          flat(scales_cols, scale_bytes(cols, rows))};
  for (int i = 0; i < 7; ++i) {
    if (overlap(made[i], rw) || (i >= 2 && (overlap(made[i], rx) || overlap(made[i], rr)))) return DEMO_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(made[i], made[j])) return DEMO_EINVAL;
  }
  DeviceInfo dev;
  if ((s = device_info(&dev)) != DEMO_OK) return s;
  NormParams q;
  std::memset(&q, 0, sizeof(q));
  q.x = x;
  q.residual = residual;
  q.weight = weight;
  q.total = total;
  q.out = out;
  q.rstd = rstd;
  q.codes = codes_cols == nullptr ? codes_rows : nullptr;
  q.scales = scales_rows;
  q.rows = rows;
  q.cols = cols;
  q.ldx = row_stride(rows, ldx);
  q.ldr = row_stride(rows, ldr);
  q.ldt = row_stride(rows, ldt);
  q.ldo = row_stride(rows, ldo);
  q.col_blocks = static_cast<unsigned int>(up(cols, kBlock) / kBlock);
  q.fmt = fmt;
  q.inv = 1.0 / static_cast<double>(cols);
  q.eps = eps;
  q.inv_hi = static_cast<float>(q.inv);
  q.inv_lo = static_cast<float>(q.inv - static_cast<double>(q.inv_hi));
  q.eps_hi = static_cast<float>(eps);
  q.eps_lo = static_cast<float>(eps - static_cast<double>(q.eps_hi));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((s = to_status(launch_norm(q, dtype, weight_dtype, dev.sms, st))) != DEMO_OK || codes_cols == nullptr) return s;
  QuantParams c;
  std::memset(&c, 0, sizeof(c));
  c.x = residual != nullptr ? total : x;
  c.ldx = residual != nullptr ? q.ldt : q.ldx;
  c.rows = rows;
  c.cols = cols;
  c.row_blocks = static_cast<unsigned int>(up(rows, kBlock) / kBlock);
  c.col_blocks = q.col_blocks;
  c.codes_rows = codes_rows;
  c.scales_rows = scales_rows;
  c.codes_cols = codes_cols;
  c.scales_cols = scales_cols;
  c.rstd = rstd;
  c.weight = weight;
  c.weight_dtype = weight_dtype;
  return to_status(launch_quantize(c, dtype, fmt, st));
}

size_t demo_rms_norm_grad_workspace(int64_t rows, int64_t cols) {
  if (rows <= 1 || cols <= 0 || cols > kNormCols) return 0;
  return static_cast<size_t>((rows < kNormParts ? rows : kNormParts) * cols * 4);
}

int demo_rms_norm_grad(const void* dy, int64_t lddy, const void* total, int64_t ldt, int dtype, const void* weight,
                       int weight_dtype, const float* rstd, int64_t rows, int64_t cols, const void* past, int64_t ldp,
                       void* dx, int64_t lddx, float* dweight, int add, void* workspace, size_t workspace_bytes,
                       void* stream) {
  int s = check_norm(dtype, weight_dtype, rows, cols);
  if (s != DEMO_OK) return s;
  if (add < 0 || add > 1) return DEMO_EINVAL;
  if (cols == 0) return DEMO_OK;
  if (dweight != nullptr && !at(dweight, 4)) return DEMO_EALIGN;
  if (rows > 0) {
    if ((s = check_matrix(dy, rows, cols, lddy, dtype, false)) != DEMO_OK) return s;
    if ((s = check_matrix(total, rows, cols, ldt, dtype, false)) != DEMO_OK) return s;
    if ((s = check_matrix(weight, 1, cols, cols, weight_dtype, false)) != DEMO_OK) return s;
    if (past != nullptr && (s = check_matrix(past, rows, cols, ldp, dtype, false)) != DEMO_OK) return s;
    if ((s = check_matrix(dx, rows, cols, lddx, dtype, true)) != DEMO_OK) return s;
    if (rstd == nullptr) return DEMO_EINVAL;
    if (!at(rstd, 4)) return DEMO_EALIGN;
    const size_t need = dweight != nullptr ? demo_rms_norm_grad_workspace(rows, cols) : 0;
    if (workspace_bytes < need) return DEMO_ENOSPACE;
    if (need > 0 && workspace == nullptr) return DEMO_EINVAL;
    if (need > 0 && !at(workspace, 16)) return DEMO_EALIGN;
    const int64_t size = elem_size(dtype);
    const Region rdx = matrix(dx, rows, cols, lddx, size), rdw = flat(dweight, 4 * cols),
                 rwork = flat(need > 0 ? workspace : nullptr, static_cast<int64_t>(need));
    for (const Region& in : {matrix(dy, rows, cols, lddy, size), matrix(total, rows, cols, ldt, size),
                             matrix(past, rows, cols, ldp, size)}) {
      if (!same(in, rdx) && overlap(in, rdx)) return DEMO_EINVAL;
      if (overlap(in, rdw) || overlap(in, rwork)) return DEMO_EINVAL;
    }
    for (const Region& in : {flat(weight, cols * elem_size(weight_dtype)), flat(rstd, 4 * rows)})
      if (overlap(in, rdx) || overlap(in, rdw) || overlap(in, rwork)) return DEMO_EINVAL;
    if (overlap(rdx, rdw) || overlap(rdx, rwork) || overlap(rdw, rwork)) return DEMO_EINVAL;
  } else if (dweight == nullptr || add) {
    return DEMO_OK;  // a sum over nothing, added
  }
  DeviceInfo dev;
  if ((s = device_info(&dev)) != DEMO_OK) return s;
  NormGradParams q;
  std::memset(&q, 0, sizeof(q));
  q.dy = dy;
  q.total = total;
  q.weight = weight;
  q.rstd = rstd;
  q.past = past;
  q.dx = dx;
  q.dw = dweight;
  q.partials = static_cast<float*>(workspace);
  q.rows = rows;
  q.cols = cols;
  q.lddy = row_stride(rows, lddy);
  q.ldt = row_stride(rows, ldt);
  q.ldp = row_stride(rows, ldp);
  q.lddx = row_stride(rows, lddx);
  q.add = add;
  q.inv = static_cast<float>(1.0 / static_cast<double>(cols));
  return to_status(launch_norm_grad(q, dtype, weight_dtype, dev.sms, static_cast<cudaStream_t>(stream)));
}

int demo_embedding(const void* tokens, int token_bytes, int64_t token_rows, int64_t token_cols, int64_t ldtokens,
                   const void* table, int64_t ldt, int table_dtype, int64_t vocab, int64_t cols, float scale, void* out,
                   int64_t ldo, int out_dtype, void* stream) {
  if (!valid_dtype(table_dtype) || !valid_dtype(out_dtype) || !std::isfinite(scale)) return DEMO_EINVAL;
  if (vocab < 0 || cols < 0 || vocab > kMaxDim || cols > kMaxDim) return DEMO_EINVAL;
  int s = check_tokens(tokens, token_bytes, token_rows, token_cols, ldtokens);
  if (s != DEMO_OK) return s;
  const int64_t n = token_rows * token_cols;
  if (n == 0 || cols == 0) return DEMO_OK;
  if (n > kMaxElems / cols) return DEMO_EINVAL;
  if (vocab > 0 && (s = check_matrix(table, vocab, cols, ldt, table_dtype, false)) != DEMO_OK) return s;
  if ((s = check_matrix(out, n, cols, ldo, out_dtype, true)) != DEMO_OK) return s;
  const Region ro = matrix(out, n, cols, ldo, elem_size(out_dtype));
  if (overlap(ro, matrix(tokens, token_rows, token_cols, ldtokens, token_bytes)) ||
      overlap(ro, matrix(table, vocab, cols, ldt, elem_size(table_dtype))))
    return DEMO_EINVAL;
  DeviceInfo dev;
  if ((s = device_info(&dev)) != DEMO_OK) return s;
  LookupParams q;
  std::memset(&q, 0, sizeof(q));
  q.tokens = tokens_of(tokens, token_bytes, token_rows, token_cols, ldtokens);
  q.table = table;
  q.out = out;
  q.n = n;
  q.vocab = vocab;
  q.cols = cols;
  q.ldt = row_stride(vocab, ldt);
  q.ldo = row_stride(n, ldo);
  q.scale = scale;
  return to_status(launch_lookup(q, table_dtype, out_dtype, static_cast<cudaStream_t>(stream)));
}

size_t demo_embedding_grad_workspace(int64_t n, int64_t cols) {
  if (n <= 0 || cols <= 0 || n > kMaxDim || cols > kMaxDim) return 0;
  const EmbedWorkspace w(n, cols);
  return static_cast<size_t>(w.keys + w.positions + w.parts);
}

int demo_embedding_grad(const void* tokens, int token_bytes, int64_t token_rows, int64_t token_cols, int64_t ldtokens,
                        const void* dy, int64_t lddy, int dtype, int64_t vocab, int64_t cols, float scale, float* grad,
                        int64_t ldg, int add, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype) || !std::isfinite(scale) || add < 0 || add > 1) return DEMO_EINVAL;
  if (vocab < 0 || cols < 0 || vocab > kMaxDim || cols > kMaxDim) return DEMO_EINVAL;
  int s = check_tokens(tokens, token_bytes, token_rows, token_cols, ldtokens);
  if (s != DEMO_OK) return s;
  const int64_t n = token_rows * token_cols;
  if (vocab == 0 || cols == 0 || (n == 0 && add)) return DEMO_OK;
  if (n > kMaxElems / cols || vocab > kMaxElems / cols) return DEMO_EINVAL;
  if ((s = check_matrix(grad, vocab, cols, ldg, DEMO_F32, true)) != DEMO_OK) return s;
  const EmbedWorkspace w(n, cols);
  if (n > 0) {
    if ((s = check_matrix(dy, n, cols, lddy, dtype, false)) != DEMO_OK) return s;
    const int64_t need = w.keys + w.positions + w.parts;
    if (workspace_bytes < static_cast<size_t>(need)) return DEMO_ENOSPACE;
    if (need > 0 && workspace == nullptr) return DEMO_EINVAL;
    if (need > 0 && !at(workspace, 16)) return DEMO_EALIGN;
    const Region rg = matrix(grad, vocab, cols, ldg, 4), rw = flat(need > 0 ? workspace : nullptr, need);
    for (const Region& in : {matrix(tokens, token_rows, token_cols, ldtokens, token_bytes),
                             matrix(dy, n, cols, lddy, elem_size(dtype))})
      if (overlap(rg, in) || overlap(rw, in)) return DEMO_EINVAL;
    if (overlap(rg, rw)) return DEMO_EINVAL;
  }
  DeviceInfo dev;
  if ((s = device_info(&dev)) != DEMO_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* work = static_cast<char*>(workspace);
  SortParams t;
  std::memset(&t, 0, sizeof(t));
  EmbedGradParams q;
  std::memset(&q, 0, sizeof(q));
  t.tokens = tokens_of(tokens, token_bytes, token_rows, token_cols, ldtokens);
  t.vocab = vocab;
  q.dy = dy;
  q.grad = grad;
  q.vocab = vocab;
  q.cols = cols;
  q.lddy = row_stride(n, lddy);
  q.ldg = row_stride(vocab, ldg);
  q.piece = w.piece;
  q.add = add;
  q.scale = scale;
  if (n > 0 && n <= kFewTokens) {
    q.n = static_cast<int>(n);
    return to_status(launch_embed_grad(q, t.tokens, dtype, st));
  }
  if (n > 0) {
    q.keys = t.keys = reinterpret_cast<int*>(work);
    q.positions = t.positions = reinterpret_cast<unsigned short*>(work + w.keys);
    q.parts = reinterpret_cast<float*>(work + w.keys + w.positions);
  }
  // As many tokens at a time as one cluster sorts; the later ones are added.
  int64_t first = 0;
  t.grad = grad;
  t.cols = cols;
  t.ldg = q.ldg;
  // Written anew: what no token names is 0.  Without tokens the first kernel fills everything.
  if (!add) t.filled = n == 0 ? vocab : filled_rows(w.batch, vocab, cols);
  q.zero_from = add ? vocab : t.filled;
  do {
    const int64_t left = n - first;
    t.n = q.n = static_cast<int>(left < w.batch ? left : w.batch);
    t.first = q.first = first;
    if ((s = to_status(launch_sort_tokens(t, dev.sms, st))) != DEMO_OK) return s;
    if (t.n == 0) break;  // no tokens: the table is filled, nothing is summed
    if ((s = to_status(launch_embed_grad(q, t.tokens, dtype, st))) != DEMO_OK) return s;
    t.filled = 0;
    q.zero_from = vocab;
    q.add = 1;
    first += t.n;
  } while (first < n);
  return DEMO_OK;
}

size_t demo_grad_workspace(int count) {
  return count < 0 ? 0 : static_cast<size_t>(clip_launches(count)) * kClipParts * sizeof(double);
}

int demo_grad_norm(int count, const void* const* g, const int64_t* n, int dtype, float* norm, void* workspace,
                   size_t workspace_bytes, void* stream) {
  int s = check_grads(count, g, n, dtype, nullptr, dtype, norm, true, workspace, workspace_bytes);
  if (s != DEMO_OK) return s;
  DeviceInfo dev;
  if ((s = device_info(&dev)) != DEMO_OK) return s;
  double* parts = static_cast<double*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (count > kClipFew) {
    ClipParams<kClipTensors> q;
    return norm_of_list(&q, count, g, n, dtype, dev.sms, parts, norm, st);
  }
  ClipParams<kClipFew> q;
  if (fill_small(&q, count, g, n, nullptr, elem_size(dtype), norm)) {
    q.only_norm = 1;
    return to_status(launch_small_clip(q, dtype, dtype, st));
  }
  return norm_of_list(&q, count, g, n, dtype, dev.sms, parts, norm, st);
}

int demo_clip_grads(int count, const void* const* g, const int64_t* n, int dtype, void* const* out, int out_dtype,
                    double max_norm, float* norm, int norm_given, void* workspace, size_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.0) || norm_given < 0 || norm_given > 1) return DEMO_EINVAL;
  if (!valid_dtype(out_dtype) || (out_dtype != dtype && out_dtype != DEMO_F32)) return DEMO_EINVAL;
  if (out == nullptr && (out_dtype != dtype || count < 0 || (count > 0 && g == nullptr))) return DEMO_EINVAL;
  // Without `out` the gradients themselves are written.
  void* const* to = out != nullptr ? out : const_cast<void* const*>(g);
  int s = check_grads(count, g, n, dtype, to, out_dtype, norm, !norm_given, workspace, workspace_bytes);
  if (s != DEMO_OK) return s;
  DeviceInfo dev;
  if ((s = device_info(&dev)) != DEMO_OK) return s;
  double* parts = static_cast<double*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (count > kClipFew) {
    ClipParams<kClipTensors> q;
    return clip_list(&q, count, g, n, dtype, to, out_dtype, max_norm, dev.sms, parts, norm, norm_given, st);
  }
  ClipParams<kClipFew> q;
  if (!norm_given && fill_small(&q, count, g, n, to, elem_size(dtype), norm)) {
    q.only_norm = 0;
    q.in_place = all_in_place(q);
    q.max_norm = max_norm;
    return to_status(launch_small_clip(q, dtype, out_dtype, st));
  }
  return clip_list(&q, count, g, n, dtype, to, out_dtype, max_norm, dev.sms, parts, norm, norm_given, st);
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
