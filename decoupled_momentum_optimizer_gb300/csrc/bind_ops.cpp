// Calls of the norm, embedding and clipping operators from Python without the interpreter's share: one C function
// takes the tensors, checks them, allocates the results and enqueues the call (from Python a small call took
// 12 to 35 us, most of it between the tensors and the C entry point; clipping 193 tensors took 300).
//
// These functions take the plain calls only.  Whatever they do not take (a wrong type, shape, device or
// stride, a tensor that autograd follows, another current device, an uninitialised library, no memory) they
// leave to the Python bindings by returning NotImplemented, so every refusal and every error is raised in one
// place.  A status that the library returns comes back as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/forward_grad.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <vector>

#include "../../include/demo.h"

namespace {

// Thrown (and caught at each function's end) where the call is not a plain one.
struct Other {};

int code_of(at::ScalarType t) {
  if (t == at::kFloat) return DEMO_F32;
  if (t == at::kBFloat16) return DEMO_BF16;
  if (t == at::kHalf) return DEMO_F16;
  throw Other();
}

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Other();
  return THPVariable_Unpack(o);
}

// One call: its device (the first tensor's), which must be the current one.
struct Call {
  bool recorded = c10::GradMode::is_enabled();
  int tangents = -1;  // whether forward-mode tangents are followed: a level is open, and this is no autograd.Function
  int device = -1;
  std::vector<c10::TensorImpl*> written;  // given tensors that the call writes

  // Few tensors have any autograd data, and only then is it worth to ask for the level (a lock).
  bool has_tangent(const at::Tensor& t) {
    if (t.unsafeGetTensorImpl()->autograd_meta() == nullptr) return false;
    if (tangents < 0)
      tangents = c10::AutogradState::get_tls_state().get_fw_grad_mode() &&
                 torch::autograd::ForwardADLevel::try_get_by_idx(0) != nullptr;
    return tangents != 0 && t._fw_grad(0).defined();
  }
  const at::Tensor& take(PyObject* o) {
    const at::Tensor& t = tensor(o);
    if (!t.is_cuda() || (recorded && t.requires_grad()) || has_tangent(t)) throw Other();
    const int d = static_cast<int>(t.get_device());
    if (device < 0) {
      if (c10::cuda::current_device() != d) throw Other();
      device = d;
    } else if (device != d) {
      throw Other();
    }
    return t;
  }
  const at::Tensor& take_written(PyObject* o) {
    const at::Tensor& t = take(o);
    written.push_back(t.unsafeGetTensorImpl());
    return t;
  }
  // What autograd saved of them before is out of date (tensors of inference mode have no count).
  void count_written() const {
    for (c10::TensorImpl* t : written)
      if (!t->is_inference()) t->bump_version();
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
  at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(sizes, type, c10::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)),
                                             std::nullopt));
  }
};

struct Matrix {
  void* p = nullptr;
  int64_t ld = 0, rows = 0, cols = 0;
};

// A tensor seen as rows of its last dimension.
Matrix matrix(const at::Tensor& t) {
  const int64_t dims = t.dim();
  if (dims < 1) throw Other();
  Matrix m;
  m.p = t.data_ptr();
  m.cols = t.size(dims - 1);
  if (m.cols == 0) throw Other();
  m.rows = t.numel() / m.cols;
  if (m.cols > 1 && m.rows > 0 && t.stride(dims - 1) != 1) throw Other();
  m.ld = m.cols;
  if (dims == 2) {
    m.ld = t.stride(0);
  } else if (m.rows > 1 && !t.is_contiguous()) {
    throw Other();
  }
  return m;
}

Matrix like(const at::Tensor& t, const at::Tensor& x) {
  if (t.scalar_type() != x.scalar_type() || t.sizes() != x.sizes()) throw Other();
  return matrix(t);
}

// A contiguous float32 tensor of n elements.
float* floats(const at::Tensor& t, int64_t n) {
  if (t.scalar_type() != at::kFloat || t.numel() != n || !t.is_contiguous()) throw Other();
  return static_cast<float*>(t.data_ptr());
}

const void* weight_of(Call& call, PyObject* o, const at::Tensor& x, int64_t cols, int* code) {
  const at::Tensor& w = call.take(o);
  if ((w.scalar_type() != at::kFloat && w.scalar_type() != x.scalar_type()) || w.dim() != 1 || w.size(0) != cols ||
      !w.is_contiguous())
    throw Other();
  *code = code_of(w.scalar_type());
  return w.data_ptr();
}

struct TokenRows {
  const void* p;
  int bytes;
  int64_t rows, cols, ld;
};

TokenRows token_rows(const at::Tensor& t) {
  const int bytes = t.scalar_type() == at::kLong ? 8 : t.scalar_type() == at::kInt ? 4 : 0;
  if (bytes == 0 || !t.is_contiguous()) throw Other();
  return TokenRows{t.data_ptr(), bytes, 1, t.numel(), t.numel()};
}

bool given(PyObject* o) { return o != Py_None; }
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}
PyObject* whole_number(int64_t v) {
  PyObject* o = PyLong_FromLongLong(v);
  if (o == nullptr) throw Other();
  return o;
}
PyObject* wrap_or_none(const at::Tensor& t) {
  if (!t.defined()) return none();
  PyObject* o = THPVariable_Wrap(t);
  if (o == nullptr) throw Other();
  return o;
}
// An object that was passed in, or the tensor that was made in its place.
PyObject* passed(PyObject* o, const at::Tensor& made) {
  if (!given(o)) return wrap_or_none(made);
  Py_INCREF(o);
  return o;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Other();
  }
  return v;
}
bool truth(PyObject* o) {
  if (o == Py_True) return true;
  if (o == Py_False) return false;
  throw Other();
}

// The results, complete before the library is called: nothing can fail after it.
struct Results {
  PyObject* p;
  explicit Results(PyObject* o) : p(o) {
    if (p == nullptr) throw Other();
  }
  explicit Results(Py_ssize_t n) : Results(PyTuple_New(n)) {}
  Results(const Results&) = delete;
  ~Results() { Py_XDECREF(p); }
  void set(Py_ssize_t i, PyObject* o) { PyTuple_SET_ITEM(p, i, o); }
  // The results where the library took the call; its status otherwise, or NotImplemented where it was not ready.
  PyObject* after(const Call& call, int status) {
    if (status != DEMO_OK) {
      if (status == DEMO_ENOTINIT) throw Other();
      return PyLong_FromLong(status);
    }
    call.count_written();
    PyObject* o = p;
    p = nullptr;
    return o;
  }
};

// The body's result; NotImplemented for a call that is not plain.
template <typename F>
PyObject* plain(Py_ssize_t n, Py_ssize_t want, F body) {
  try {
    if (n == want) return body();
  } catch (...) {
    PyErr_Clear();
  }
  Py_RETURN_NOTIMPLEMENTED;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// (x, weight, eps, residual, values, form, fmt, save, out, total, rstd) with form 0 none, 1 rows, 2 columns, 3 both ->
// (out, total, rstd, and with a form: row codes, row scales, column codes, column scales, rows, columns)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 11, [&]() -> PyObject* {
    Call call;
    const at::Tensor& x = call.take(a[0]);
    const int dtype = code_of(x.scalar_type());
    const Matrix mx = matrix(x);
    int weight_dtype;
    const void* weight = weight_of(call, a[1], x, mx.cols, &weight_dtype);
    const double eps = number(a[2]);
    Matrix mr, mt, mo;
    at::Tensor total, out, rstd, codes[2], scales[2];
    if (given(a[3])) {
      mr = like(call.take(a[3]), x);
      if (given(a[9])) {
        mt = like(call.take_written(a[9]), x);
      } else {
        total = call.empty(x.sizes(), x.scalar_type());
        mt = Matrix{total.data_ptr(), mx.cols};
      }
    } else if (given(a[9])) {
      throw Other();
    }
    if (given(a[8])) {
      mo = like(call.take_written(a[8]), x);
    } else if (truth(a[4])) {
      out = call.empty(x.sizes(), x.scalar_type());
      mo = Matrix{out.data_ptr(), mx.cols};
    }
    const long form = PyLong_AsLong(a[5]), fmt = PyLong_AsLong(a[6]);
    if (form < 0 || form > 3 || fmt < 0 || fmt > 1 || (form != 0 && x.dim() != 2)) throw Other();
    const int64_t sizes[2] = {mx.rows, mx.cols};
    for (int f = 0; f < 2; ++f) {
      if (!(form >> f & 1)) continue;
      const int64_t rows = sizes[f], k = sizes[1 - f], blocks = up(k, 128) / 128;
      codes[f] = call.empty({rows, blocks * 128}, fmt == DEMO_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2);
      scales[f] = call.empty({blocks, up(rows, 4)}, at::kFloat);
    }
    float* factors = nullptr;
    const bool save = truth(a[7]);
    if (given(a[10])) {
      factors = floats(call.take_written(a[10]), mx.rows);
    } else if (save || (form & 2)) {
      rstd = call.empty({mx.rows}, at::kFloat);
      factors = static_cast<float*>(rstd.data_ptr());
    }
    const auto at_ptr = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    Results r(form == 0 ? 3 : 9);
    r.set(0, passed(a[8], out));
    r.set(1, given(a[3]) ? passed(a[9], total) : passed(a[0], total));
    r.set(2, given(a[10]) || save ? passed(a[10], rstd) : none());
    for (int f = 0; form != 0 && f < 2; ++f) {
      r.set(3 + 2 * f, wrap_or_none(codes[f]));
      r.set(4 + 2 * f, wrap_or_none(scales[f]));
      r.set(7 + f, whole_number(sizes[f]));
    }
    return r.after(call, demo_rms_norm(mx.p, mx.ld, mr.p, mr.ld, dtype, weight, weight_dtype, mx.rows, mx.cols, eps, mt.p,
                                       mt.ld, mo.p, mo.ld, factors, static_cast<int>(fmt), at_ptr(codes[0]),
                                       static_cast<float*>(at_ptr(scales[0])), at_ptr(codes[1]),
                                       static_cast<float*>(at_ptr(scales[1])), call.stream()));
  });
}

// (dy, total, weight, rstd, past, out, dweight, add, weight_grad) -> (dx, dweight)
PyObject* rms_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 9, [&]() -> PyObject* {
    Call call;
    const at::Tensor& dy = call.take(a[0]);
    const int dtype = code_of(dy.scalar_type());
    const Matrix md = matrix(dy), mt = like(call.take(a[1]), dy);
    int weight_dtype;
    const void* weight = weight_of(call, a[2], dy, md.cols, &weight_dtype);
    const float* rstd = floats(call.take(a[3]), md.rows);
    Matrix mp, mo;
    if (given(a[4])) mp = like(call.take(a[4]), dy);
    at::Tensor out, dweight, work;
    if (given(a[5])) {
      mo = like(call.take_written(a[5]), dy);
    } else {
      out = call.empty(dy.sizes(), dy.scalar_type());
      mo = Matrix{out.data_ptr(), md.cols};
    }
    const bool add = truth(a[7]);
    float* dw = nullptr;
    size_t need = 0;
    if (truth(a[8])) {
      if (given(a[6])) {
        dw = floats(call.take_written(a[6]), md.cols);
      } else {
        if (add) throw Other();
        dweight = call.empty({md.cols}, at::kFloat);
        dw = static_cast<float*>(dweight.data_ptr());
      }
      need = demo_rms_norm_grad_workspace(md.rows, md.cols);
      if (need > 0) work = call.empty({static_cast<int64_t>(need)}, at::kByte);
    } else if (given(a[6])) {
      throw Other();
    }
    Results r(2);
    r.set(0, passed(a[5], out));
    r.set(1, passed(a[6], dweight));
    return r.after(call, demo_rms_norm_grad(md.p, md.ld, mt.p, mt.ld, dtype, weight, weight_dtype, rstd, md.rows, md.cols,
                                            mp.p, mp.ld, mo.p, mo.ld, dw, add, need > 0 ? work.data_ptr() : nullptr, need,
                                            call.stream()));
  });
}

// [*tokens.shape, cols]
std::vector<int64_t> rows_shape(const at::Tensor& tokens, int64_t cols) {
  std::vector<int64_t> s(tokens.sizes().begin(), tokens.sizes().end());
  s.push_back(cols);
  return s;
}

// (tokens, table, scale, dtype, out) -> out
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 5, [&]() -> PyObject* {
    Call call;
    const at::Tensor& tokens = call.take(a[0]);
    const TokenRows t = token_rows(tokens);
    const at::Tensor& table = call.take(a[1]);
    if (table.dim() != 2) throw Other();
    const Matrix mt = matrix(table);
    const float scale = static_cast<float>(number(a[2]));
    at::Tensor out;
    Matrix mo;
    at::ScalarType type = table.scalar_type();
    if (given(a[4])) {
      const at::Tensor& o = call.take_written(a[4]);
      if (given(a[3]) || o.sizes() != at::IntArrayRef(rows_shape(tokens, mt.cols))) throw Other();
      type = o.scalar_type();
      mo = matrix(o);
    } else {
      if (given(a[3])) {
        if (!THPDtype_Check(a[3])) throw Other();
        type = reinterpret_cast<THPDtype*>(a[3])->scalar_type;
      }
      code_of(type);
      out = call.empty(rows_shape(tokens, mt.cols), type);
      mo = Matrix{out.data_ptr(), mt.cols};
    }
    const int table_code = code_of(table.scalar_type()), code = code_of(type);
    Results r(passed(a[4], out));
    return r.after(call, demo_embedding(t.p, t.bytes, t.rows, t.cols, t.ld, mt.p, mt.ld, table_code, mt.rows, mt.cols, scale,
                                        mo.p, mo.ld, code, call.stream()));
  });
}

// (tokens, dy, vocab, scale, out, add) -> out
PyObject* embedding_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 6, [&]() -> PyObject* {
    Call call;
    const at::Tensor& tokens = call.take(a[0]);
    const TokenRows t = token_rows(tokens);
    const at::Tensor& dy = call.take(a[1]);
    const Matrix md = matrix(dy);
    if (dy.sizes().slice(0, dy.dim() - 1) != tokens.sizes()) throw Other();
    const float scale = static_cast<float>(number(a[3]));
    const bool add = truth(a[5]);
    int64_t vocab = -1;
    if (given(a[2])) {
      vocab = PyLong_AsLongLong(a[2]);
      if (vocab < 0) {
        PyErr_Clear();
        throw Other();
      }
    }
    at::Tensor out;
    Matrix mo;
    if (given(a[4])) {
      const at::Tensor& o = call.take_written(a[4]);
      if (o.dim() != 2 || o.scalar_type() != at::kFloat || o.size(1) != md.cols || (vocab >= 0 && o.size(0) != vocab)) throw Other();
      mo = matrix(o);
    } else {
      if (add || vocab < 0) throw Other();
      out = call.empty({vocab, md.cols}, at::kFloat);
      mo = Matrix{out.data_ptr(), md.cols, vocab, md.cols};
    }
    const size_t need = demo_embedding_grad_workspace(t.cols, md.cols);
    at::Tensor work;
    if (need > 0) work = call.empty({static_cast<int64_t>(need)}, at::kByte);
    const int code = code_of(dy.scalar_type());
    Results r(passed(a[4], out));
    return r.after(call, demo_embedding_grad(t.p, t.bytes, t.rows, t.cols, t.ld, md.p, md.ld, code, mo.rows, mo.cols, scale,
                                             static_cast<float*>(mo.p), mo.ld, add,
                                             need > 0 ? work.data_ptr() : nullptr, need, call.stream()));
  });
}

// The tensors of a list (or the one that is given): one dtype, contiguous.
struct List {
  std::vector<void*> p;
  std::vector<int64_t> n;
  int dtype = 0;

  List(Call& call, PyObject* o, bool written) {
    if (THPVariable_Check(o)) {
      add(call, o, written);
      return;
    }
    if (!PyList_Check(o) && !PyTuple_Check(o)) throw Other();
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(o);
    if (count == 0) throw Other();
    p.reserve(static_cast<size_t>(count));
    n.reserve(static_cast<size_t>(count));
    if (written) call.written.reserve(static_cast<size_t>(count));
    for (Py_ssize_t i = 0; i < count; ++i) add(call, PySequence_Fast_GET_ITEM(o, i), written);
  }
  void add(Call& call, PyObject* o, bool written) {
    const at::Tensor& t = written ? call.take_written(o) : call.take(o);
    const int code = code_of(t.scalar_type());
    if (p.empty())
      dtype = code;
    else if (code != dtype)
      throw Other();
    if (!t.is_contiguous()) throw Other();
    p.push_back(t.data_ptr());
    n.push_back(t.numel());
  }
  int count() const { return static_cast<int>(p.size()); }
};

// (gradients, out) -> norm
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 2, [&]() -> PyObject* {
    Call call;
    const List g(call, a[0], false);
    at::Tensor norm;
    float* np = given(a[1]) ? floats(call.take_written(a[1]), 1) : nullptr;
    if (np == nullptr) {
      norm = call.empty({}, at::kFloat);
      np = static_cast<float*>(norm.data_ptr());
    }
    const size_t need = demo_grad_workspace(g.count());
    const at::Tensor work = call.empty({static_cast<int64_t>(need)}, at::kByte);
    Results r(passed(a[1], norm));
    return r.after(call, demo_grad_norm(g.count(), g.p.data(), g.n.data(), g.dtype, np, work.data_ptr(), need, call.stream()));
  });
}

// (gradients, max_norm, norm, out) -> norm
PyObject* clip_grads(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 4, [&]() -> PyObject* {
    Call call;
    const List g(call, a[0], !given(a[3]));
    const double max_norm = number(a[1]);
    at::Tensor norm, work;
    float* np = given(a[2]) ? floats(call.take(a[2]), 1) : nullptr;
    size_t need = 0;
    if (np == nullptr) {
      norm = call.empty({}, at::kFloat);
      np = static_cast<float*>(norm.data_ptr());
      need = demo_grad_workspace(g.count());
      work = call.empty({static_cast<int64_t>(need)}, at::kByte);
    }
    void* const* to = nullptr;
    int out_dtype = g.dtype;
    std::optional<List> o;
    if (given(a[3])) {
      o.emplace(call, a[3], true);
      if (o->n != g.n) throw Other();
      to = o->p.data();
      out_dtype = o->dtype;
    }
    Results r(passed(a[2], norm));
    return r.after(call, demo_clip_grads(g.count(), g.p.data(), g.n.data(), g.dtype, to, out_dtype, max_norm, np,
                                         given(a[2]), need > 0 ? work.data_ptr() : nullptr, need, call.stream()));
  });
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(rms_norm),  CALL(rms_norm_grad), CALL(embedding), CALL(embedding_grad),
                         CALL(grad_norm), CALL(clip_grads),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `torch` is the version that this file was compiled against: tensors are read through inlined accessors, so the module
// is for that one alone.
PyMODINIT_FUNC PyInit__bind_ops() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch", DEMO_TORCH) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
