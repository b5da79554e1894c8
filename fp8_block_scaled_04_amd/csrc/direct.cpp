// The calls of expert routing, the weighted combine and the 4-bit products,
// from Python without ctypes: a decoding step makes them by the hundred, and
// their checks and marshalling in Python cost 3 us a call, as much as the
// launch.  Each function here takes the tensors of the binding's function of
// the same name.  It checks types, shapes, strides and devices, launches on the
// current stream and returns the status, or None where anything is not as
// expected: the binding's own checks then say what is wrong (or take what is
// only unusual, such as a subclass of Tensor).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>

#include "fp8gemm.h"

namespace {

PyObject* g_current_device;  // callables: () -> device index, device index -> stream address
PyObject* g_raw_stream;

// What does not fit is left to the binding.
struct Unusual {};

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_CheckExact(o)) throw Unusual();
  return THPVariable_Unpack(o);
}

int as_int(int64_t v) {
  if (v < INT_MIN || v > INT_MAX) throw Unusual();
  return int(v);
}
int as_int(PyObject* o) {
  if (!PyLong_Check(o)) throw Unusual();
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Unusual();
  }
  return as_int(int64_t(v));
}
float as_float(PyObject* o) {
  if (PyFloat_Check(o)) return float(PyFloat_AS_DOUBLE(o));
  return float(as_int(o));
}

int float_type(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return FP8G_F32;
  if (t.scalar_type() == at::kBFloat16) return FP8G_BF16;
  throw Unusual();
}

// The address of a dense tensor of the given type, shape and device.
void* dense(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, int device) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || !t.is_cuda() || t.get_device() != device)
    throw Unusual();
  return t.data_ptr();
}
void* dense(PyObject* o, at::ScalarType type, at::IntArrayRef shape, int device) {
  return dense(tensor(o), type, shape, device);
}
void* dense_or_null(PyObject* o, at::ScalarType type, at::IntArrayRef shape, int device) {
  return o == Py_None ? nullptr : dense(o, type, shape, device);
}

// A matrix whose rows are dense; their stride may exceed their length.
struct Matrix {
  int64_t rows, cols, ld;
  int device;
  void* at;
  explicit Matrix(const at::Tensor& t) {
    if (!t.is_cuda() || t.dim() != 2) throw Unusual();
    rows = t.size(0), cols = t.size(1), ld = rows < 2 || !cols ? cols : t.stride(0), device = t.get_device();
    if (ld < cols || (cols > 1 && t.stride(1) != 1)) throw Unusual();
    at = t.data_ptr();
  }
};

void* stream_of(int device) {
  PyObject* now = PyObject_CallNoArgs(g_current_device);
  const bool same = now && PyLong_AsLong(now) == device;
  PyObject* at = same ? PyObject_CallOneArg(g_raw_stream, now) : nullptr;
  void* s = at ? PyLong_AsVoidPtr(at) : nullptr;
  Py_XDECREF(now);
  Py_XDECREF(at);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    throw Unusual();
  }
  if (!same) throw Unusual();
  return s;
}

// status = call() without the interpreter's lock.
template <typename Call>
int released(Call&& call) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  return status;
}

// body() -> status, None for whatever it throws.
template <typename Body>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, Body&& body) {
  if (given != wanted || !g_current_device) Py_RETURN_NONE;
  try {
    return PyLong_FromLong(body());
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // logits, topk, score_func, bias, expert_groups, topk_groups, group_score, renormalize, scale, expert_idx, weights
  return guarded(n, 11, [&] {
    const at::Tensor& t = tensor(a[0]);
    const Matrix l(t);
    const int type = float_type(t), topk = as_int(a[1]), T = as_int(l.rows), E = as_int(l.cols);
    const int score = as_int(a[2]), groups = as_int(a[4]), topk_groups = as_int(a[5]), group_score = as_int(a[6]);
    const int renormalize = PyObject_IsTrue(a[7]);
    if (topk < 0 || renormalize < 0) throw Unusual();
    const float scale = as_float(a[8]);
    const auto* bias = static_cast<const float*>(dense_or_null(a[3], at::kFloat, {E}, l.device));
    auto* idx = static_cast<int32_t*>(dense(a[9], at::kInt, {T, topk}, l.device));
    auto* w = static_cast<float*>(dense(a[10], at::kFloat, {T, topk}, l.device));
    void* s = stream_of(l.device);
    return released([&] {
      return fp8_moe_route(l.at, type, l.ld, bias, T, E, score, groups, topk_groups, group_score, topk, renormalize,
                           scale, idx, w, s);
    });
  });
}

PyObject* moe_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // logits, expert_idx, grad_weights, grad_logits, score_func, renormalize, scale
  return guarded(n, 7, [&] {
    const at::Tensor &t = tensor(a[0]), &g = tensor(a[3]), &i = tensor(a[1]);
    const Matrix l(t), gl(g);
    if (g.scalar_type() != t.scalar_type() || gl.rows != l.rows || gl.cols != l.cols || gl.device != l.device ||
        i.dim() != 2)
      throw Unusual();
    const int type = float_type(t), T = as_int(l.rows), E = as_int(l.cols), topk = as_int(i.size(1));
    const auto* idx = static_cast<const int32_t*>(dense(i, at::kInt, {T, topk}, l.device));
    const auto* gw = static_cast<const float*>(dense(a[2], at::kFloat, {T, topk}, l.device));
    const int score = as_int(a[4]), renormalize = PyObject_IsTrue(a[5]);
    if (renormalize < 0) throw Unusual();
    const float scale = as_float(a[6]);
    void* s = stream_of(l.device);
    return released([&] {
      return fp8_moe_route_backward(l.at, type, l.ld, idx, gw, T, E, score, topk, renormalize, scale, gl.at, gl.ld, s);
    });
  });
}

// The operands that the combine and its gradient share; y is the tensor of the experts' rows.
struct Combine {
  int T, n, rows, topk, device;
  uint16_t *y, *tokens;
  const int32_t* dst;
  const float* weights;
  Combine(const at::Tensor& rows_, PyObject* dst_, PyObject* weights_, const at::Tensor& tokens_) {
    if (!tokens_.is_cuda() || tokens_.dim() != 2 || rows_.dim() < 1) throw Unusual();
    device = tokens_.get_device();
    T = as_int(tokens_.size(0)), n = as_int(tokens_.size(1));
    if (n == 0 || rows_.sizes().back() != n) throw Unusual();
    tokens = static_cast<uint16_t*>(dense(tokens_, at::kBFloat16, {T, n}, device));
    y = static_cast<uint16_t*>(dense(rows_, at::kBFloat16, rows_.sizes(), device));
    rows = as_int(rows_.numel() / n);
    const at::Tensor& pairs = tensor(dst_ != Py_None ? dst_ : weights_);
    if (pairs.dim() != 2) throw Unusual();
    topk = as_int(pairs.size(1));
    dst = static_cast<const int32_t*>(dense_or_null(dst_, at::kInt, {T, topk}, device));
    weights = static_cast<const float*>(dense_or_null(weights_, at::kFloat, {T, topk}, device));
    if (!dst && rows != int64_t(T) * topk) throw Unusual();
  }
};

PyObject* moe_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // y, dst_row, weights, out
  return guarded(n, 4, [&] {
    const Combine c(tensor(a[0]), a[1], a[2], tensor(a[3]));
    void* s = stream_of(c.device);
    return released([&] { return fp8_moe_combine(c.y, c.rows, c.n, c.dst, c.weights, c.T, c.topk, c.tokens, s); });
  });
}

PyObject* moe_combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // grad_out, y, dst_row, weights, grad_y, grad_weights
  return guarded(n, 6, [&] {
    const at::Tensor& gy = tensor(a[4]);
    const Combine c(gy, a[2], a[3], tensor(a[0]));
    auto* gw = static_cast<float*>(dense_or_null(a[5], at::kFloat, {c.T, c.topk}, c.device));
    const auto* y = gw || a[5] != Py_None
                        ? static_cast<const uint16_t*>(dense(a[1], at::kBFloat16, gy.sizes(), c.device))
                        : nullptr;
    void* s = stream_of(c.device);
    return released([&] {
      return fp8_moe_combine_backward(c.tokens, y, c.rows, c.n, c.dst, c.weights, c.T, c.topk, c.y, gw, s);
    });
  });
}

// The operands of a 4-bit product, of one matrix (experts < 0) or of `experts`.
struct W4 {
  int n, group, scales_type, out_type;
  const uint8_t *w, *zeros;
  const void* scales;
  void* out;
  W4(const at::Tensor& x, const Matrix& m, int64_t rows, const at::Tensor& w_, const at::Tensor& scales_,
     PyObject* zeros_, const at::Tensor& out_, int64_t experts) {
    const int lead = experts < 0 ? 0 : 1;
    if (x.scalar_type() != at::kBFloat16 || scales_.dim() != 2 + lead || m.cols == 0 || m.cols % 2) throw Unusual();
    n = as_int(scales_.size(lead));
    const int64_t groups = scales_.size(lead + 1);
    if (groups == 0 || m.cols % groups) throw Unusual();
    group = as_int(m.cols / groups);
    scales_type = float_type(scales_), out_type = float_type(out_);
    const int64_t code_shape[] = {experts, n, m.cols / 2}, group_shape[] = {experts, n, groups};
    const at::IntArrayRef codes(code_shape + 1 - lead, 2 + lead), per_group(group_shape + 1 - lead, 2 + lead);
    w = static_cast<const uint8_t*>(dense(w_, at::kByte, codes, m.device));
    scales = dense(scales_, scales_.scalar_type(), per_group, m.device);
    zeros = static_cast<const uint8_t*>(dense_or_null(zeros_, at::kByte, per_group, m.device));
    out = dense(out_, out_.scalar_type(), {rows, n}, m.device);
  }
};

PyObject* w4_matvec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // x, w, scales, out, w_format, zeros
  return guarded(n, 6, [&] {
    const at::Tensor& x = tensor(a[0]);
    const Matrix m(x);
    const W4 p(x, m, m.rows, tensor(a[1]), tensor(a[2]), a[5], tensor(a[3]), -1);
    const int rows = as_int(m.rows), k = as_int(m.cols), format = as_int(a[4]);
    void* s = stream_of(m.device);
    return released([&] {
      return fp8_w4_matvec(static_cast<const uint16_t*>(m.at), m.ld, p.w, format, p.scales, p.scales_type, p.zeros,
                           p.group, p.out, p.out_type, rows, p.n, k, s);
    });
  });
}

PyObject* w4_matvec_experts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // x, expert_idx, w, scales, out, w_format, zeros
  return guarded(n, 7, [&] {
    const at::Tensor &x = tensor(a[0]), &i = tensor(a[1]), &w = tensor(a[2]);
    const Matrix m(x);
    const int64_t pairs = i.numel();
    if (w.dim() != 3 || (pairs && (m.rows == 0 || pairs % m.rows))) throw Unusual();
    const W4 p(x, m, pairs, w, tensor(a[3]), a[6], tensor(a[4]), w.size(0));
    const auto* idx = static_cast<const int32_t*>(dense(i, at::kInt, i.sizes(), m.device));
    const int rows = as_int(m.rows), k = as_int(m.cols), P = as_int(pairs), E = as_int(w.size(0));
    const int format = as_int(a[5]);
    void* s = stream_of(m.device);
    return released([&] {
      return fp8_w4_matvec_experts(static_cast<const uint16_t*>(m.at), m.ld, rows, idx, P, p.w, format, p.scales,
                                   p.scales_type, p.zeros, p.group, p.out, p.out_type, E, p.n, k, s);
    });
  });
}

PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "setup(current_device, raw_stream)");
    return nullptr;
  }
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(g_current_device, a[0]);
  Py_XSETREF(g_raw_stream, a[1]);
  Py_RETURN_NONE;
}

#define FP8G_DIRECT(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FP8G_DIRECT(setup),
                           FP8G_DIRECT(moe_route),
                           FP8G_DIRECT(moe_route_backward),
                           FP8G_DIRECT(moe_combine),
                           FP8G_DIRECT(moe_combine_backward),
                           FP8G_DIRECT(w4_matvec),
                           FP8G_DIRECT(w4_matvec_experts),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_direct", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__direct() { return PyModule_Create(&g_module); }
