// The calls of expert routing, the weighted combine, the 4-bit products and the
// feed-forward block, from Python without ctypes: a decoding step makes them by the hundred, and
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

// FP8 codes of a format: bytes, or torch's type of it.
uint8_t* codes(const at::Tensor& t, int format, at::IntArrayRef shape, int device) {
  const at::ScalarType type = format == FP8G_E4M3   ? at::kFloat8_e4m3fn
                              : format == FP8G_E5M2 ? at::kFloat8_e5m2
                                                    : throw Unusual();
  return static_cast<uint8_t*>(dense(t, t.scalar_type() == type ? type : at::kByte, shape, device));
}

// Scales [..][ld] with ld >= rows.
float* scales_mn(const at::Tensor& t, int64_t groups, int64_t rows, int device, int64_t* ld) {
  if (t.dim() != 2 || t.size(0) != groups || t.size(1) < rows) throw Unusual();
  *ld = t.size(1);
  return static_cast<float*>(dense(t, at::kFloat, t.sizes(), device));
}

struct Workspace {
  void* at = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, int device) {
    if (o == Py_None) return;
    const at::Tensor& t = tensor(o);
    at = dense(t, t.scalar_type(), t.sizes(), device);
    bytes = t.nbytes();
  }
};

int64_t groups_of(int64_t k) { return (k + 127) / 128; }

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Unusual();
  return v;
}

PyObject* gemm_nt_epilogue(PyObject*, PyObject* const* a, Py_ssize_t n_) {
  // lhs, lhs_scales, rhs, rhs_scales, out, bias, activation, residual, preact, lhs_format, rhs_format, workspace
  return guarded(n_, 12, [&] {
    const at::Tensor &l = tensor(a[0]), &r = tensor(a[2]);
    if (l.dim() != 2 || r.dim() != 2 || !l.is_cuda()) throw Unusual();
    const int device = l.get_device(), m = as_int(l.size(0)), k = as_int(l.size(1)), n = as_int(r.size(0));
    const int activation = as_int(a[6]), lf = as_int(a[9]), rf = as_int(a[10]);
    int64_t ld;
    const uint8_t* lhs = codes(l, lf, {m, k}, device);
    const float* ls = scales_mn(tensor(a[1]), groups_of(k), m, device, &ld);
    const uint8_t* rhs = codes(r, rf, {n, k}, device);
    const auto* rs = static_cast<const float*>(dense(a[3], at::kFloat, {groups_of(n), groups_of(k)}, device));
    auto* out = static_cast<uint16_t*>(dense(a[4], at::kBFloat16, {m, n}, device));
    const int bias_type = a[5] == Py_None ? FP8G_F32 : float_type(tensor(a[5]));
    const void* bias = dense_or_null(a[5], bias_type == FP8G_F32 ? at::kFloat : at::kBFloat16, {n}, device);
    const auto* residual = static_cast<const uint16_t*>(dense_or_null(a[7], at::kBFloat16, {m, n}, device));
    auto* preact = static_cast<uint16_t*>(dense_or_null(a[8], at::kBFloat16, {m, n}, device));
    const Workspace w(a[11], device);
    void* s = stream_of(device);
    return released([&] {
      return fp8_gemm_nt_epilogue(lhs, lf, ls, ld, rhs, rf, rs, bias, bias_type, activation, residual, preact, out, m,
                                  n, k, w.at, w.bytes, s);
    });
  });
}

PyObject* epilogue_backward(PyObject*, PyObject* const* a, Py_ssize_t n_) {
  // grad_out, preact, activation, grad_preact, grad_bias, workspace
  return guarded(n_, 6, [&] {
    const at::Tensor& z = tensor(a[1]);
    if (z.dim() != 2 || !z.is_cuda()) throw Unusual();
    const int device = z.get_device(), m = as_int(z.size(0)), n = as_int(z.size(1)), activation = as_int(a[2]);
    const auto* zp = static_cast<const uint16_t*>(dense(z, at::kBFloat16, {m, n}, device));
    const auto* go = static_cast<const uint16_t*>(dense(a[0], at::kBFloat16, {m, n}, device));
    auto* gz = static_cast<uint16_t*>(dense(a[3], at::kBFloat16, {m, n}, device));
    auto* gb = static_cast<float*>(dense_or_null(a[4], at::kFloat, {n}, device));
    const Workspace w(a[5], device);
    if (!w.at && gb && fp8_epilogue_backward_workspace_bytes(m, n)) throw Unusual();  // to be allocated
    void* s = stream_of(device);
    return released([&] { return fp8_epilogue_backward(go, zp, activation, m, n, gz, gb, w.at, w.bytes, s); });
  });
}

// The parameters of the norms: all of one type, a gate of one row or of one for each.
struct NormParams {
  const void *post, *gate, *pre;
  int type = FP8G_F32, gate_rows = 1;
  NormParams(PyObject* post_, PyObject* gate_, PyObject* pre_, int post_norm, int T, int n, int device) {
    if (post_ != Py_None && !post_norm) throw Unusual();
    PyObject* any = post_ != Py_None ? post_ : gate_ != Py_None ? gate_ : pre_;
    if (any != Py_None) type = float_type(tensor(any));
    const at::ScalarType t = type == FP8G_F32 ? at::kFloat : at::kBFloat16;
    post = dense_or_null(post_, t, {n}, device);
    pre = dense_or_null(pre_, t, {n}, device);
    gate = nullptr;
    if (gate_ == Py_None) return;
    const at::Tensor& g = tensor(gate_);
    if (g.dim() == 2) {
      gate_rows = as_int(g.size(0));
      if (gate_rows != 1 && gate_rows != T) throw Unusual();
      gate = dense(g, t, {gate_rows, n}, device);
    } else {
      gate = dense(g, t, {n}, device);
    }
  }
};

at::ScalarType scalar(int type) { return type == FP8G_F32 ? at::kFloat : at::kBFloat16; }

PyObject* norm_residual(PyObject*, PyObject* const* a, Py_ssize_t n_) {
  // x, residual, h, y, q, q_scales, pre_weight, post_norm, post_weight, gate, residual_scale, kind, eps, q_format
  return guarded(n_, 14, [&] {
    const at::Tensor& xt = tensor(a[0]);
    const Matrix x(xt);
    const int device = x.device, T = as_int(x.rows), n = as_int(x.cols), type = float_type(xt);
    PyObject* any = a[1] != Py_None ? a[1] : a[2];
    const int stream_type = any == Py_None ? FP8G_F32 : float_type(tensor(any));
    const void* residual = nullptr;
    int64_t r_ld = n, q_ld = T;
    if (a[1] != Py_None) {
      const Matrix r(tensor(a[1]));
      if (r.rows != T || r.cols != n || r.device != device) throw Unusual();
      residual = r.at, r_ld = r.ld;
    }
    void* h = dense_or_null(a[2], scalar(stream_type), {T, n}, device);
    void* y = dense_or_null(a[3], scalar(type), {T, n}, device);
    const int format = as_int(a[13]), post_norm = truth(a[7]), kind = as_int(a[11]);
    uint8_t* q = a[4] == Py_None ? nullptr : codes(tensor(a[4]), format, {T, n}, device);
    float* qs = q || a[4] != Py_None ? scales_mn(tensor(a[5]), groups_of(n), T, device, &q_ld) : nullptr;
    const NormParams p(a[8], a[9], a[6], post_norm, T, n, device);
    const float scale = as_float(a[10]), eps = as_float(a[12]);
    void* s = stream_of(device);
    return released([&] {
      return fp8_norm_residual(x.at, type, x.ld, residual, r_ld, stream_type, T, n, kind, eps, post_norm, p.post,
                               p.gate, p.gate_rows, scale, p.pre, p.type, h, y, q, format, qs, q_ld, s);
    });
  });
}

PyObject* norm_residual_backward(PyObject*, PyObject* const* a, Py_ssize_t n_) {
  // grad_h, grad_y, x, h, grad_x, grad_residual, grad_pre_weight, grad_post_weight, grad_gate, pre_weight, post_norm,
  // post_weight, gate, residual_scale, kind, eps, workspace
  return guarded(n_, 17, [&] {
    if (a[0] == Py_None || a[1] == Py_None || a[2] == Py_None || a[3] == Py_None || a[16] == Py_None) throw Unusual();
    const at::Tensor &gh = tensor(a[0]), &xt = tensor(a[2]);
    const Matrix x(xt);
    const int device = x.device, T = as_int(x.rows), n = as_int(x.cols);
    const int type = float_type(xt), stream_type = float_type(gh), post_norm = truth(a[10]), kind = as_int(a[14]);
    const at::ScalarType xs = scalar(type), rs = scalar(stream_type);
    const void *ghp = dense(gh, rs, {T, n}, device), *gyp = dense(a[1], xs, {T, n}, device);
    const void* h = dense(a[3], rs, {T, n}, device);
    void *gx = dense_or_null(a[4], xs, {T, n}, device), *gr = dense_or_null(a[5], rs, {T, n}, device);
    auto* g_pre = static_cast<float*>(dense_or_null(a[6], at::kFloat, {n}, device));
    auto* g_post = static_cast<float*>(dense_or_null(a[7], at::kFloat, {n}, device));
    const NormParams p(a[11], a[12], a[9], post_norm, T, n, device);
    if (a[8] != Py_None && a[12] == Py_None) throw Unusual();
    auto* g_gate = a[8] == Py_None ? nullptr
                                   : static_cast<float*>(dense(a[8], at::kFloat, tensor(a[12]).sizes(), device));
    const float scale = as_float(a[13]), eps = as_float(a[15]);
    const Workspace w(a[16], device);
    void* s = stream_of(device);
    return released([&] {
      return fp8_norm_residual_backward(ghp, gyp, x.at, type, x.ld, h, stream_type, T, n, kind, eps, post_norm, p.post,
                                        p.gate, p.gate_rows, scale, p.pre, p.type, gx, gr, g_pre, g_post, g_gate, w.at,
                                        w.bytes, s);
    });
  });
}

PyObject* moe_few_tokens(PyObject*, PyObject* const* a, Py_ssize_t n_) {
  // x, expert_idx, weights, up, up_scales, down, down_scales, out, activation, workspace
  return guarded(n_, 10, [&] {
    const at::Tensor &xt = tensor(a[0]), &i = tensor(a[1]), &d = tensor(a[5]);
    const Matrix x(xt);
    if (xt.scalar_type() != at::kBFloat16 || i.dim() != 2 || d.dim() != 3 || a[9] == Py_None) throw Unusual();
    const int device = x.device, T = as_int(x.rows), hidden = as_int(x.cols), topk = as_int(i.size(1));
    const int E = as_int(d.size(0)), inter = as_int(d.size(2)), activation = as_int(a[8]);
    const auto* idx = static_cast<const int32_t*>(dense(i, at::kInt, {T, topk}, device));
    const auto* weights = static_cast<const float*>(dense_or_null(a[2], at::kFloat, {T, topk}, device));
    const int64_t kh = groups_of(hidden), ki = groups_of(inter);
    const uint8_t* up = codes(tensor(a[3]), FP8G_E4M3, {E, 2 * int64_t(inter), hidden}, device);
    const auto* us = static_cast<const float*>(dense(a[4], at::kFloat, {E, groups_of(2 * int64_t(inter)), kh}, device));
    const uint8_t* down = codes(d, FP8G_E4M3, {E, hidden, inter}, device);
    const auto* ds = static_cast<const float*>(dense(a[6], at::kFloat, {E, kh, ki}, device));
    auto* out = static_cast<uint16_t*>(dense(a[7], at::kBFloat16, {T, hidden}, device));
    const Workspace w(a[9], device);
    void* s = stream_of(device);
    return released([&] {
      return fp8_moe_few_tokens(static_cast<const uint16_t*>(x.at), x.ld, idx, weights, T, topk, up, us, down, ds, E,
                                hidden, inter, activation, out, w.at, w.bytes, s);
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
                           FP8G_DIRECT(gemm_nt_epilogue),
                           FP8G_DIRECT(epilogue_backward),
                           FP8G_DIRECT(norm_residual),
                           FP8G_DIRECT(norm_residual_backward),
                           FP8G_DIRECT(moe_few_tokens),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_direct", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__direct() { return PyModule_Create(&g_module); }
