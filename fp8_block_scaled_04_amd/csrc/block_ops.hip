// Host side of the norms between blocks and of the dense epilogue's gradients
// (declared in fp8gemm.h): validation and launches.  Nothing here allocates,
// synchronises or reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "epilogue_grad_kernel.hpp"
#include "fp8gemm.h"
#include "norm_kernel.hpp"

namespace {

using fp8g::NormArgs;
using fp8g::NormGradArgs;

constexpr int kNormMaxColumns = 16384;  // 8 columns x 4 pieces x 512 threads
// Workgroups of a gradient's pass, at most: what 256 CUs hold at once, by their registers 1024 threads each.
constexpr int grad_slices(int n) { return n > 4096 ? 256 : 512; }
constexpr int64_t kMaxBlocks = 0xffffffff / 1024;  // workgroups of up to 1024 threads: their number is 32 bits
constexpr int kMaxRows = 1 << 30;  // the kernels' row numbers are 32 bits, with room for a slice behind the last

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int launched() { return hipGetLastError() == hipSuccess ? FP8G_OK : FP8G_ELAUNCH; }
bool float_type(int t) { return t == FP8G_F32 || t == FP8G_BF16; }

template <typename... P>
bool all_aligned16(P... p) {
  return (aligned16(p) && ...);
}

int check_norm(int num_rows, int n, int kind, int x_dtype, int stream_dtype, int param_dtype, int gate_rows,
               const void* gate, float eps) {
  if (num_rows < 0 || n < 0 || (kind != FP8G_NORM_RMS && kind != FP8G_NORM_LAYER)) return FP8G_EINVAL;
  if (!float_type(x_dtype) || !float_type(stream_dtype) || !float_type(param_dtype) || !(eps >= 0.f))
    return FP8G_EINVAL;
  if (gate && gate_rows != 1 && gate_rows != num_rows) return FP8G_EINVAL;
  if (n % 8 != 0 || n > kNormMaxColumns || num_rows > kMaxRows) return FP8G_EUNSUPPORTED;
  return FP8G_OK;
}

// f(X{}, R{}, layer) for the types of x and of the residual stream.
template <typename F>
int by_types(int x_dtype, int stream_dtype, int kind, F&& f) {
  auto with = [&](auto x, auto r) {
    return kind == FP8G_NORM_LAYER ? f(x, r, std::true_type{}) : f(x, r, std::false_type{});
  };
  if (x_dtype == FP8G_F32) return stream_dtype == FP8G_F32 ? with(float{}, float{}) : with(float{}, uint16_t{});
  return stream_dtype == FP8G_F32 ? with(uint16_t{}, float{}) : with(uint16_t{}, uint16_t{});
}

template <typename X, typename R, bool LAYER, int C>
int launch_norm(const NormArgs& a, hipStream_t s) {
  const int threads = int(cdiv(cdiv(a.n / 8, C), 64) * 64), rows = threads == 64 ? 4 : 1;
  const int64_t blocks = cdiv(a.rows, rows);
  if (blocks > kMaxBlocks) return FP8G_EUNSUPPORTED;
  hipLaunchKernelGGL((fp8g::norm_residual_kernel<X, R, LAYER, C>), dim3(unsigned(blocks)),
                     dim3(unsigned(threads), unsigned(rows)), 0, s, a);
  return launched();
}

// Rows that a workgroup of the gradients takes at a time: what 512 threads hold, a piece of 8 columns each.
int grad_rows(int n) { return n > 4096 ? 1 : std::min<int>(fp8g::kNormGradRows, int(512 / (cdiv(n, 512) * 64))); }

template <typename X, typename R, bool LAYER, bool ROW_GATE, int C, int MAX_THREADS, bool IN_LDS>
int launch_norm_backward(const NormGradArgs& a, int slices, hipStream_t s) {
  const int threads = int(cdiv(cdiv(a.n / 8, C), 64) * 64), rows = grad_rows(a.n);
  const int of_rows = rows > 1 ? rows * threads * 8 : C > 1 ? 2 * a.n : 0;  // floats: sums of rows, or over them
  const int lds = std::max(IN_LDS ? 3 * a.n : 0, of_rows) * int(sizeof(float));
  hipLaunchKernelGGL((fp8g::norm_residual_backward_kernel<X, R, LAYER, ROW_GATE, C, MAX_THREADS, IN_LDS>),
                     dim3(unsigned(slices)), dim3(unsigned(threads), unsigned(rows)), lds, s, a);
  return launched();
}

template <typename X, typename R, bool LAYER, bool ROW_GATE>
int launch_norm_backward(const NormGradArgs& a, int slices, hipStream_t s) {
  if (a.n > 8192) return launch_norm_backward<X, R, LAYER, ROW_GATE, 2, 1024, false>(a, slices, s);
  const bool again = a.rows_per_slice > grad_rows(a.n);  // more than one round: the parameters are read again
  if (grad_rows(a.n) == 1)
    return again ? launch_norm_backward<X, R, LAYER, ROW_GATE, 1, 1024, true>(a, slices, s)
                 : launch_norm_backward<X, R, LAYER, ROW_GATE, 1, 1024, false>(a, slices, s);
  return again ? launch_norm_backward<X, R, LAYER, ROW_GATE, 1, 512, true>(a, slices, s)
               : launch_norm_backward<X, R, LAYER, ROW_GATE, 1, 512, false>(a, slices, s);
}

// Rows of a slice and slices of a gradient's pass.
int slice_rows(int64_t rows, int64_t at_most) { return int(cdiv(rows, std::min<int64_t>(rows, at_most))); }

// The same for the gradients of the norms: two rounds at least where there are many, so that the sums are of fewer slices
// (512 x 4096: 16.7 us, 19.3 with a row each; but 257 x 2048 11.7 us, 13.3 with two).
int norm_slice_rows(int rows, int n) {
  const int at_once = grad_rows(n);
  const int64_t groups = cdiv(rows, at_once);
  return at_once * std::max(slice_rows(groups, grad_slices(n)), groups > 384 ? 2 : 1);
}

void launch_column_sums(const float* partial, int slices, int sets, int n, float* out0, float* out1, float* out2,
                        hipStream_t s) {
  hipLaunchKernelGGL(fp8g::column_sums_kernel, dim3(unsigned(cdiv(n, 64)), unsigned(sets)),
                     dim3(64 * fp8g::kSumRuns), 0, s, partial, slices, n, out0, out1, out2);
}

// Slices of the epilogue's gradients: about 8192 workgroups, 32 rows each at least, so that those of a CU are at all
// stages at once (8192 x 4096 39.8 us, 42.3 with 2048 workgroups; 16384 x 4096 73.8 and 79.6; 2048 x 4096 12.6, 14.5 with
// 64 rows); but 512 slices at most, whose sums are the second kernel's work (32768 x 512: 23.9 us, 26.1 with 1024).
int epilogue_slice_rows(int m, int n) {
  const int64_t columns = cdiv(n, fp8g::kEpilogueColumns);
  return int(std::max<int64_t>(32, slice_rows(m, std::clamp<int64_t>(8192 / columns, 1, 512))));
}

}  // namespace

extern "C" {

size_t fp8_epilogue_backward_workspace_bytes(int m, int n) {
  if (m <= 0 || n <= 0) return 0;
  const int64_t slices = cdiv(m, epilogue_slice_rows(m, n));
  return slices > 1 ? size_t(slices) * size_t(n) * sizeof(float) : 0;
}

int fp8_epilogue_backward(const uint16_t* grad_out, const uint16_t* preact, int activation, int m, int n,
                          uint16_t* grad_preact, float* grad_bias, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (m < 0 || n < 0 || activation < FP8G_ACT_NONE || activation > FP8G_ACT_SILU) return FP8G_EINVAL;
  if (n % 8 != 0 || m > kMaxRows || cdiv(n, 64) > kMaxBlocks) return FP8G_EUNSUPPORTED;
  if (n == 0) return FP8G_OK;
  auto s = static_cast<hipStream_t>(stream);
  if (grad_bias && !aligned16(grad_bias)) return FP8G_EINVAL;
  if (m == 0) {
    if (!grad_bias) return FP8G_OK;
    launch_column_sums(nullptr, 0, 1, n, grad_bias, nullptr, nullptr, s);  // sums of nothing
    return launched();
  }
  if (!grad_out || !preact || !grad_preact || !all_aligned16(grad_out, preact, grad_preact, workspace))
    return FP8G_EINVAL;
  const int rows = epilogue_slice_rows(m, n);
  const int64_t slices = cdiv(m, rows), columns = cdiv(n, fp8g::kEpilogueColumns);
  float* partial = grad_bias;
  if (grad_bias && slices > 1) {
    if (!workspace || workspace_bytes < fp8_epilogue_backward_workspace_bytes(m, n)) return FP8G_EINVAL;
    partial = static_cast<float*>(workspace);
  }
  hipLaunchKernelGGL(fp8g::epilogue_backward_kernel, dim3(unsigned(columns), unsigned(slices)), dim3(256), 0, s,
                     grad_out, preact, activation, m, n, rows, grad_preact, partial);
  if (const int st = launched()) return st;
  if (partial == grad_bias) return FP8G_OK;
  launch_column_sums(partial, int(slices), 1, n, grad_bias, nullptr, nullptr, s);
  return launched();
}

int fp8_norm_residual(const void* x, int x_dtype, int64_t x_ld, const void* residual, int64_t residual_ld,
                      int stream_dtype, int num_rows, int n, int kind, float eps, int post_norm,
                      const void* post_weight, const void* gate, int gate_rows, float residual_scale,
                      const void* pre_weight, int param_dtype, void* h, void* y, uint8_t* q, int q_format,
                      float* q_scales, int64_t q_scales_ld, void* stream) {
  if (int st = check_norm(num_rows, n, kind, x_dtype, stream_dtype, param_dtype, gate_rows, gate, eps)) return st;
  if (q_format != FP8G_E4M3 && q_format != FP8G_E5M2) return FP8G_EINVAL;
  if (x_ld < n || (residual && residual_ld < n)) return FP8G_EINVAL;
  if (x_ld % 8 != 0 || (residual && residual_ld % 8 != 0)) return FP8G_EUNSUPPORTED;
  if (q && q_scales_ld < num_rows) return FP8G_EUNSUPPORTED;
  if (num_rows == 0 || n == 0) return FP8G_OK;
  if (!x || (!h && !y && !q) || (q && !q_scales)) return FP8G_EINVAL;
  if (!all_aligned16(x, residual, post_weight, gate, pre_weight, h, y, q, q_scales)) return FP8G_EINVAL;
  NormArgs a{};
  a.x = x; a.residual = residual; a.post_weight = post_weight; a.gate = gate; a.pre_weight = pre_weight;
  a.h = h; a.y = y; a.q = q; a.q_scales = q_scales;
  a.x_ld = x_ld; a.residual_ld = residual_ld; a.q_ld = q_scales_ld;
  a.rows = num_rows; a.n = n;
  a.post_norm = post_norm != 0; a.gate_per_row = gate && gate_rows != 1; a.params_bf16 = param_dtype == FP8G_BF16;
  a.q_e5m2 = q_format == FP8G_E5M2;
  a.eps = eps; a.residual_scale = residual_scale;
  auto s = static_cast<hipStream_t>(stream);
  return by_types(x_dtype, stream_dtype, kind, [&](auto x_, auto r_, auto layer) {
    using X = decltype(x_);
    using R = decltype(r_);
    constexpr bool L = decltype(layer)::value;
    if (n > 8192) return launch_norm<X, R, L, 4>(a, s);
    // Two pieces a thread for many long rows: 16384 x 7168 174 us, 218 with one, 184 with four; but 8192 x 4096 54.9 us
    // with one and 61.6 with two, a row of 7168 4.8 and 5.1.
    if (n > 4096 && num_rows > 1024) return launch_norm<X, R, L, 2>(a, s);
    return launch_norm<X, R, L, 1>(a, s);
  });
}

size_t fp8_norm_residual_backward_workspace_bytes(int num_rows, int n) {
  if (num_rows <= 0 || n <= 0) return 0;
  return size_t(cdiv(num_rows, norm_slice_rows(num_rows, n))) * 3 * size_t(n) * sizeof(float);
}

int fp8_norm_residual_backward(const void* grad_h, const void* grad_y, const void* x, int x_dtype, int64_t x_ld,
                               const void* h, int stream_dtype, int num_rows, int n, int kind, float eps,
                               int post_norm, const void* post_weight, const void* gate, int gate_rows,
                               float residual_scale, const void* pre_weight, int param_dtype, void* grad_x,
                               void* grad_residual, float* grad_pre_weight, float* grad_post_weight, float* grad_gate,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_norm(num_rows, n, kind, x_dtype, stream_dtype, param_dtype, gate_rows, gate, eps)) return st;
  if (x && x_ld < n) return FP8G_EINVAL;
  if (x && x_ld % 8 != 0) return FP8G_EUNSUPPORTED;
  if ((grad_post_weight && !post_norm) || (grad_gate && !gate)) return FP8G_EINVAL;
  if (n == 0) return FP8G_OK;
  if (!all_aligned16(grad_h, grad_y, x, h, post_weight, gate, pre_weight, grad_x, grad_residual, grad_pre_weight,
                     grad_post_weight, grad_gate, workspace))
    return FP8G_EINVAL;
  auto s = static_cast<hipStream_t>(stream);
  float* shared_gate = gate && gate_rows == 1 ? grad_gate : nullptr;
  const bool sums = grad_pre_weight || grad_post_weight || shared_gate;
  if (num_rows == 0) {
    if (!sums) return FP8G_OK;
    launch_column_sums(nullptr, 0, 3, n, grad_pre_weight, grad_post_weight, shared_gate, s);  // sums of nothing
    return launched();
  }
  if ((!grad_h && !grad_y) || (grad_y && !h) || (!x && (post_norm || gate)) || (grad_pre_weight && !grad_y))
    return FP8G_EINVAL;
  if (!grad_x && !grad_residual && !grad_gate && !sums) return FP8G_EINVAL;
  if (sums && (!workspace || workspace_bytes < fp8_norm_residual_backward_workspace_bytes(num_rows, n)))
    return FP8G_EINVAL;
  NormGradArgs a{};
  a.grad_h = grad_h; a.grad_y = grad_y; a.x = post_norm || gate ? x : nullptr; a.h = h;
  a.post_weight = post_norm ? post_weight : nullptr; a.gate = gate; a.pre_weight = pre_weight;
  a.grad_x = grad_x; a.grad_residual = grad_residual;
  a.grad_gate = gate && gate_rows != 1 ? grad_gate : nullptr;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  a.x_ld = x_ld;
  a.rows = num_rows; a.n = n; a.rows_per_slice = norm_slice_rows(num_rows, n);
  a.post_norm = post_norm != 0; a.params_bf16 = param_dtype == FP8G_BF16;
  a.eps = eps; a.residual_scale = residual_scale;
  const int slices = int(cdiv(num_rows, a.rows_per_slice));
  const int st = by_types(x_dtype, stream_dtype, kind, [&](auto x_, auto r_, auto layer) {
    using X = decltype(x_);
    using R = decltype(r_);
    constexpr bool L = decltype(layer)::value;
    return gate && gate_rows != 1 ? launch_norm_backward<X, R, L, true>(a, slices, s)
                                  : launch_norm_backward<X, R, L, false>(a, slices, s);
  });
  if (st || !sums) return st;
  launch_column_sums(a.partial, slices, 3, n, grad_pre_weight, grad_post_weight, shared_gate, s);
  return launched();
}

}  // extern "C"
