// Host side of expert routing and of the weighted combine (declared in
// fp8gemm.h): validation and launches.  Nothing here allocates, synchronises
// or reads device memory.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "combine_kernel.hpp"
#include "fp8gemm.h"
#include "route_kernel.hpp"

namespace {

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
int launched() { return hipGetLastError() == hipSuccess ? FP8G_OK : FP8G_ELAUNCH; }

// Checks common to the routing and its gradient.
int check_route(int logits_dtype, int64_t ld, int num_tokens, int num_experts, int score_func, int topk) {
  if (logits_dtype != FP8G_F32 && logits_dtype != FP8G_BF16) return FP8G_EINVAL;
  if (score_func != FP8G_SOFTMAX && score_func != FP8G_SIGMOID) return FP8G_EINVAL;
  if (num_tokens < 0 || num_experts < 1 || ld < num_experts || topk < 1 || topk > num_experts) return FP8G_EINVAL;
  if (num_experts > fp8g::kRouteMaxExperts || topk > fp8g::kRouteMaxTopk) return FP8G_EUNSUPPORTED;
  return FP8G_OK;
}

int check_combine(int rows, int n, const int32_t* dst_row, const float* weights, int num_tokens, int topk) {
  if (rows < 0 || n < 0 || num_tokens < 0 || topk < 1) return FP8G_EINVAL;
  if (n % 8 != 0) return FP8G_EUNSUPPORTED;
  if ((dst_row && !aligned(dst_row, 4)) || (weights && !aligned(weights, 4))) return FP8G_EINVAL;
  return FP8G_OK;
}

}  // namespace

extern "C" {

int fp8_moe_route(const void* logits, int logits_dtype, int64_t logits_ld, const float* bias, int num_tokens,
                  int num_experts, int score_func, int expert_groups, int topk_groups, int group_score, int topk,
                  int renormalize, float scale, int32_t* expert_idx, float* weights, void* stream) {
  if (int st = check_route(logits_dtype, logits_ld, num_tokens, num_experts, score_func, topk)) return st;
  if (group_score != FP8G_GROUP_MAX && group_score != FP8G_GROUP_TOP2) return FP8G_EINVAL;
  if (expert_groups < 1 || num_experts % expert_groups != 0 || topk_groups < 1 || topk_groups > expert_groups ||
      int64_t(num_experts / expert_groups) * topk_groups < topk)
    return FP8G_EINVAL;
  if (expert_groups > fp8g::kRouteMaxGroups) return FP8G_EUNSUPPORTED;
  if (num_tokens == 0) return FP8G_OK;
  if (!logits || !expert_idx || !weights) return FP8G_EINVAL;
  if (!aligned(logits, logits_dtype == FP8G_F32 ? 4 : 2) || (bias && !aligned(bias, 4)) || !aligned(expert_idx, 4) ||
      !aligned(weights, 4))
    return FP8G_EINVAL;
  const fp8g::RouteShape r{num_tokens, num_experts, expert_groups, topk_groups, topk,
                           score_func, group_score, renormalize != 0, scale};
  const dim3 grid(unsigned(cdiv64(num_tokens, 4)));
  auto s = static_cast<hipStream_t>(stream);
  if (logits_dtype == FP8G_F32)
    hipLaunchKernelGGL(fp8g::moe_route_kernel<float>, grid, dim3(256), 0, s, static_cast<const float*>(logits),
                       logits_ld, bias, r, expert_idx, weights);
  else
    hipLaunchKernelGGL(fp8g::moe_route_kernel<uint16_t>, grid, dim3(256), 0, s, static_cast<const uint16_t*>(logits),
                       logits_ld, bias, r, expert_idx, weights);
  return launched();
}

int fp8_moe_route_backward(const void* logits, int logits_dtype, int64_t logits_ld, const int32_t* expert_idx,
                           const float* grad_weights, int num_tokens, int num_experts, int score_func, int topk,
                           int renormalize, float scale, void* grad_logits, int64_t grad_ld, void* stream) {
  if (int st = check_route(logits_dtype, logits_ld, num_tokens, num_experts, score_func, topk)) return st;
  if (grad_ld < num_experts) return FP8G_EINVAL;
  if (num_tokens == 0) return FP8G_OK;
  if (!logits || !expert_idx || !grad_weights || !grad_logits) return FP8G_EINVAL;
  const unsigned a = logits_dtype == FP8G_F32 ? 4 : 2;
  if (!aligned(logits, a) || !aligned(grad_logits, a) || !aligned(expert_idx, 4) || !aligned(grad_weights, 4))
    return FP8G_EINVAL;
  const fp8g::RouteShape r{num_tokens, num_experts, 1, 1, topk, score_func, 0, renormalize != 0, scale};
  const dim3 grid(unsigned(cdiv64(num_tokens, 4)));
  auto s = static_cast<hipStream_t>(stream);
  if (logits_dtype == FP8G_F32)
    hipLaunchKernelGGL(fp8g::moe_route_backward_kernel<float>, grid, dim3(256), 0, s,
                       static_cast<const float*>(logits), logits_ld, expert_idx, grad_weights, r,
                       static_cast<float*>(grad_logits), grad_ld);
  else
    hipLaunchKernelGGL(fp8g::moe_route_backward_kernel<uint16_t>, grid, dim3(256), 0, s,
                       static_cast<const uint16_t*>(logits), logits_ld, expert_idx, grad_weights, r,
                       static_cast<uint16_t*>(grad_logits), grad_ld);
  return launched();
}

int fp8_moe_combine(const uint16_t* y, int y_rows, int n, const int32_t* dst_row, const float* weights,
                    int num_tokens, int topk, uint16_t* out, void* stream) {
  if (int st = check_combine(y_rows, n, dst_row, weights, num_tokens, topk)) return st;
  if (num_tokens == 0 || n == 0) return FP8G_OK;
  if (!out || !aligned(out, 16) || (y_rows > 0 && !y) || (y && !aligned(y, 16))) return FP8G_EINVAL;
  hipLaunchKernelGGL(fp8g::moe_combine_kernel, dim3(unsigned(num_tokens), unsigned(cdiv64(n, 2048))), dim3(256), 0,
                     static_cast<hipStream_t>(stream), y, y_rows, n, dst_row, weights, topk, out);
  return launched();
}

int fp8_moe_combine_backward(const uint16_t* grad_out, const uint16_t* y, int y_rows, int n, const int32_t* dst_row,
                             const float* weights, int num_tokens, int topk, uint16_t* grad_y, float* grad_weights,
                             void* stream) {
  if (int st = check_combine(y_rows, n, dst_row, weights, num_tokens, topk)) return st;
  if (grad_weights && !aligned(grad_weights, 4)) return FP8G_EINVAL;
  if (num_tokens == 0) return FP8G_OK;
  if (n > 0 && (!grad_out || !aligned(grad_out, 16))) return FP8G_EINVAL;
  if (n > 0 && y_rows > 0 && (!grad_y || !aligned(grad_y, 16) || (grad_weights && (!y || !aligned(y, 16)))))
    return FP8G_EINVAL;
  if (n == 0 && !grad_weights) return FP8G_OK;
  hipLaunchKernelGGL(fp8g::moe_combine_backward_kernel, dim3(unsigned(num_tokens)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), grad_out, y, y_rows, n, dst_row, weights, topk, grad_y,
                     grad_weights);
  return launched();
}

}  // extern "C"
