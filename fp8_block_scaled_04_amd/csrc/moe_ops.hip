// Host side of expert routing and of the weighted combine (declared in
// fp8gemm.h): validation and launches.  Nothing here allocates, synchronises
// or reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "combine_kernel.hpp"
#include "fp8gemm.h"
#include "route_kernel.hpp"

namespace {

constexpr int64_t kRouteFullLanes = 2048 * 64;  // two waves on each SIMD of 256 CUs

// Up to this many tokens the combine's gradient takes a workgroup per pair.  Measured with 8 pairs a token: 32 tokens
// of 7168 4.0 us against 11.5 us for a workgroup per token, 256 of 4096 9.9 against 13.2, 512 of 4096 16.9 against
// 16.3, 4096 of 1024 53.1 against 39.1.
constexpr int kCombinePairTokens = 256;

constexpr int kCombineMaxColumns = 1 << 30;  // a thread's column is an int, and steps up to 8192 past the row's end

constexpr int64_t kMaxBlocks = 0xffffffff / 256;  // of 256 threads in a launch: their number is 32 bits

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

int log2_up(int v) {
  int n = 0;
  while ((1 << n) < v) ++n;
  return n;
}

template <typename L, int V, int KL>
int launch_route(const L* logits, int64_t ld, const float* bias, const fp8g::RouteShape& r, fp8g::RouteLanes lanes,
                 int32_t* expert_idx, float* weights, hipStream_t s) {
  const unsigned piece = std::min<unsigned>(V * sizeof(L), 16);
  lanes.vector = (r.E / r.groups) % V == 0 && ld * sizeof(L) % piece == 0 && aligned(logits, piece) &&
                 (!bias || aligned(bias, std::min(V * 4, 16)));
  const int64_t grid = cdiv64(int64_t(r.T) << lanes.log2_lanes, 256);
  if (grid > kMaxBlocks) return FP8G_EUNSUPPORTED;
  hipLaunchKernelGGL((fp8g::moe_route_kernel<L, V, KL>), dim3(unsigned(grid)), dim3(256), 0, s, logits, ld, bias, r,
                     lanes, expert_idx, weights);
  return launched();
}

template <typename L, int V>
int launch_route(const L* logits, int64_t ld, const float* bias, const fp8g::RouteShape& r, fp8g::RouteLanes lanes,
                 int32_t* expert_idx, float* weights, hipStream_t s) {
  if (r.topk <= 4) return launch_route<L, V, 4>(logits, ld, bias, r, lanes, expert_idx, weights, s);
  if (r.topk <= 8) return launch_route<L, V, 8>(logits, ld, bias, r, lanes, expert_idx, weights, s);
  if (r.topk <= 16) return launch_route<L, V, 16>(logits, ld, bias, r, lanes, expert_idx, weights, s);
  return launch_route<L, V, 32>(logits, ld, bias, r, lanes, expert_idx, weights, s);
}

// log2 of the lanes per token: enough waves to fill the device, at least
// 2^least, at most a wave and one per expert place (2^places).
int route_lanes(int num_tokens, int least, int places) {
  int n = 6;
  while (n > 0 && (int64_t(num_tokens) << (n - 1)) >= kRouteFullLanes) --n;
  return std::min(std::max(n, least), std::min(6, places));
}

template <typename L>
int launch_route(const L* logits, int64_t ld, const float* bias, const fp8g::RouteShape& r, int32_t* expert_idx,
                 float* weights, hipStream_t s) {
  const int group_log2 = log2_up(r.E / r.groups), groups_log2 = log2_up(r.groups);
  // a lane per group at least, and per 16 experts (16 against 32: 16.2 and 17.6 us for 32768 tokens of 256)
  const int n = route_lanes(r.T, std::max(groups_log2, groups_log2 + group_log2 - 4), groups_log2 + group_log2);
  const fp8g::RouteLanes lanes{n, n - groups_log2, 0};
  switch (std::max(0, group_log2 - lanes.log2_group_lanes)) {
    case 0: return launch_route<L, 1>(logits, ld, bias, r, lanes, expert_idx, weights, s);
    case 1: return launch_route<L, 2>(logits, ld, bias, r, lanes, expert_idx, weights, s);
    case 2: return launch_route<L, 4>(logits, ld, bias, r, lanes, expert_idx, weights, s);
    case 3: return launch_route<L, 8>(logits, ld, bias, r, lanes, expert_idx, weights, s);
    case 4: return launch_route<L, 16>(logits, ld, bias, r, lanes, expert_idx, weights, s);
    default: return launch_route<L, 32>(logits, ld, bias, r, lanes, expert_idx, weights, s);
  }
}

template <typename L, int V>
int launch_route_backward(const L* logits, int64_t ld, const int32_t* expert_idx, const float* grad_weights,
                          const fp8g::RouteShape& r, int n, L* grad, int64_t grad_ld, hipStream_t s) {
  const unsigned piece = std::min<unsigned>(V * sizeof(L), 16);
  const fp8g::RouteLanes lanes{n, n,
                               r.E % V == 0 && ld * sizeof(L) % piece == 0 && grad_ld * sizeof(L) % piece == 0 &&
                                   aligned(logits, piece) && aligned(grad, piece)};
  const int64_t grid = cdiv64(int64_t(r.T) << n, 256);
  if (grid > kMaxBlocks) return FP8G_EUNSUPPORTED;
  hipLaunchKernelGGL((fp8g::moe_route_backward_kernel<L, V>), dim3(unsigned(grid)), dim3(256), 0, s, logits, ld,
                     expert_idx, grad_weights, r, lanes, grad, grad_ld);
  return launched();
}

template <typename L>
int launch_route_backward(const L* logits, int64_t ld, const int32_t* expert_idx, const float* grad_weights,
                          const fp8g::RouteShape& r, L* grad, int64_t grad_ld, hipStream_t s) {
  const int places = std::max(log2_up(r.E), log2_up(r.topk));
  const int n = route_lanes(r.T, std::max(log2_up(r.topk), places - 4), places);  // a lane per pick at least
  switch (places - n) {
    case 0: return launch_route_backward<L, 1>(logits, ld, expert_idx, grad_weights, r, n, grad, grad_ld, s);
    case 1: return launch_route_backward<L, 2>(logits, ld, expert_idx, grad_weights, r, n, grad, grad_ld, s);
    case 2: return launch_route_backward<L, 4>(logits, ld, expert_idx, grad_weights, r, n, grad, grad_ld, s);
    case 3: return launch_route_backward<L, 8>(logits, ld, expert_idx, grad_weights, r, n, grad, grad_ld, s);
    default: return launch_route_backward<L, 16>(logits, ld, expert_idx, grad_weights, r, n, grad, grad_ld, s);
  }
}

int check_combine(int rows, int n, const int32_t* dst_row, const float* weights, int num_tokens, int topk) {
  if (rows < 0 || n < 0 || num_tokens < 0 || topk < 1) return FP8G_EINVAL;
  if (n % 8 != 0 || n > kCombineMaxColumns) return FP8G_EUNSUPPORTED;
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
  auto s = static_cast<hipStream_t>(stream);
  return logits_dtype == FP8G_F32
             ? launch_route(static_cast<const float*>(logits), logits_ld, bias, r, expert_idx, weights, s)
             : launch_route(static_cast<const uint16_t*>(logits), logits_ld, bias, r, expert_idx, weights, s);
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
  auto s = static_cast<hipStream_t>(stream);
  return logits_dtype == FP8G_F32
             ? launch_route_backward(static_cast<const float*>(logits), logits_ld, expert_idx, grad_weights, r,
                                     static_cast<float*>(grad_logits), grad_ld, s)
             : launch_route_backward(static_cast<const uint16_t*>(logits), logits_ld, expert_idx, grad_weights, r,
                                     static_cast<uint16_t*>(grad_logits), grad_ld, s);
}

int fp8_moe_combine(const uint16_t* y, int y_rows, int n, const int32_t* dst_row, const float* weights,
                    int num_tokens, int topk, uint16_t* out, void* stream) {
  if (int st = check_combine(y_rows, n, dst_row, weights, num_tokens, topk)) return st;
  if (num_tokens == 0 || n == 0) return FP8G_OK;
  if (!out || !aligned(out, 16) || (y_rows > 0 && !y) || (y && !aligned(y, 16))) return FP8G_EINVAL;
  for (int64_t first = 0; first < num_tokens; first += kMaxBlocks)
    hipLaunchKernelGGL(fp8g::moe_combine_kernel,
                       dim3(unsigned(std::min(num_tokens - first, kMaxBlocks)), unsigned(cdiv64(n, 2048))), dim3(256),
                       0, static_cast<hipStream_t>(stream), y, y_rows, n, dst_row, weights, topk, out, first);
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
  const int64_t pairs = int64_t(num_tokens) * topk;
  auto s = static_cast<hipStream_t>(stream);
  if (num_tokens <= kCombinePairTokens && pairs <= kMaxBlocks) {
    hipLaunchKernelGGL(fp8g::moe_combine_backward_kernel<true>, dim3(unsigned(pairs)), dim3(256), 0, s, grad_out, y,
                       y_rows, n, dst_row, weights, topk, grad_y, grad_weights, int64_t(0));
    return launched();
  }
  for (int64_t first = 0; first < num_tokens; first += kMaxBlocks)
    hipLaunchKernelGGL(fp8g::moe_combine_backward_kernel<false>,
                       dim3(unsigned(std::min(num_tokens - first, kMaxBlocks))), dim3(256), 0, s, grad_out, y, y_rows,
                       n, dst_row, weights, topk, grad_y, grad_weights, first);
  return launched();
}

}  // extern "C"
