// Host side of the mixture-of-experts layer for a few tokens (declared in
// fp8gemm.h): validation and launches.  Nothing here allocates, synchronises or
// reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8gemm.h"
#include "host_common.hpp"
#include "moe_few_kernel.hpp"

namespace {

using fp8g::MoeFewArgs;
using namespace fp8g::host;

constexpr int kMaxTopk = fp8g::kFewMaxTopk, kMaxExperts = fp8g::kFewMaxExperts, kMaxWidth = 65536;

// Tokens that one pair of launches takes.
int chunk_tokens(int topk) { return std::min(fp8g::kFewTokens, fp8g::kFewMaxPairs / topk); }

template <int TX, int R, int WAVES, typename Plan>
int launch_down(const MoeFewArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((fp8g::moe_few_down_kernel<TX, R, WAVES, Plan>), dim3(unsigned(a.hidden / (16 * R))),
                     dim3(WAVES * fp8g::kWave), 0, s, a);
  return launched("moe few down");
}

template <int TX, typename Plan, int DOWN2_WAVES>
int launch_both(const MoeFewArgs& a, int64_t tiles, hipStream_t s) {
  const int64_t units = tiles * (a.inter / fp8g::kFewGroup);
  const int64_t grid = std::min<int64_t>(units, int64_t(device_cus()) * fp8g::few_up_per_cu(TX));
  hipLaunchKernelGGL((fp8g::moe_few_up_kernel<TX, Plan>), dim3(unsigned(grid)),
                     dim3(fp8g::kFewUpWaves * fp8g::kWave), 0, s, a);
  if (const int st = launched("moe few up")) return st;
  return a.hidden / 16 <= device_cus() ? launch_down<TX, 1, 8, Plan>(a, s) : launch_down<TX, 2, DOWN2_WAVES, Plan>(a, s);
}

template <int TX>
int launch_tokens(const MoeFewArgs& a, hipStream_t s) {
  return launch_both<TX, fp8g::FewTokenPlan<TX>, 8>(a, std::min(a.tokens * a.topk, a.experts), s);
}

template <int TX>
int launch_pairs(const MoeFewArgs& a, hipStream_t s) {
  const int pairs = a.tokens * a.topk;
  return launch_both<TX, fp8g::FewPairPlan<TX>, 4>(a, std::min(pairs, a.experts + pairs / TX), s);
}

int launch(const MoeFewArgs& a, hipStream_t s) {
  if (a.tokens == 1) return launch_tokens<1>(a, s);
  if (a.tokens == 2) return launch_tokens<2>(a, s);
  if (a.tokens <= 4) return launch_tokens<4>(a, s);
  const int pairs = a.tokens * a.topk;
  if (pairs <= 2 * a.experts) return launch_pairs<4>(a, s);
  if (pairs <= 6 * a.experts) return launch_pairs<8>(a, s);
  return launch_pairs<16>(a, s);
}

}  // namespace

extern "C" {

size_t fp8_moe_few_tokens_workspace_bytes(int num_tokens, int topk, int inter) {
  if (num_tokens <= 0 || topk <= 0 || topk > kMaxTopk || inter <= 0) return 0;
  const size_t values = size_t(std::min(num_tokens, chunk_tokens(topk))) * size_t(topk) * size_t(inter);
  return values * sizeof(uint16_t) + values / fp8g::kFewGroup;
}

int fp8_moe_few_tokens(const uint16_t* x, int64_t x_ld, const int32_t* expert_idx, const float* weights,
                       int num_tokens, int topk, const uint8_t* up, const float* up_scales, const uint8_t* down,
                       const float* down_scales, int num_experts, int hidden, int inter, int activation,
                       uint16_t* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (num_tokens < 0 || topk < 1 || num_experts < 1 || hidden < 0 || inter < 0) return FP8G_EINVAL;
  if (activation < FP8G_ACT_NONE || activation > FP8G_ACT_SILU || x_ld < hidden) return FP8G_EINVAL;
  if (topk > kMaxTopk || num_experts > kMaxExperts || hidden % 128 != 0 || inter % 128 != 0 || inter == 0 ||
      hidden > kMaxWidth || inter > kMaxWidth || x_ld % 8 != 0)
    return FP8G_EUNSUPPORTED;
  if (num_tokens == 0 || hidden == 0) return FP8G_OK;
  if (!x || !expert_idx || !up || !up_scales || !down || !down_scales || !out || !workspace) return FP8G_EINVAL;
  if (!aligned16(x) || !aligned16(up) || !aligned16(up_scales) || !aligned16(down) || !aligned16(down_scales) ||
      !aligned16(out) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(expert_idx) & 3) ||
      (reinterpret_cast<uintptr_t>(weights) & 3))
    return FP8G_EINVAL;
  if (workspace_bytes < fp8_moe_few_tokens_workspace_bytes(num_tokens, topk, inter)) return FP8G_EINVAL;
  const int step = chunk_tokens(topk);
  for (int t = 0; t < num_tokens; t += step) {
    MoeFewArgs a{};
    a.x = x + t * x_ld; a.x_ld = x_ld;
    a.expert_idx = expert_idx + int64_t(t) * topk;
    a.weights = weights ? weights + int64_t(t) * topk : nullptr;
    a.up = up; a.up_scales = up_scales; a.down = down; a.down_scales = down_scales;
    a.mid = static_cast<uint16_t*>(workspace);
    a.exponents = reinterpret_cast<int8_t*>(a.mid + size_t(std::min(step, num_tokens)) * topk * inter);
    a.out = out + int64_t(t) * hidden;
    a.tokens = std::min(step, num_tokens - t); a.topk = topk; a.experts = num_experts;
    a.hidden = hidden; a.inter = inter; a.activation = activation;
    auto s = static_cast<hipStream_t>(stream);
    if (const int st = launch(a, s)) return st;
  }
  return FP8G_OK;
}

}  // extern "C"
