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

// The workspace: the second kernel's arrival counters (always in the same place, so that no call's values lie where
// another's counters are), its slices' sums, then mid and its exponents.
constexpr size_t kCounterBytes = size_t(kMaxWidth / 16) * sizeof(unsigned long long);
struct Layout {
  int tokens;  // of a launch
  size_t partial, mid, exponents, bytes;
};
// Slices that `row_tiles` workgroups of the second kernel may be cut into: as many as there are CUs for.
int max_slices(int row_tiles) {
  int slices = 1;
  while (2 * slices <= fp8g::kFewMaxSlices && row_tiles * 2 * slices <= device_cus()) slices *= 2;
  return slices;
}

Layout layout(int num_tokens, int topk, int hidden, int inter) {
  Layout l{};
  l.tokens = std::min(num_tokens, chunk_tokens(topk));
  const size_t values = size_t(l.tokens) * topk * inter;
  l.partial = kCounterBytes;
  const int slices = max_slices(hidden / 32);
  l.mid = l.partial + (slices > 1 ? size_t(slices) * l.tokens * hidden * sizeof(float) : 0);
  l.exponents = l.mid + values * sizeof(uint16_t);
  l.bytes = l.exponents + values / fp8g::kFewGroup;
  return l;
}

// The second kernel, cut into slices where that leaves every workgroup 56 KB or more to stream (30 tokens, 40 experts of
// 768 x 384: 24.1 us, uncut 34.4; 64 tokens, 64 experts of 2048 x 768: 85 and 122; but one token, 8 experts of 2048 x
// 768, 98 KB in all: 18.2 cut in two, uncut 17.6).
template <int TX, int R, int WAVES, typename Plan>
int launch_down(const MoeFewArgs& a, int64_t tiles, hipStream_t s) {
  const int row_tiles = a.hidden / (16 * R);
  const int64_t bytes = tiles * 16 * R * a.inter;  // of a workgroup
  int slices = max_slices(row_tiles);
  while (slices > 1 && bytes / slices < 56 * 1024) slices /= 2;
  hipLaunchKernelGGL((fp8g::moe_few_down_kernel<TX, R, WAVES, Plan>), dim3(unsigned(row_tiles), unsigned(slices)),
                     dim3(WAVES * fp8g::kWave), 0, s, a);
  return launched("moe few down");
}

template <int TX, int R, typename Plan>
int launch_up(const MoeFewArgs& a, int64_t tiles, hipStream_t s) {
  const int64_t units = tiles * (a.inter / (8 * R));
  const int64_t grid = std::min<int64_t>(units, int64_t(device_cus()) * fp8g::kFewUpPerCu<TX>);
  hipLaunchKernelGGL((fp8g::moe_few_up_kernel<TX, R, Plan>), dim3(unsigned(grid)),
                     dim3(fp8g::kFewUpWaves * fp8g::kWave), 0, s, a);
  return launched("moe few up");
}

// Up to TX tokens.  Second kernel: 16 rows a workgroup as long as every one has a CU (one token, 4096 x 1408: 37.9 us, 39.3
// with 32 rows), else 32 (7168 x 2048: 67.7 us, 75.4 with 16).
template <int TX>
int launch_tokens(const MoeFewArgs& a, hipStream_t s) {
  using Plan = fp8g::FewTokenPlan<TX>;
  const int64_t tiles = std::min(a.tokens * a.topk, a.experts);
  if (const int st = launch_up<TX, 2, Plan>(a, tiles, s)) return st;
  return a.hidden / 16 <= device_cus() ? launch_down<TX, 1, 8, Plan>(a, tiles, s)
                                       : launch_down<TX, 2, 8, Plan>(a, tiles, s);
}

// Tiles of 16 pairs also where an expert has few: columns cost little (5 tokens, 64 experts of 2048 x 768: 37.5 us, 38.0
// by tiles of 4; 64 tokens, 16 experts of 4096 x 2048: 119.5, 269 by tiles of 4, 165 by 8).  32 rows of G and of U a unit
// halve what the activations and a unit's end cost (64 tokens, 128 experts of 7168 x 2048: 916 us, 970 with 16 rows; 64
// experts of 2048 x 768: 85.0 and 92.7); with few pairs an expert and long rows 16 share the work out more evenly (7
// tokens, 16 experts of 4096 x 2048: 70.6, 73.9 with 32; 16 tokens, 4 of 128 experts of 4096 x 1408: 143 and 148).
int launch_pairs(const MoeFewArgs& a, hipStream_t s) {
  using Plan = fp8g::FewPairPlan<16>;
  const int pairs = a.tokens * a.topk;
  const int64_t tiles = std::min(pairs, a.experts + pairs / 16);
  const bool wide = a.hidden <= 2048 || pairs >= 4 * a.experts;
  if (const int st = wide ? launch_up<16, 4, Plan>(a, tiles, s) : launch_up<16, 2, Plan>(a, tiles, s)) return st;
  return launch_down<16, 2, 4, Plan>(a, std::min(pairs, a.experts), s);
}

int launch(const MoeFewArgs& a, hipStream_t s) {
  if (a.tokens == 1) return launch_tokens<1>(a, s);
  if (a.tokens == 2) return launch_tokens<2>(a, s);
  return a.tokens <= 4 ? launch_tokens<4>(a, s) : launch_pairs(a, s);
}

}  // namespace

extern "C" {

size_t fp8_moe_few_tokens_workspace_bytes(int num_tokens, int topk, int hidden, int inter) {
  if (num_tokens <= 0 || topk <= 0 || topk > kMaxTopk || hidden <= 0 || inter <= 0) return 0;
  return layout(num_tokens, topk, hidden, inter).bytes;
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
  if (workspace_bytes < fp8_moe_few_tokens_workspace_bytes(num_tokens, topk, hidden, inter)) return FP8G_EINVAL;
  const Layout l = layout(num_tokens, topk, hidden, inter);
  char* const at = static_cast<char*>(workspace);
  for (int t = 0; t < num_tokens; t += l.tokens) {
    MoeFewArgs a{};
    a.x = x + t * x_ld; a.x_ld = x_ld;
    a.expert_idx = expert_idx + int64_t(t) * topk;
    a.weights = weights ? weights + int64_t(t) * topk : nullptr;
    a.up = up; a.up_scales = up_scales; a.down = down; a.down_scales = down_scales;
    a.counters = reinterpret_cast<unsigned long long*>(at); a.tag = counter_tag();
    a.partial = reinterpret_cast<float*>(at + l.partial);
    a.mid = reinterpret_cast<uint16_t*>(at + l.mid);
    a.exponents = reinterpret_cast<int8_t*>(at + l.exponents);
    a.out = out + int64_t(t) * hidden;
    a.tokens = std::min(l.tokens, num_tokens - t); a.topk = topk; a.experts = num_experts;
    a.hidden = hidden; a.inter = inter; a.activation = activation;
    auto s = static_cast<hipStream_t>(stream);
    if (const int st = launch(a, s)) return st;
  }
  return FP8G_OK;
}

}  // extern "C"
