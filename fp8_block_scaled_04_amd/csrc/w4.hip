// Host side of the 4-bit matrix-vector products (declared in fp8gemm.h):
// validation and launches.  Nothing here allocates, synchronises or reads
// device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8gemm.h"
#include "w4_kernel.hpp"

namespace {

using fp8g::W4Args;

constexpr int kFullWaves = 2048;      // 8 on each of 256 CUs
constexpr int kStreamBytes = 64 * 1024;  // activations of a streaming workgroup, at most
constexpr int kStreamWorkgroups = 2048;   // workgroups a long stream is dealt to
constexpr int kMaxColumns = 1 << 20;  // row offsets within a workgroup's 256 rows fit 32 bits

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check(const W4Args& a, int w_format, int scales_dtype, int out_dtype, int group, bool* empty) {
  *empty = false;
  if (w_format != FP8G_INT4 && w_format != FP8G_E2M1) return FP8G_EINVAL;
  if (scales_dtype != FP8G_F32 && scales_dtype != FP8G_BF16) return FP8G_EINVAL;
  if (out_dtype != FP8G_F32 && out_dtype != FP8G_BF16) return FP8G_EINVAL;
  if (a.m < 0 || a.n < 0 || a.k < 0 || a.x_ld < a.k) return FP8G_EINVAL;
  if (w_format == FP8G_E2M1 && a.zeros) return FP8G_EINVAL;
  if ((group != 32 && group != 64 && group != 128) || a.k % group != 0 || a.k > kMaxColumns || a.x_ld % 8 != 0)
    return FP8G_EUNSUPPORTED;
  if (a.m == 0 || a.n == 0) {
    *empty = true;
    return FP8G_OK;
  }
  if (!a.out || !aligned(a.out, 16)) return FP8G_EINVAL;
  if (a.k > 0) {
    if (!a.x || !a.w || !a.scales) return FP8G_EINVAL;
    if (!aligned(a.x, 16) || !aligned(a.w, 16) || !aligned(a.scales, 16) || (a.zeros && !aligned(a.zeros, 16)))
      return FP8G_EINVAL;
  }
  return FP8G_OK;
}

int64_t cdiv64(int64_t x, int64_t y) { return (x + y - 1) / y; }

template <int FMT, bool Z, int G, int TX, int R, int U, bool ROUTED>
int launch_kernel(W4Args a, hipStream_t s) {
  a.by_pair = ROUTED && a.m <= a.experts;
  const int64_t slots = !ROUTED ? cdiv64(a.m, TX) : a.by_pair ? a.m : int64_t(a.experts) + 1;
  if (slots > 65535) return FP8G_EUNSUPPORTED;
  const int64_t sets = cdiv64(a.n, 16 * R) * slots, blocks = cdiv64(a.k, 128 * U);
  // Rows for every place of the CUs, and a tile's activations fit LDS: whole rows per wave.
  const int64_t x_bytes = (blocks * (256 * U) + 1023) / 1024 * 1024 * TX;
  if (sets >= kFullWaves && x_bytes <= kStreamBytes) {
    using L = fp8g::W4StreamRing<Z, G, TX, R, U>;
    const int64_t row_sets = cdiv64(a.n, 16 * R);
    a.reps = int(std::max<int64_t>(1, sets / (fp8g::kW4Waves * kStreamWorkgroups)));
    const int lds = fp8g::kW4Waves * L::kWave + int(x_bytes);
    hipLaunchKernelGGL((fp8g::w4_stream_kernel<FMT, Z, G, TX, R, U, ROUTED>),
                       dim3(unsigned(cdiv64(row_sets, fp8g::kW4Waves * a.reps)), unsigned(slots)),
                       dim3(fp8g::kW4Waves * fp8g::kWave), lds, s, a);
    return hipGetLastError() == hipSuccess ? FP8G_OK : FP8G_ELAUNCH;
  }
  // k is split over the waves of a workgroup until there is a wave for each of the CUs' places
  int lks = 0;
  while (lks < 3 && (sets << lks) < kFullWaves && (2 << lks) <= blocks) ++lks;
  const int waves = lks == 3 ? 8 : 4;
  a.split_log2 = lks;
  const int lds = waves * fp8g::W4Ring<Z, G, TX, R, U>::kWave;
  hipLaunchKernelGGL((fp8g::w4_kernel<FMT, Z, G, TX, R, U, ROUTED>),
                     dim3(unsigned(cdiv64(a.n, (waves >> lks) * 16 * R)), unsigned(slots)),
                     dim3(waves * fp8g::kWave), lds, s, a);
  return hipGetLastError() == hipSuccess ? FP8G_OK : FP8G_ELAUNCH;
}

template <int FMT, bool Z, int G, bool ROUTED>
int launch_tiles(const W4Args& a, hipStream_t s) {
  constexpr int kSteps = G == 32 ? 1 : 2;  // 128-column steps of a block: four groups or fewer
  // tokens per expert: hardly ever above 1, 4 with 1/8, 1 on average
  if (ROUTED ? a.m <= a.experts / 8 : a.m == 1) return launch_kernel<FMT, Z, G, 1, 1, kSteps, ROUTED>(a, s);
  if (ROUTED ? a.m <= a.experts : a.m <= 4) return launch_kernel<FMT, Z, G, 4, 1, kSteps, ROUTED>(a, s);
  const int64_t sets = cdiv64(a.n, 32) * (ROUTED ? a.experts : cdiv64(a.m, 16));
  if (sets * fp8g::kW4Waves < kFullWaves / 2) return launch_kernel<FMT, Z, G, 16, 1, 1, ROUTED>(a, s);
  return launch_kernel<FMT, Z, G, 16, 2, 1, ROUTED>(a, s);
}

template <int FMT, bool Z>
int launch_group(const W4Args& a, int group, hipStream_t s) {
  if (a.expert_idx)
    return group == 32 ? launch_tiles<FMT, Z, 32, true>(a, s)
           : group == 64 ? launch_tiles<FMT, Z, 64, true>(a, s)
                         : launch_tiles<FMT, Z, 128, true>(a, s);
  return group == 32 ? launch_tiles<FMT, Z, 32, false>(a, s)
         : group == 64 ? launch_tiles<FMT, Z, 64, false>(a, s)
                       : launch_tiles<FMT, Z, 128, false>(a, s);
}

int launch(const W4Args& a, int w_format, int group, hipStream_t s) {
  if (a.k == 0) {  // empty sums
    const int64_t bytes = int64_t(a.m) * a.n * (a.out_f32 ? 4 : 2), blocks = cdiv64(bytes / 4 + 1, 256);
    if (blocks > 0x7fffffff) return FP8G_EUNSUPPORTED;
    hipLaunchKernelGGL(fp8g::w4_zero_kernel, dim3(unsigned(blocks)), dim3(256), 0, s, static_cast<uint32_t*>(a.out),
                       bytes / 4, int(bytes % 4));
    return hipGetLastError() == hipSuccess ? FP8G_OK : FP8G_ELAUNCH;
  }
  if (w_format == FP8G_E2M1) return launch_group<FP8G_E2M1, false>(a, group, s);
  return a.zeros ? launch_group<FP8G_INT4, true>(a, group, s) : launch_group<FP8G_INT4, false>(a, group, s);
}

}  // namespace

extern "C" {

int fp8_w4_matvec(const uint16_t* x, int64_t x_ld, const uint8_t* w, int w_format, const void* w_scales,
                  int scales_dtype, const uint8_t* w_zeros, int group, void* out, int out_dtype, int m, int n, int k,
                  void* stream) {
  const W4Args a{x, x_ld, w, w_scales, w_zeros, out, scales_dtype == FP8G_BF16, out_dtype == FP8G_F32, m, n, k, nullptr, 1, 1, 0, 0, 0};
  bool empty;
  if (int st = check(a, w_format, scales_dtype, out_dtype, group, &empty)) return st;
  return empty ? FP8G_OK : launch(a, w_format, group, static_cast<hipStream_t>(stream));
}

int fp8_w4_matvec_experts(const uint16_t* x, int64_t x_ld, int x_rows, const int32_t* expert_idx, int num_pairs,
                          const uint8_t* w, int w_format, const void* w_scales, int scales_dtype,
                          const uint8_t* w_zeros, int group, void* out, int out_dtype, int num_experts, int n, int k,
                          void* stream) {
  if (num_pairs < 0 || x_rows < 0 || num_experts < 1) return FP8G_EINVAL;
  if (num_pairs > 0 && (x_rows == 0 || num_pairs % x_rows != 0)) return FP8G_EINVAL;
  const W4Args a{x, x_ld, w, w_scales, w_zeros, out, scales_dtype == FP8G_BF16, out_dtype == FP8G_F32, num_pairs, n, k, expert_idx, num_experts,
                 num_pairs > 0 ? num_pairs / x_rows : 1, 0, 0, 0};
  bool empty;
  if (int st = check(a, w_format, scales_dtype, out_dtype, group, &empty)) return st;
  if (empty) return FP8G_OK;
  if (!expert_idx || !aligned(expert_idx, 4)) return FP8G_EINVAL;
  return launch(a, w_format, group, static_cast<hipStream_t>(stream));
}

}  // extern "C"
