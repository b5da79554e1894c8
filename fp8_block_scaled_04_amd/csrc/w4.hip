// Host side of the 4-bit matrix-vector products (declared in fp8gemm.h):
// validation and launches.  Nothing here allocates, synchronises or reads
// device memory.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fp8gemm.h"
#include "w4_kernel.hpp"

namespace {

using fp8g::W4Args;

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check(const W4Args& a, int w_format, int scales_dtype, int out_dtype, bool* empty) {
  *empty = false;
  if (w_format != FP8G_INT4 && w_format != FP8G_E2M1) return FP8G_EINVAL;
  if (scales_dtype != FP8G_F32 && scales_dtype != FP8G_BF16) return FP8G_EINVAL;
  if (out_dtype != FP8G_F32 && out_dtype != FP8G_BF16) return FP8G_EINVAL;
  if (a.m < 0 || a.n < 0 || a.k < 0 || a.x_ld < a.k) return FP8G_EINVAL;
  if (w_format == FP8G_E2M1 && a.zeros) return FP8G_EINVAL;
  if ((a.group != 32 && a.group != 64 && a.group != 128) || a.k % a.group != 0 || a.x_ld % 8 != 0)
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

template <int FMT, typename S, typename O>
int launch(const W4Args& a, hipStream_t s) {
  const int64_t grid = (int64_t(a.n) + 3) / 4 * a.m;
  if (grid > 0x7fffffff) return FP8G_EUNSUPPORTED;
  hipLaunchKernelGGL((fp8g::w4_kernel<FMT, S, O>), dim3(unsigned(grid)), dim3(256), 0, s, a);
  return hipGetLastError() == hipSuccess ? FP8G_OK : FP8G_ELAUNCH;
}

template <int FMT, typename S>
int launch(const W4Args& a, int out_dtype, hipStream_t s) {
  return out_dtype == FP8G_F32 ? launch<FMT, S, float>(a, s) : launch<FMT, S, uint16_t>(a, s);
}

int launch(const W4Args& a, int w_format, int scales_dtype, int out_dtype, hipStream_t s) {
  if (w_format == FP8G_INT4)
    return scales_dtype == FP8G_F32 ? launch<FP8G_INT4, float>(a, out_dtype, s)
                                    : launch<FP8G_INT4, uint16_t>(a, out_dtype, s);
  return scales_dtype == FP8G_F32 ? launch<FP8G_E2M1, float>(a, out_dtype, s)
                                  : launch<FP8G_E2M1, uint16_t>(a, out_dtype, s);
}

}  // namespace

extern "C" {

int fp8_w4_matvec(const uint16_t* x, int64_t x_ld, const uint8_t* w, int w_format, const void* w_scales,
                  int scales_dtype, const uint8_t* w_zeros, int group, void* out, int out_dtype, int m, int n, int k,
                  void* stream) {
  const W4Args a{x, x_ld, w, w_scales, w_zeros, out, m, n, k, group, nullptr, 1, 1};
  bool empty;
  if (int st = check(a, w_format, scales_dtype, out_dtype, &empty)) return st;
  return empty ? FP8G_OK : launch(a, w_format, scales_dtype, out_dtype, static_cast<hipStream_t>(stream));
}

int fp8_w4_matvec_experts(const uint16_t* x, int64_t x_ld, int x_rows, const int32_t* expert_idx, int num_pairs,
                          const uint8_t* w, int w_format, const void* w_scales, int scales_dtype,
                          const uint8_t* w_zeros, int group, void* out, int out_dtype, int num_experts, int n, int k,
                          void* stream) {
  if (num_pairs < 0 || x_rows < 0 || num_experts < 1) return FP8G_EINVAL;
  if (num_pairs > 0 && (x_rows == 0 || num_pairs % x_rows != 0)) return FP8G_EINVAL;
  const W4Args a{x, x_ld, w, w_scales, w_zeros, out, num_pairs, n, k, group, expert_idx, num_experts,
                 num_pairs > 0 ? num_pairs / x_rows : 1};
  bool empty;
  if (int st = check(a, w_format, scales_dtype, out_dtype, &empty)) return st;
  if (empty) return FP8G_OK;
  if (!expert_idx || !aligned(expert_idx, 4)) return FP8G_EINVAL;
  return launch(a, w_format, scales_dtype, out_dtype, static_cast<hipStream_t>(stream));
}

}  // extern "C"
