// Host side of the 4-bit matrix-vector products (declared in fp8gemm.h):
// validation and launches.  Nothing here allocates, synchronises or reads
// device memory.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fp8gemm.h"
#include "w4_launch.hpp"

namespace {

using fp8g::W4Args;

constexpr int kMaxColumns = 1 << 20;  // byte offsets within a workgroup's 128 rows fit 32 bits
constexpr int kMaxRows = 1 << 30;

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check(const W4Args& a, int w_format, int scales_dtype, int out_dtype, int group, bool* empty) {
  *empty = false;
  if (w_format != FP8G_INT4 && w_format != FP8G_E2M1) return FP8G_EINVAL;
  if (scales_dtype != FP8G_F32 && scales_dtype != FP8G_BF16) return FP8G_EINVAL;
  if (out_dtype != FP8G_F32 && out_dtype != FP8G_BF16) return FP8G_EINVAL;
  if (a.m < 0 || a.n < 0 || a.k < 0 || a.x_ld < a.k) return FP8G_EINVAL;
  if (w_format == FP8G_E2M1 && a.zeros) return FP8G_EINVAL;
  if ((group != 32 && group != 64 && group != 128) || a.k % group != 0 || a.k > kMaxColumns || a.n > kMaxRows ||
      a.x_ld % 8 != 0)
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

// out[m][n] = 0 (an empty reduction): `words` dwords and, if `tail`, a BF16 value after them.
__global__ void __launch_bounds__(256) w4_zero_kernel(uint32_t* __restrict__ out, int64_t words, int tail) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < words) out[i] = 0;
  if (i == words && tail) *reinterpret_cast<uint16_t*>(out + words) = 0;
}

int launch(const W4Args& a, int w_format, int group, hipStream_t s) {
  if (a.k == 0) {  // empty sums
    const int64_t bytes = int64_t(a.m) * a.n * (a.out_f32 ? 4 : 2), blocks = bytes / 1024 + 1;
    if (blocks > 0x7fffffff) return FP8G_EUNSUPPORTED;
    hipLaunchKernelGGL(w4_zero_kernel, dim3(unsigned(blocks)), dim3(256), 0, s, static_cast<uint32_t*>(a.out),
                       bytes / 4, int(bytes % 4));
    return hipGetLastError() == hipSuccess ? FP8G_OK : FP8G_ELAUNCH;
  }
  if (w_format == FP8G_E2M1) return fp8g::host::launch_w4<2>(a, group, s);
  return a.zeros ? fp8g::host::launch_w4<1>(a, group, s) : fp8g::host::launch_w4<0>(a, group, s);
}

}  // namespace

extern "C" {

int fp8_w4_matvec(const uint16_t* x, int64_t x_ld, const uint8_t* w, int w_format, const void* w_scales,
                  int scales_dtype, const uint8_t* w_zeros, int group, void* out, int out_dtype, int m, int n, int k,
                  void* stream) {
  const W4Args a{x, x_ld, w, w_scales, w_zeros, out, scales_dtype == FP8G_BF16, out_dtype == FP8G_F32, m, n, k,
                 nullptr, 1, 1, 0, 0};
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
  const W4Args a{x, x_ld, w, w_scales, w_zeros, out, scales_dtype == FP8G_BF16, out_dtype == FP8G_F32, num_pairs, n, k,
                 expert_idx, num_experts, num_pairs > 0 ? num_pairs / x_rows : 1, 0, 0};
  bool empty;
  if (int st = check(a, w_format, scales_dtype, out_dtype, group, &empty)) return st;
  if (empty) return FP8G_OK;
  if (!expert_idx || !aligned(expert_idx, 4)) return FP8G_EINVAL;
  return launch(a, w_format, group, static_cast<hipStream_t>(stream));
}

}  // extern "C"
