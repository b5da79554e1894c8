// Arguments and launches of the 4-bit product kernels, one object file per
// kind of matrix (w4_launch.hip is compiled once for each), so that the
// library's instantiations build in parallel.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace fp8g {

struct W4Args {
  const uint16_t* x;
  int64_t x_ld;
  const uint8_t* w;
  const void* scales;
  const uint8_t* zeros;
  void* out;
  int scales_bf16, out_f32;
  int m, n, k;                // m: tokens, or pairs in the routed form
  const int32_t* expert_idx;  // routed form, else NULL
  int experts, x_div;         // experts; pairs per row of x
  // set at the launch
  int split_log2;             // 2^this waves of a workgroup share rows and split k
  int reps;                   // streaming kernel: row sets a wave takes
};

namespace host {

// KIND 0: INT4, 1: INT4 with zero points, 2: E2M1.  k > 0, m > 0, n > 0, arguments checked.
template <int KIND>
int launch_w4(const W4Args& a, int group, hipStream_t s);
template <>
int launch_w4<0>(const W4Args& a, int group, hipStream_t s);
template <>
int launch_w4<1>(const W4Args& a, int group, hipStream_t s);
template <>
int launch_w4<2>(const W4Args& a, int group, hipStream_t s);

}  // namespace host
}  // namespace fp8g
