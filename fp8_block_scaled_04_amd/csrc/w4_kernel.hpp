// Products of a few rows with a 4-bit matrix, for gfx950.
//
//   out[i][r] = sum over c of x[i][c] * v(r, c),   x BF16, FP32 sums,
//   v(r, c) = (code(r, c) - zero(r, c / g)) * scale(r, c / g)   (INT4; zero 8
//             where there are no zero points)
//   v(r, c) = e2m1(code(r, c)) * scale(r, c / g)                (E2M1)
// Codes are packed two to a byte along the row, the even column in the low
// four bits.  Routed form: pair p = t * topk + j multiplies its row of x with
// the matrix of expert expert_idx[p]; a row of zeros where that is none.
#pragma once

#include "device_common.hpp"

namespace fp8g {

constexpr int kW4Int4 = 0, kW4E2M1 = 1;

struct W4Args {
  const uint16_t* x;
  int64_t x_ld;
  const uint8_t* w;
  const void* scales;
  const uint8_t* zeros;
  void* out;
  int m, n, k, group;
  const int32_t* expert_idx;  // routed form
  int experts, x_div;         // experts; pairs per row of x
};

__device__ __forceinline__ float scale_at(const float* s, int64_t i) { return s[i]; }
__device__ __forceinline__ float scale_at(const uint16_t* s, int64_t i) {
  return __uint_as_float(uint32_t(s[i]) << 16);
}

template <int FMT>
__device__ __forceinline__ float w4_value(uint32_t code) {
  if constexpr (FMT == kW4Int4) return float(int(code));
  const uint32_t mag = code & 7, e = mag >> 1, m = mag & 1;
  const float v = e ? (1.f + 0.5f * float(m)) * float(1u << e) * 0.5f : 0.5f * float(m);
  return code & 8 ? -v : v;
}

// One wave per output element, lanes along the row: 8 codes (a dword) each.
template <int FMT, typename S, typename O>
__global__ void __launch_bounds__(256) w4_kernel(W4Args a) {
  const int lane = threadIdx.x & (kWave - 1);
  const unsigned blocks = (unsigned(a.n) + 3) / 4;
  const int r = int(blockIdx.x % blocks) * 4 + int(threadIdx.x >> 6);
  const int64_t i = blockIdx.x / blocks;
  if (r >= a.n) return;
  int64_t e = 0, xi = i;
  if (a.expert_idx) {
    e = a.expert_idx[i];
    xi = i / a.x_div;
  }
  float acc = 0.f;
  if (e >= 0 && (!a.expert_idx || e < a.experts)) {
    const int groups = a.k / a.group;
    const int64_t row = e * a.n + r;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(a.w + row * (a.k / 2));
    for (int c = lane * 8; c < a.k; c += kWave * 8) {
      const uint32_t q = w[c / 8];
      const int64_t g = row * groups + c / a.group;
      const float s = scale_at(static_cast<const S*>(a.scales), g);
      const float z = FMT == kW4Int4 ? (a.zeros ? float(a.zeros[g]) : 8.f) : 0.f;
      float part = 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        part = fmaf(w4_value<FMT>((q >> (4 * u)) & 15) - z, __uint_as_float(uint32_t(a.x[xi * a.x_ld + c + u]) << 16),
                    part);
      acc = fmaf(s, part, acc);
    }
  }
#pragma unroll
  for (int s = 32; s; s >>= 1) acc += __shfl_xor(acc, s, kWave);
  if (lane == 0) {
    if constexpr (sizeof(O) == 4) static_cast<float*>(a.out)[i * a.n + r] = acc;
    else static_cast<uint16_t*>(a.out)[i * a.n + r] = uint16_t(pack_bf16x2(acc, 0.f));
  }
}

}  // namespace fp8g
