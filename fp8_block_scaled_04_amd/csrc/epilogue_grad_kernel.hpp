// Gradients of what follows the dense product:
//   grad_z = bf16( grad_out act'(z) ),   grad_bias[n] = sum over rows of grad_out act'(z)
// z as the forward pass left it in BF16; sums FP32, of the values before their
// rounding.
#pragma once

#include "activation.hpp"
#include "epilogue_kernel.hpp"  // packing of 8 BF16 values

namespace fp8g {

// Grid: x column blocks of 256 (a thread holds 8 columns of every 8th row), y
// slices of `rows_per_slice` rows.  Sums go over a thread's rows, then its
// workgroup's eight threads of a column, then (column_sums_kernel) the slices,
// each in order.  partial: [slices][n], or grad_bias itself where there is one
// slice; NULL: no sums.  Bound by memory, with eight rows of a thread's columns on
// their way (8192 x 4096 with its sums 39.8 us, 5.1 TB/s; with four rows 41.4).
constexpr int kEpilogueColumns = 256;
__global__ void __launch_bounds__(256) epilogue_backward_kernel(const uint16_t* grad_out, const uint16_t* preact,
                                                                int activation, int m, int n, int rows_per_slice,
                                                                uint16_t* grad_preact, float* partial) {
  constexpr int AHEAD = 8;
  __shared__ float sums[8][kEpilogueColumns + 4];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col = blockIdx.x * kEpilogueColumns + 8 * tx;
  const int first = blockIdx.y * rows_per_slice, last = min(m, first + rows_per_slice);
  float acc[8] = {};
  if (col < n)
    by_activation(activation, [&](auto tag) __attribute__((always_inline)) {
    constexpr int ACT = decltype(tag)::value;
    for (int r = first + ty; r < last; r += 8 * AHEAD) {
      uint4 g[AHEAD], z[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {  // rows past the end: the last one again
        const int64_t at = int64_t(min(r + 8 * u, last - 1)) * n + col;
        g[u] = *reinterpret_cast<const uint4*>(grad_out + at);
        z[u] = *reinterpret_cast<const uint4*>(preact + at);
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        if (r + 8 * u >= last) break;
        float a[8], b[8];
        unpack_bf16x8(g[u], a);
        unpack_bf16x8(z[u], b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] *= activate_grad<ACT>(b[i]);
          acc[i] += a[i];
        }
        *reinterpret_cast<uint4*>(grad_preact + int64_t(r + 8 * u) * n + col) = pack_bf16x8(a);
      }
    }
    });
  if (!partial) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[ty][8 * tx + i] = acc[i];
  __syncthreads();
  const int c = blockIdx.x * kEpilogueColumns + threadIdx.x;
  if (c >= n) return;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += sums[i][threadIdx.x];
  partial[int64_t(blockIdx.y) * n + c] = v;
}

// out[y][c] = sum over s < slices of partial[s][y][c] (rows of n, `sets` = gridDim.y of them side by side): 16 runs of
// slices per column, each in order, then the runs.  Grid: x column blocks of 64, y sets.
constexpr int kSumRuns = 16;
__global__ void __launch_bounds__(64 * kSumRuns) column_sums_kernel(const float* partial, int slices, int n,
                                                                    float* out0, float* out1, float* out2) {
  constexpr int AHEAD = 16;
  __shared__ float sums[kSumRuns][64];
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6, c = blockIdx.x * 64 + tx, sets = gridDim.y;
  const int per = (slices + kSumRuns - 1) / kSumRuns, s0 = ty * per, s1 = min(slices, s0 + per);
  float* out = blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2;
  if (!out) return;
  float v = 0.f;
  if (c < n)
    for (int s = s0; s < s1; s += AHEAD) {
      float t[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) t[u] = partial[(int64_t(min(s + u, s1 - 1)) * sets + blockIdx.y) * n + c];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) v += s + u < s1 ? t[u] : 0.f;
    }
  sums[ty][tx] = v;
  __syncthreads();
  if (ty != 0 || c >= n) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kSumRuns; ++i) v += sums[i][tx];
  out[c] = v;
}

}  // namespace fp8g
