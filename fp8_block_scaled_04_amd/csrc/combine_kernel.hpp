// Weighted sum of the experts' output rows of every token, for gfx950, and
// its gradients.
//
//   out[t]      = bf16( sum over j with 0 <= d_tj < rows of w_tj * y[d_tj] )
//   grad_y[d]   = bf16( w_tj * grad_out[t] )            for d = d_tj
//   grad_w[t,j] = < grad_out[t], y[d_tj] >              (0 for a dropped pair)
// with d_tj = dst_row[t][j], or t * topk + j without one, and w = 1 without
// weights.  Sums and products are FP32, in a fixed order (no atomics), with
// one rounding to BF16 at the end.
//
// Bound by memory: every row is read once and written once, 16 bytes a lane.
// 4096 tokens x 8 rows of 7168: 108 us (4.9 TB/s, the rate of a large copy);
// the gradients of 4001 x 4 x 4096: 60.6 us (4.9 TB/s).
#pragma once

#include "device_common.hpp"

namespace fp8g {

__device__ __forceinline__ void unpack8(const v4i& a, float v[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __int_as_float(a[i] << 16);
    v[2 * i + 1] = __int_as_float(a[i] & 0xffff0000);
  }
}
__device__ __forceinline__ v4i pack8(const float v[8]) {
  v4i a;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = int(pack_bf16x2(v[2 * i], v[2 * i + 1]));
  return a;
}

__device__ __forceinline__ int pair_row(const int32_t* dst, int64_t pair, int rows) {
  const int64_t d = dst ? int64_t(dst[pair]) : pair;
  return d >= 0 && d < rows ? int(d) : -1;
}

// Grid: tokens from `first` on x column blocks of 2048; a thread holds 8 columns.
__global__ void __launch_bounds__(256) moe_combine_kernel(const uint16_t* __restrict__ y, int rows, int n,
                                                          const int32_t* __restrict__ dst,
                                                          const float* __restrict__ weights, int topk,
                                                          uint16_t* __restrict__ out, int64_t first) {
  const int64_t t = first + blockIdx.x;
  const int c = (blockIdx.y * 256 + threadIdx.x) * 8;
  if (c >= n) return;
  float acc[8] = {};
  for (int j = 0; j < topk; ++j) {
    const int d = pair_row(dst, t * topk + j, rows);
    if (d < 0) continue;
    const float w = weights ? weights[t * topk + j] : 1.f;
    float v[8];
    unpack8(*reinterpret_cast<const v4i*>(y + int64_t(d) * n + c), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[i], acc[i]);
  }
  *reinterpret_cast<v4i*>(out + t * n + c) = pack8(acc);
}

// PAIRS = false: a workgroup per token from `first` on, which takes its pairs one after the
// other (its row of grad_out then comes from the cache after the first).
// PAIRS = true: a workgroup per pair of all tokens.  A thread holds up to kBwdChunks pieces
// of 8 columns at a time, all loaded before any is used.
constexpr int kBwdChunks = 4;
template <bool PAIRS>
__global__ void __launch_bounds__(256) moe_combine_backward_kernel(const uint16_t* __restrict__ grad_out,
                                                                   const uint16_t* __restrict__ y, int rows, int n,
                                                                   const int32_t* __restrict__ dst,
                                                                   const float* __restrict__ weights, int topk,
                                                                   uint16_t* __restrict__ grad_y,
                                                                   float* __restrict__ grad_w, int64_t first) {
  __shared__ float part[4];
  const int64_t t = PAIRS ? int64_t(blockIdx.x) / topk : first + blockIdx.x;
  const int j0 = PAIRS ? int(blockIdx.x - t * topk) : 0, j1 = PAIRS ? j0 + 1 : topk;
  for (int j = j0; j < j1; ++j) {
    const int d = pair_row(dst, t * topk + j, rows);
    const float w = weights ? weights[t * topk + j] : 1.f;
    const uint16_t* go = grad_out + t * n;
    float dot = 0.f;
    if (d >= 0)
      for (int c0 = threadIdx.x * 8; c0 < n; c0 += 2048 * kBwdChunks) {
        v4i gv[kBwdChunks], yv[kBwdChunks];
#pragma unroll
        for (int u = 0; u < kBwdChunks; ++u) {
          const int c = min(c0 + u * 2048, n - 8);
          gv[u] = *reinterpret_cast<const v4i*>(go + c);
          if (grad_w) yv[u] = *reinterpret_cast<const v4i*>(y + int64_t(d) * n + c);
        }
#pragma unroll
        for (int u = 0; u < kBwdChunks; ++u) {
          const int c = c0 + u * 2048;
          if (c >= n) break;
          float g[8], v[8], o[8];
          unpack8(gv[u], g);
          if (grad_w) {
            unpack8(yv[u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = fmaf(g[i], v[i], dot);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = w * g[i];
          *reinterpret_cast<v4i*>(grad_y + int64_t(d) * n + c) = pack8(o);
        }
      }
    if (grad_w) {
#pragma unroll
      for (int s = 32; s; s >>= 1) dot += __shfl_xor(dot, s, kWave);
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
      __syncthreads();
      if (threadIdx.x == 0) grad_w[t * topk + j] = (part[0] + part[1]) + (part[2] + part[3]);
      __syncthreads();
    }
  }
}

}  // namespace fp8g
