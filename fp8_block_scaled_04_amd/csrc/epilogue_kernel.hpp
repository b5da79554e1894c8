// What follows the dense product, applied to its FP32 sums before their one
// rounding:
//
//   z = acc + bias[n]             (z itself as BF16 too, where it is asked for)
//   out = bf16( act(z) + residual )
//
// The tile goes through LDS as FP32, in row order, so that one piece
// of code does everything: a thread keeps 8 columns (and their bias) for all of
// its rows, reads the residual and writes the output in whole 16-byte pieces
// of rows, and the activation is chosen once per piece in a loop instead of in
// an unrolled copy for every accumulator.  The 256 x 256 tile, whose FP32 form
// is twice the ring, goes in two halves.
//
// What it adds to the product: the tile's way through LDS and the activation,
// which no matrix instruction of the workgroup overlaps, and the residual's and
// the pre-activations' bytes (4096 x 4096 x 7168, GELU_TANH and
// pre-activations 115 us, the product alone 100; 4001 x 7168 x 16384 with a
// residual 430 and 415; 64 x 2112 x 7168 split over k, SiLU and a residual 10.4
// and 9.6).  The residual of the next rows is read while these are written.
#pragma once

#include "activation.hpp"
#include "gemm_kernel.hpp"

namespace fp8g {

__device__ __forceinline__ void unpack_bf16x8(const uint4& a, float v[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack_bf16x8(const float v[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

template <>
struct EpilogueOf<kDenseEpilogue> {
  // What stands for a bias or residual that is not there: -0, to which any sum adds without a change (0 would make of a
  // sum of -0 a 0).
  static constexpr float kNone = -0.f;
  static constexpr uint32_t kNone2 = 0x80008000u;  // two of BF16

  // N (4 or 8) consecutive values of the bias, from column `col` on.
  template <int N>
  static __device__ __forceinline__ void load_bias(const GemmParams& p, int col, float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = kNone;
    if (!p.bias) return;
    if (p.bias_bf16) {
      const uint2* q = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.bias) + col);
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint2 w = q[i / 4];
        b[i] = __uint_as_float(w.x << 16), b[i + 1] = __uint_as_float(w.x & 0xffff0000u);
        b[i + 2] = __uint_as_float(w.y << 16), b[i + 3] = __uint_as_float(w.y & 0xffff0000u);
      }
    } else {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + col);
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 w = q[i / 4];
        b[i] = w.x, b[i + 1] = w.y, b[i + 2] = w.z, b[i + 3] = w.w;
      }
    }
  }

  // Four sums of the split-K fix-up, at out[at] in column `col`.  What they meet is loaded with the partial sums, which
  // are waited for all together.
  struct Four {
    float b[4];
    uint2 r;
    __device__ __forceinline__ void load(const GemmParams& p, int64_t at, int col) {
      load_bias(p, col, b);
      r = make_uint2(kNone2, kNone2);
      if (p.residual) r = *reinterpret_cast<const uint2*>(p.residual + at);
    }
    __device__ __forceinline__ void store(const GemmParams& p, const v4f& sum, int64_t at) const {
      float z[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = sum[i] + b[i];
      if (p.preact)
        *reinterpret_cast<uint2*>(p.preact + at) = make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
      by_activation(p.activation, [&](auto tag) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = i < 2 ? r.x : r.y;
          y[i] = activate<decltype(tag)::value>(z[i]) + __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
        }
      });
      *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    }
  };

  // A whole tile from the accumulators (write_tile's arguments; SMEM bytes of LDS, free once the K loop is done).
  template <int BM, int BN, int TM, int TN, int SMEM>
  static __device__ __forceinline__ void store_tile(const GemmParams& p, const v4f (&acc)[TN][TM], uint8_t* smem,
                                                    bool holder, int wrow_m, int wrow_n, int m0, int n0, int rows,
                                                    int shape_n) {
    constexpr int LDT = BN + 4;  // padded row stride (floats) of the staged tile
    constexpr int PASSES = BM * LDT * 4 <= SMEM ? 1 : 2, PR = BM / PASSES;
    static_assert(PR * LDT * 4 <= SMEM && PR % (16 * TM) == 0, "a pass is whole waves' rows and fits");
    constexpr int CHUNKS = BN / 8, AHEAD = 4;
    const int lane = threadIdx.x & (kWave - 1);
    float* stage = reinterpret_cast<float*>(smem);
    const int c8 = 8 * (threadIdx.x % CHUNKS), col = n0 + c8;  // n % 8 == 0: a piece is all in or all out
    const int r0 = threadIdx.x / CHUNKS, step = blockDim.x / CHUNKS;
    const bool in = col < shape_n;
    float b[8] = {};
    if (in) load_bias(p, col, b);
    for (int pass = 0; pass < PASSES; ++pass) {
      const int first = pass * PR, last = min(PR, rows - m0 - first);  // rows of this pass
      const int64_t at0 = int64_t(m0 + first) * shape_n + col;
      const bool work = in && r0 < last;
      uint4 next[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) next[u] = make_uint4(kNone2, kNone2, kNone2, kNone2);
      auto load = [&](int r) {  // of the residual; rows past the end: the last one again
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          next[u] = *reinterpret_cast<const uint4*>(p.residual + at0 + int64_t(min(r + u * step, last - 1)) * shape_n);
      };
      if (work && p.residual) load(r0);
      __syncthreads();  // the ring, or the rows staged before, are read
      if (holder && wrow_m / PR == pass) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int j = 0; j < TM; ++j)
            *reinterpret_cast<v4f*>(stage + (wrow_m - first + 16 * j + (lane & 15)) * LDT + wrow_n + 16 * i +
                                    4 * (lane >> 4)) = acc[i][j];
      }
      __syncthreads();
      if (!work) continue;
      by_activation(p.activation, [&](auto tag) __attribute__((always_inline)) {
        constexpr int ACT = decltype(tag)::value;
        for (int r = r0; r < last; r += AHEAD * step) {
          uint4 res[AHEAD];
#pragma unroll
          for (int u = 0; u < AHEAD; ++u) res[u] = next[u];
          if (p.residual && r + AHEAD * step < last) load(r + AHEAD * step);
#pragma unroll
          for (int u = 0; u < AHEAD; ++u) {
            const int row = r + u * step;
            if (row >= last) break;
            const v4f lo = *reinterpret_cast<const v4f*>(stage + row * LDT + c8);
            const v4f hi = *reinterpret_cast<const v4f*>(stage + row * LDT + c8 + 4);
            float z[8], y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = (i < 4 ? lo[i] : hi[i - 4]) + b[i];
            const int64_t at = at0 + int64_t(row) * shape_n;
            if (p.preact) *reinterpret_cast<uint4*>(p.preact + at) = pack_bf16x8(z);
            unpack_bf16x8(res[u], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] += activate<ACT>(z[i]);
            *reinterpret_cast<uint4*>(p.out + at) = pack_bf16x8(y);
          }
        }
      });
    }
  }
};

template <>
struct EpilogueFour<kDenseEpilogue> { using type = EpilogueOf<kDenseEpilogue>::Four; };

}  // namespace fp8g
