// Products of a few rows with a 4-bit matrix, for gfx950.
//
//   out[i][r] = sum over c of x[i][c] * v(r, c),   x BF16, FP32 sums,
//   v(r, c) = (code(r, c) - zero(r, c / g)) * scale(r, c / g)   (INT4; zero 8
//             where there are no zero points)
//   v(r, c) = e2m1(code(r, c)) * scale(r, c / g)                (E2M1)
// Codes are packed two to a byte along the row, the even column in the low
// four bits.  Routed form: pair p multiplies its row of x with the matrix of
// expert expert_idx[p]; a row of zeros where that is none.
//
// Each group's sum is formed by BF16 matrix instructions (16 tokens x 16
// matrix rows x 32 columns): codes 0..15 and E2M1 values are exact in BF16,
// and the group's scale and zero point are applied to the FP32 sum,
//     sum (code - zero) * scale * x = scale * (sum code * x - zero * sum x),
// with sum x from the same instruction against ones.  The difference rounds as
// its larger sum does: where a group's activations share a sign, as terms of
// code + zero instead of code - zero (4 x 512 x 7168 against 64 bits: up to 6e-7
// of the outputs' norm, 1e-7 for random signs; an FP32 product of the decoded
// matrix 5e-7 to 1e-6).
//
// What bounds it: the codes are read once, 0.5 byte a weight, and a CU has to
// decode what it reads.  A lane's 16 bytes take 36 (INT4) or 16 (E2M1) vector
// instructions of 4 cycles to decode and more again around that, so the
// codes' way from memory to LDS runs by direct copies (no registers, several
// blocks ahead) and the waves carry as little else as they can.  Measured on
// gfx950: a direct copy of 1 KB takes the CU's memory pipe 17 cycles when
// four consecutive lanes read 64 bytes, 64 cycles when every lane reads a row
// of its own, as the operand layout has it; so rows are copied by four or
// eight lanes and turned in LDS.
// Time per call of many issued back to back, three sets of inputs in turn (most
// of which stay in the last-level cache), and with more sets than that holds:
//   one token       4096 x 7168 INT4, groups of 128       5.8 us (2.6 TB/s)    6.4
//   5 tokens        2111 x 7168 E2M1, groups of 32        5.6 us (1.5 TB/s)    7.1
//   16 tokens       7168 x 16384 INT4 with zero points   19.0 us (3.4 TB/s)   23.3
//   8 experts       4096 x 2048, one token               10.1 us (3.6 TB/s)   11.0
//   128 experts     7168 x 2048, 64 tokens, 8 each        204 us (4.9 TB/s)
// An empty launch takes 1.7.
#pragma once

#include "device_common.hpp"
#include "w4_launch.hpp"

namespace fp8g {

constexpr int kW4Int4 = 0, kW4E2M1 = 1;
constexpr int kW4Waves = 8;     // per workgroup, at most (4 where k is split less: two workgroups fit a CU)
// Rings of a workgroup of 8 waves, at most: with a tile's pairs each, two workgroups of 4 fit a CU's 160 KB.
constexpr int kW4LdsBytes = 156 * 1024;
constexpr int kW4MaxExperts = 4096;  // their counts take the rings' place in LDS
constexpr int kW4MaxPairs = 65536;   // every workgroup looks through them
// Routed form, tiles of up to 4 pairs: a workgroup row per pair; of 16: per expert.
constexpr bool w4_by_pair(int tx) { return tx < 16; }

typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v4f mfma16x16x32(const v4i& a, const v4i& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf16, a), __builtin_bit_cast(v8bf16, b), c, 0, 0,
                                                 0);
}

// Eight codes -> eight BF16 values, in column order.  INT4: the byte 0000qqqq
// read as E4M3 is q * 2^-9 for every q (0..7 are that format's subnormals,
// 8..15 its first binade), so the conversion with scale 2^9 gives q exactly.
template <int FMT>
__device__ __forceinline__ v4i w4_decode(unsigned q) {
  v4i f;
  if constexpr (FMT == kW4Int4) {
    const unsigned even = q & 0x0f0f0f0fu, odd = (q >> 4) & 0x0f0f0f0fu;
    const unsigned lo = __builtin_amdgcn_perm(odd, even, 0x05010400u);
    const unsigned hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
    f[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false));
    f[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true));
    f[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false));
    f[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true));
  } else {
    f[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 0));
    f[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 1));
    f[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 2));
    f[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 3));
  }
  return f;
}

// Workgroup barrier after this wave's LDS accesses; copies to LDS stay in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Waits until at most N of the wave's copies are in flight.
template <int N>
__device__ __forceinline__ void copies_left() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Copies to LDS as in copy16_to_lds, of one scale or zero point per lane into
// lane i's dword, and of 16 bytes per lane from addresses of its own.
__device__ __forceinline__ void copy4_scale_to_lds(const void* base, unsigned index, uint32_t lds, bool two_bytes) {
  if (two_bytes)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, %2"
                 ::"s"(uniform(int(lds))), "v"(index * 2), "s"(uniform_ptr(base)) : "memory");
  else
    copy4_to_lds(base, index * 4, lds);
}
__device__ __forceinline__ void copy1_zero_to_lds(const uint8_t* base, unsigned byte, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, %2"
               ::"s"(uniform(int(lds))), "v"(byte), "s"(uniform_ptr(base)) : "memory");
}
__device__ __forceinline__ void copy16_scattered_to_lds(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               ::"s"(uniform(int(lds))), "v"(src) : "memory");
}

__device__ const v4i kW4Zeros = {0, 0, 0, 0};

// Scales (or zero points) of 16 R rows, F = U * 128 / G groups a block.  A
// copy brings four groups of 16 rows, a dword per lane, four lanes per row
// (a lane per row, as one group would have it, takes the memory pipe four
// times as long): parts of a block where it has four groups or more, else a
// period of 4 / F blocks at once.
template <int R, int F>
struct W4Scales {
  static constexpr int kParts = F >= 4 ? F / 4 : 1, kPeriod = F >= 4 ? 1 : 4 / F;
  static constexpr int kCopies = kParts * R, kBytes = kCopies * 256;  // of a period
  unsigned v[R][F];
  // What a lane (column `col` of the matrix operand) needs for a block, the i-th of its period.
  __device__ __forceinline__ void read(const char* at, int col, int i) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (F >= 4) {
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          const v4i t = *reinterpret_cast<const v4i*>(at + (h * R + r) * 256 + col * 16);
#pragma unroll
          for (int f = 0; f < 4; ++f) v[r][4 * h + f] = unsigned(t[f]);
        }
      } else if constexpr (F == 2) {
        const v2u t = *reinterpret_cast<const v2u*>(at + r * 256 + col * 16 + i * 8);
        v[r][0] = t.x;
        v[r][1] = t.y;
      } else {
        v[r][0] = *reinterpret_cast<const unsigned*>(at + r * 256 + col * 16 + i * 4);
      }
    }
  }
};

// Where a row's 16-byte pieces lie in a block's codes [row][4 U pieces]: piece
// p at p ^ w4_swap(row), so that the 16 rows of an operand read meet no bank
// twice while the copies read 64 U bytes of a row in one run.
template <int U>
__device__ __forceinline__ constexpr int w4_swap(int row) {
  static_assert(U == 1 || U == 2, "four or eight pieces per row");
  return U == 2 ? (row >> 1) & 7 : (row >> 2) & 3;
}

// The token in a lane's operand row (its `col`).  Up to four tokens stand in
// the rows 0, 4, 8, 12, so that result register 0 is all a lane has to scale;
// eight in the rows 0, 1, 4, 5, ..., so that it is 0 and 1.
template <int TX>
__device__ __forceinline__ int w4_token(int col) {
  return TX == 16 ? col : TX == 8 ? (col >> 2) * 2 + (col & 1) : TX == 4 ? col >> 2 : 0;
}

// A block: U steps of 128 columns by 16 R rows of the matrix and TX tokens,
// as a lane (operand row `col`, columns' `quarter`) holds it.  Groups of 128
// columns take a lane's 16 bytes of codes as four operands (dword j of the
// four quarters is operand j, all of one group); shorter groups read dword
// `quarter` of piece j, so that operand j holds 32 consecutive columns.
template <int FMT, bool Z, int G, int TX, int R, int U>
struct W4Block {
  static constexpr int Q = 128 / G, F = U * Q, JG = 4 / Q;  // groups per step and block; instructions per group
  static constexpr int A = TX == 16 ? 4 : TX == 8 ? 2 : 1;  // result registers in use: tokens A * quarter ..
  using Scales = W4Scales<R, F>;
  v4i q[U][R], x[U][4];
  Scales s, z;

  __device__ __forceinline__ void read_codes(const char* at, int quarter, int col) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = r * 16 + col, swap = w4_swap<U>(row);
        const char* p = at + row * (64 * U);
        if constexpr (G == 128) {
          q[u][r] = *reinterpret_cast<const v4i*>(p + ((4 * u + quarter) ^ swap) * 16);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q[u][r][j] = *reinterpret_cast<const int*>(p + ((4 * u + j) ^ swap) * 16 + quarter * 4);
        }
      }
  }
  // `at`: the block's units of the lane's token, [16 U units of 8 columns], unit i at i ^ token.
  __device__ __forceinline__ void read_x(const char* at, int quarter, int token) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int unit = 16 * u + (G == 128 ? 4 * quarter + j : 4 * j + quarter);
        x[u][j] = *reinterpret_cast<const v4i*>(at + (unit ^ token) * 16);
      }
  }
  // acc[r][i] += the block's products; g0 its first group, of `groups` per row.
  __device__ __forceinline__ void products(float (&acc)[R][A], unsigned g0, unsigned groups, unsigned scale_shift) {
    if (g0 + F > groups) {  // no scale may meet the empty columns' zero sums
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int r = 0; r < R; ++r) s.v[r][f] = g0 + f < groups ? s.v[r][f] : 0;
    }
    const v4i ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
    const v4f zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v4f part[R], sum;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int r = 0; r < R; ++r)
          part[r] = mfma16x16x32(x[u][j], w4_decode<FMT>(unsigned(q[u][r][j])), j % JG ? part[r] : zero);
        if constexpr (FMT == kW4Int4) sum = mfma16x16x32(x[u][j], ones, j % JG ? sum : zero);
        if (j % JG != JG - 1) continue;
        const int f = u * Q + j / JG;  // the group's place in the block
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float scale = __uint_as_float(s.v[r][f] << scale_shift);
          float zero_point = 8.f;
          if constexpr (Z) zero_point = float(z.v[r][f]);
#pragma unroll
          for (int v = 0; v < A; ++v) {
            float p = part[r][v];
            if constexpr (FMT == kW4Int4) p = fmaf(-zero_point, sum[v], p);
            acc[r][v] = fmaf(scale, p, acc[r][v]);
          }
        }
      }
    }
  }
};

__device__ __forceinline__ void w4_store(const W4Args& a, int64_t at, float v) {
  if (a.out_f32) static_cast<float*>(a.out)[at] = v;
  else static_cast<uint16_t*>(a.out)[at] = uint16_t(pack_bf16x2(v, 0.f));
}

// A group's codes are summed before their scale, so the sums of activations of
// 1e34 or more may pass FP32's range where the product does not (for INT4 both
// sums may, and their difference is a NaN).  An infinity or a NaN never leaves
// an FP32 sum again, so such a product shows at the end, and only there: it is
// formed anew from the definition, in FP64, by the whole wave, after all of its
// outputs are stored (the way there then costs one compare an output, and no
// time that could be measured).  The result is the definition's for every
// input, infinities among them.  A token with a NaN, as a row of padding may
// have, has NaN everywhere and is only looked through, once a wave.  16 tokens
// of 7168 x 16384, 18 us: 21 with a NaN in one token, 26 in all; 250 and 700
// with an infinity, where every output is formed anew.
constexpr int kW4Ahead = 4;  // loads of 512 columns in flight
template <int FMT, bool Z, int G>
__device__ __forceinline__ float w4_product(const W4Args& a, int64_t w_row, int64_t x_row) {
  const int lane = threadIdx.x & (kWave - 1);
  const uint8_t* w = a.w + w_row * (a.k >> 1);
  const uint16_t* x = a.x + x_row * a.x_ld;
  double sum = 0.;
  for (int c0 = lane * 8; c0 < a.k; c0 += kWave * 8 * kW4Ahead) {  // 8 columns, of one group
    unsigned q[kW4Ahead];
    v4i xs[kW4Ahead];
    float scale[kW4Ahead], zero[kW4Ahead];
#pragma unroll
    for (int u = 0; u < kW4Ahead; ++u) {
      const int c = min(c0 + u * kWave * 8, a.k - 8);
      const int64_t g = w_row * (a.k / G) + c / G;
      q[u] = *reinterpret_cast<const unsigned*>(w + (c >> 1));
      xs[u] = *reinterpret_cast<const v4i*>(x + c);
      scale[u] = a.scales_bf16 ? __uint_as_float(unsigned(static_cast<const uint16_t*>(a.scales)[g]) << 16)
                               : static_cast<const float*>(a.scales)[g];
      zero[u] = FMT == kW4Int4 ? 8.f : 0.f;
      if constexpr (Z) zero[u] = a.zeros[g];
    }
#pragma unroll
    for (int u = 0; u < kW4Ahead; ++u) {
      if (c0 + u * kWave * 8 >= a.k) break;
      const v4i values = w4_decode<FMT>(q[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int v = values[i / 2], b = xs[u][i / 2];
        const float value = __int_as_float(i % 2 ? v & 0xffff0000 : v << 16) - zero[u];  // exact
        sum = fma(double(__int_as_float(i % 2 ? b & 0xffff0000 : b << 16)), double(value) * double(scale[u]), sum);
      }
    }
  }
#pragma unroll
  for (int s = 32; s; s >>= 1) sum += __shfl_xor(sum, s, kWave);
  return float(sum);
}

// Whether a row of x has a NaN.
__device__ __forceinline__ bool w4_has_nan(const W4Args& a, int64_t x_row) {
  const uint16_t* x = a.x + x_row * a.x_ld;
  bool nan = false;
  for (int c0 = (threadIdx.x & (kWave - 1)) * 8; c0 < a.k; c0 += kWave * 8 * kW4Ahead) {
    v4i xs[kW4Ahead];  // those past the end are the last ones again
#pragma unroll
    for (int u = 0; u < kW4Ahead; ++u) xs[u] = *reinterpret_cast<const v4i*>(x + min(c0 + u * kWave * 8, a.k - 8));
#pragma unroll
    for (int u = 0; u < kW4Ahead; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        nan |= (xs[u][i] & 0x7fff) > 0x7f80 || (unsigned(xs[u][i]) >> 16 & 0x7fff) > 0x7f80;
  }
  return __ballot(nan) != 0;
}

// Tokens of a tile that the wave has looked through, and those of them that have a NaN.
struct W4Nans {
  unsigned looked = 0, found = 0;
};

__device__ __forceinline__ bool w4_finite(float v) { return fabsf(v) < __builtin_inff(); }

// Looks at stored outputs again, one per lane where `wanted`: at out[at], of w_row and x_row, which is token t of the
// tile.  The whole wave has to call it, the wave's stores done.  (They are read past the L1 cache, which may hold what
// was there before.)
template <int FMT, bool Z, int G>
__device__ __forceinline__ void w4_mend(const W4Args& a, bool wanted, int64_t at, int64_t w_row, int64_t x_row, int t,
                                        W4Nans& nans) {
  const int lane = threadIdx.x & (kWave - 1);
  float v = 0.f;
  if (wanted) {
    if (a.out_f32)
      v = __hip_atomic_load(static_cast<const float*>(a.out) + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else
      v = __uint_as_float(unsigned(__hip_atomic_load(static_cast<const uint16_t*>(a.out) + at, __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT)) << 16);
  }
  const bool past = !w4_finite(v);
  for (uint64_t left = __ballot(past); left;) {
    const int src = __ffsll(static_cast<unsigned long long>(left)) - 1;
    const int64_t row = __shfl(x_row, src, kWave);
    const int token = uniform(__shfl(t, src, kWave));
    if (!(nans.looked >> token & 1)) {
      nans.looked |= 1u << token;
      nans.found |= unsigned(w4_has_nan(a, row)) << token;
    }
    uint64_t done = uint64_t(1) << src;
    float u = __builtin_nanf("");
    if (nans.found >> token & 1) done = left & __ballot(t == token);
    else u = w4_product<FMT, Z, G>(a, __shfl(w_row, src, kWave), row);
    v = done >> lane & 1 ? u : v;
    left &= ~done;
  }
  if (past) w4_store(a, at, v);
}

// ---- routed form -------------------------------------------------------------
// A tile is TX pairs of one expert that follow one another, the t-th tile the
// pairs of rank t * TX .. in the order of their indices.  Grid row y takes
//   tiles of up to 4 (no more pairs than experts): the tile that pair y
//   begins, if any;
//   tiles of 16: y < experts the first tile of expert y, y = experts the pairs
//   that are routed nowhere, further rows the experts' further tiles in order
//   (c pairs of an expert make (c - 1) / 16 of them, so (a.m - 1) / 16 at
//   most), which a count of every expert's pairs finds.
// So an expert that many tokens chose has a workgroup for each of its tiles,
// not one that works through them.
template <int TX>
struct W4Tile {
  int pair[TX];
  int counts[2][kW4Waves];  // the waves' pairs in a window, of two windows in turn
};

// Of the pairs p in [from, to) with expert_idx[p] = e, those of rank first ..
// first + TX - 1 are entered in the tile, where the first found has rank
// `rank`; returns the rank after the last.  A window is LOOK consecutive
// pairs a thread.
template <int TX, int LOOK>
__device__ __forceinline__ int w4_find_pairs(const W4Args& a, int e, int from, int to, int rank, int first,
                                             W4Tile<TX>& tile) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid >> 6), waves = blockDim.x >> 6;
  int turn = 0;
  for (int win = from; win < to && rank < first + TX; win += int(blockDim.x) * LOOK, turn ^= 1) {
    const int p0 = win + tid * LOOK;
    int v[LOOK];
    bool found[LOOK];
    int before = 0, all = 0;  // the wave's pairs in lanes below this one, and all of them
#pragma unroll
    for (int i = 0; i < LOOK; ++i) v[i] = a.expert_idx[min(p0 + i, to - 1)];
#pragma unroll
    for (int i = 0; i < LOOK; ++i) {
      found[i] = v[i] == e && p0 + i < to;
      const uint64_t mask = __ballot(found[i]);
      before += __popcll(mask & ((uint64_t(1) << lane) - 1));
      all += __popcll(mask);
    }
    if (lane == 0) tile.counts[turn][wave] = all;
    lds_barrier();
    int mine = rank + before;
    for (int w = 0; w < waves; ++w) {
      const int c = tile.counts[turn][w];
      mine += w < wave ? c : 0;
      rank += c;
    }
    rank = uniform(rank);
#pragma unroll
    for (int i = 0; i < LOOK; ++i) {
      if (found[i] && mine >= first && mine < first + TX) tile.pair[mine - first] = p0 + i;
      mine += found[i];
    }
  }
  lds_barrier();
  return rank;
}

// One pair a thread where that is all of them (512 pairs, 40 experts of 4096 x 512: 30.7 us, 32.1 with four), else
// four.
template <int TX>
__device__ __forceinline__ int w4_find_pairs(const W4Args& a, int e, int from, int to, int rank, int first,
                                             W4Tile<TX>& tile) {
  return to - from <= int(blockDim.x) ? w4_find_pairs<TX, 1>(a, e, from, to, rank, first, tile)
                                      : w4_find_pairs<TX, 4>(a, e, from, to, rank, first, tile);
}

// The j-th of the experts' tiles after their first ones: its expert (-1: there are fewer) and the rank it starts at.
template <int TX>
__device__ __forceinline__ int w4_further_tile(const W4Args& a, int j, int* hist, int& first) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  for (int e = tid; e < a.experts; e += blockDim.x) hist[e] = 0;
  lds_barrier();
  for (int p = tid; p < a.m; p += blockDim.x) {
    const int v = a.expert_idx[p];
    if (v >= 0 && v < a.experts) atomicAdd(&hist[v], 1);
  }
  lds_barrier();
  int expert = -1;
  for (int c = 0; c < a.experts; c += kWave) {
    const int more = c + lane < a.experts ? max(0, (hist[c + lane] + TX - 1) / TX - 1) : 0;
    int upto = more;  // with the lanes before
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const int v = __shfl_up(upto, d, kWave);
      upto += lane >= d ? v : 0;
    }
    const uint64_t past = __ballot(upto > j);
    if (past) {
      const int at = __ffsll(static_cast<unsigned long long>(past)) - 1;
      expert = uniform(c + at);
      first = uniform((j - __shfl(upto - more, at, kWave) + 1) * TX);
      break;
    }
    j -= uniform(__shfl(upto, kWave - 1, kWave));
  }
  lds_barrier();  // hist is free again
  return expert;
}

// This workgroup's tile: its expert (a.experts: pairs routed nowhere, -1:
// nothing to do) and its number of pairs.  `scratch`: a.experts ints of LDS.
template <int TX>
__device__ __forceinline__ int w4_routed_tile(const W4Args& a, W4Tile<TX>& tile, int* scratch, int& count) {
  const int y = blockIdx.y;
  if constexpr (w4_by_pair(TX)) {
    const int e = uniform(a.expert_idx[y]);
    if (e < 0 || e >= a.experts) return a.experts;
    count = 1;
    if constexpr (TX > 1) {
      const int rank = w4_find_pairs<TX>(a, e, 0, y, 0, a.m, tile);
      if (rank % TX) return -1;  // in an earlier pair's tile
      count = min(TX, w4_find_pairs<TX>(a, e, y, a.m, rank, rank, tile) - rank);
    }
    return e;
  } else {
    if (y == a.experts) return y;
    int e = y, first = 0;
    if (y > a.experts) e = w4_further_tile<TX>(a, y - a.experts - 1, scratch, first);
    count = e < 0 ? 0 : min(TX, w4_find_pairs<TX>(a, e, 0, a.m, 0, first, tile) - first);
    return count > 0 ? e : -1;
  }
}

// out = 0 in rows row0 .. row0 + rows - 1 of the matrix for the pairs that are routed nowhere.
template <int TX>
__device__ __forceinline__ void w4_store_zeros(const W4Args& a, int row0, int rows) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid >> 6), threads = blockDim.x;
  if constexpr (w4_by_pair(TX)) {
    for (int o = tid; o < rows; o += threads) w4_store(a, int64_t(blockIdx.y) * a.n + row0 + o, 0.f);
    return;
  }
  for (int win = 0; win < a.m; win += threads) {
    const int v = win + tid < a.m ? a.expert_idx[win + tid] : 0;
    for (uint64_t left = __ballot(v < 0 || v >= a.experts); left; left &= left - 1) {
      const int p = win + wave * kWave + __ffsll(static_cast<unsigned long long>(left)) - 1;
      for (int o = lane; o < rows; o += kWave) w4_store(a, int64_t(p) * a.n + row0 + o, 0.f);
    }
  }
}

// The pair (routed form) or row that token t of the workgroup's tile is.
template <bool ROUTED, int TX>
__device__ __forceinline__ int w4_row(const W4Tile<TX>& tile, int t) {
  if constexpr (!ROUTED) return int(blockIdx.y) * TX + t;
  else if constexpr (TX == 1) return blockIdx.y;
  else return tile.pair[t];
}

// ---- k split over the waves --------------------------------------------------
// What a block needs comes to the wave's own part of LDS by direct copies,
// kBlocks blocks deep, in kCopies instructions.
template <bool Z, int G, int TX, int R, int U>
struct W4Ring {
  using Scales = W4Scales<R, U * (128 / G)>;
  static constexpr int kCodeCopies = U * R, kXCopies = (TX * U + 3) / 4;  // 1 KB each
  // Counted per block; those of a period of several blocks are not (the waits are then a little stricter).
  static constexpr int kCopies = kCodeCopies + kXCopies + (Scales::kPeriod == 1 ? Scales::kCopies * (Z ? 2 : 1) : 0);
  static constexpr int kX = kCodeCopies * 1024, kBlock = kX + kXCopies * 1024;
  static constexpr int kScaleSlot = Scales::kBytes * (Z ? 2 : 1);
  // Blocks in flight reach into this many periods.
  static constexpr int slots(int blocks) {
    return (blocks + Scales::kPeriod - 1) / Scales::kPeriod + (Scales::kPeriod > 1);
  }
  static constexpr int bytes(int blocks) { return blocks * kBlock + slots(blocks) * kScaleSlot; }
  static constexpr int deep(int blocks) {
    return bytes(blocks) * kW4Waves <= kW4LdsBytes || blocks == 2 ? blocks : deep(blocks - 1);
  }
  static constexpr int kBlocks = deep(5), kSlots = slots(kBlocks), kScales = kBlocks * kBlock;
  static constexpr int kWave = bytes(kBlocks);
  static_assert(kW4Waves * kWave <= kW4LdsBytes && kCopies * (kBlocks - 1) < 64, "LDS and vmcnt");
  static_assert(kWave >= 16 * R * 20 * 4, "the partial sums take the ring's place");
};

// For few rows.  Sets of 2^split_log2 waves of a workgroup take 16 R rows
// each, wave j of a set the blocks j, j + 2^split_log2, ...; the partial sums
// of a set are added through LDS at the end.  Nothing else is shared, so the
// waves run without barriers, each with its own copies of the activations it
// needs.
//
// Grid: x row blocks; y tiles of tokens, or the routed form's.
template <int FMT, bool Z, int G, int TX, int R, int U, bool ROUTED>
__global__ void __launch_bounds__(kW4Waves * kWave) w4_kernel(W4Args a) {
  using L = W4Ring<Z, G, TX, R, U>;
  using Block = W4Block<FMT, Z, G, TX, R, U>;
  using Scales = typename Block::Scales;
  constexpr int F = Block::F, A = Block::A, NB = L::kBlocks, kPieces = 4 * U, kUnits = 16 * U;
  constexpr int kRows = 16 * R, kRedLd = TX == 16 ? 20 : TX == 8 ? 10 : TX;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid >> 6), waves = blockDim.x >> 6;
  const int quarter = lane >> 4, col = lane & 15;
  const int lks = a.split_log2, ks = 1 << lks, kidx = wave & (ks - 1), set = wave >> lks;
  const int sets = waves >> lks, row0 = blockIdx.x * (sets * kRows);
  const unsigned half = unsigned(a.k) >> 1, groups = unsigned(a.k) / G;
  const int blocks = ((unsigned(a.k) + 128 * U - 1) / (128 * U) - kidx + ks - 1) >> lks;  // of this wave

  int e = 0, tt = min(TX, a.m - int(blockIdx.y) * TX);
  __shared__ W4Tile<TX> pairs;
  if constexpr (ROUTED) {
    e = w4_routed_tile<TX>(a, pairs, reinterpret_cast<int*>(lds), tt);
    if (e == a.experts) w4_store_zeros<TX>(a, row0, min(sets * kRows, a.n - row0));
    if (e < 0 || e == a.experts) return;
  }
  // the pair of the tile's token t, and its row of x
  const auto out_row = [&](int t) { return int64_t(w4_row<ROUTED, TX>(pairs, t)); };
  const auto x_row = [&](int t) { return int64_t(w4_row<ROUTED, TX>(pairs, t) / (ROUTED ? a.x_div : 1)); };
  const int64_t first_row = int64_t(e) * a.n + row0;
  const uint8_t* wbase = a.w + first_row * half;
  const char* sbase = static_cast<const char*>(a.scales) + ((first_row * groups) << (a.scales_bf16 ? 1 : 2));
  const uint8_t* zbase = Z ? a.zeros + first_row * groups : nullptr;
  const char* ring = lds + wave * L::kWave;
  const uint32_t ring_at = lds_addr(lds) + wave * L::kWave;

  // Code pieces past the row's end are its last piece again, scales past it the last one's; rows past the matrix its
  // last row.
  const auto row_of = [&](int r) { return unsigned(min(set * kRows + r, a.n - 1 - row0)); };
  unsigned cpos[L::kCodeCopies], cend[L::kCodeCopies], soff[R];
#pragma unroll
  for (int c = 0; c < L::kCodeCopies; ++c) {
    const int r = (c * 64 + lane) / kPieces;
    cend[c] = row_of(r) * half + half - 16;
    cpos[c] = row_of(r) * half + ((lane % kPieces) ^ w4_swap<U>(r)) * 16;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) soff[r] = row_of(r * 16 + (lane >> 2)) * groups;
  auto copy_weights = [&](int b) {
    const unsigned blk = kidx + (b << lks), at = ring_at + unsigned(b % NB) * L::kBlock;
    if (b % Scales::kPeriod == 0) {
      const unsigned to = ring_at + L::kScales + unsigned(b / Scales::kPeriod % L::kSlots) * L::kScaleSlot;
#pragma unroll
      for (int c = 0; c < Scales::kCopies; ++c) {
        const int h = c / R, r = c % R, i = lane & 3;  // part h, rows 16 r ..; the lane's i-th group
        const unsigned g = F >= 4 ? blk * F + 4 * h + i : (blk + ((i / F) << lks)) * F + i % F;
        const unsigned at_g = soff[r] + min(g, groups - 1);
        copy4_scale_to_lds(sbase, at_g, to + c * 256, a.scales_bf16);
        if constexpr (Z) copy1_zero_to_lds(zbase, at_g, to + Scales::kBytes + c * 256);
      }
    }
#pragma unroll
    for (int c = 0; c < L::kCodeCopies; ++c)
      copy16_to_lds(wbase, min(blk * (64 * U) + cpos[c], cend[c]), at + c * 1024);
  };

  const uint16_t* xsrc[L::kXCopies];  // this lane's unit of block 0; units past the end come from kW4Zeros
  int xunit[L::kXCopies];
#pragma unroll
  for (int c = 0; c < L::kXCopies; ++c) {
    const int t = (c * 64 + lane) / kUnits % TX;
    xunit[c] = (lane % kUnits) ^ (t & 15);
    xsrc[c] = a.x + x_row(min(t, tt - 1)) * a.x_ld + xunit[c] * 8;
  }
  auto copy_block = [&](int b) {
    const int unit0 = (kidx + (b << lks)) * kUnits;
    const uint32_t at = ring_at + unsigned(b % NB) * L::kBlock;
    if (unit0 + kUnits <= a.k >> 3) {
#pragma unroll
      for (int c = 0; c < L::kXCopies; ++c)
        copy16_scattered_to_lds(xsrc[c] + unit0 * 8, at + L::kX + c * 1024);
    } else {
#pragma unroll
      for (int c = 0; c < L::kXCopies; ++c)
        copy16_scattered_to_lds(
            unit0 + xunit[c] < a.k >> 3 ? static_cast<const void*>(xsrc[c] + unit0 * 8) : &kW4Zeros,
            at + L::kX + c * 1024);
    }
    copy_weights(b);
  };
#pragma unroll
  for (int b = 0; b < NB; ++b)
    if (b < blocks) copy_block(b);

  const int token = w4_token<TX>(col);
  const unsigned scale_shift = a.scales_bf16 ? 16 : 0;
  float acc[R][A] = {};
  // Waits for block b and starts its LDS reads.
  auto read = [&](Block& o, int b) {
    const int newer = min(blocks - 1 - b, NB - 1);  // blocks in flight after this one
    if (newer >= NB - 1) copies_left<(NB - 1) * L::kCopies>();
    else if (NB > 4 && newer == 3) copies_left<(NB > 4 ? 3 : 0) * L::kCopies>();
    else if (NB > 3 && newer == 2) copies_left<(NB > 3 ? 2 : 0) * L::kCopies>();
    else if (newer == 1) copies_left<L::kCopies>();
    else copies_left<0>();
    const char* at = ring + (b % NB) * L::kBlock;
    const char* scales = ring + L::kScales + b / Scales::kPeriod % L::kSlots * L::kScaleSlot;
    o.s.read(scales, col, b % Scales::kPeriod);
    if constexpr (Z) o.z.read(scales + Scales::kBytes, col, b % Scales::kPeriod);
    o.read_codes(at, quarter, col);
    o.read_x(at + L::kX + token * (kUnits * 16), quarter, token);
  };
  // Block b's products while block b + 1 is read from LDS; its place is then copied anew.
  auto turn = [&](Block& now, Block& next, int b) {
    if (b + 1 < blocks) read(next, b + 1);
    __builtin_amdgcn_sched_barrier(0);
    now.products(acc, (kidx + (b << lks)) * F, groups, scale_shift);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // block b + 1 has been read
    if (b + 1 + NB < blocks) copy_block(b + 1 + NB);
  };
  Block o0, o1;
  if (blocks > 0) {
    read(o0, 0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (NB < blocks) copy_block(NB);
  }
  for (int b = 0; b < blocks; b += 2) {
    turn(o0, o1, b);
    if (b + 1 < blocks) turn(o1, o0, b + 1);
  }

  // ---- the sets' partial sums, added in the order of their waves
  float* red = reinterpret_cast<float*>(lds);
  lds_barrier();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float* p = red + (wave * kRows + r * 16 + col) * kRedLd;
    if constexpr (TX == 16)
      *reinterpret_cast<v4f*>(p + quarter * 4) = v4f{acc[r][0], acc[r][1], acc[r][2], acc[r][3]};
    else if constexpr (TX == 8)
      *reinterpret_cast<v2f*>(p + quarter * 2) = v2f{acc[r][0], acc[r][1]};
    else if (quarter < TX) p[quarter] = acc[r][0];
  }
  lds_barrier();
  bool past = false;  // of this thread's outputs one is not finite
  const int outs = sets * kRows * TX;
  const auto place = [&](int o, int& st, int& rr, int& t, int& row) {
    rr = o % kRows, t = o / kRows % TX, st = o / (kRows * TX), row = row0 + st * kRows + rr;
    return row < a.n && t < tt;
  };
  for (int o = tid; o < outs; o += waves * kWave) {
    int st, rr, t, row;
    const bool wanted = place(o, st, rr, t, row);
    const float* p = red + ((st << lks) * kRows + rr) * kRedLd + t;
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < kW4Waves; ++j) {  // all reads at once
      const float u = p[(j & (ks - 1)) * kRows * kRedLd];
      v += j < ks ? u : 0.f;
    }
    if (!wanted) continue;
    w4_store(a, out_row(t) * a.n + row, v);
    past |= !w4_finite(v);
  }
  if (__builtin_expect(__ballot(past) == 0, 1)) return;
  copies_left<0>();  // the stores are done
  W4Nans nans;
  for (int o0 = wave * kWave; o0 < outs; o0 += waves * kWave) {
    int st, rr, t, row;
    const bool wanted = place(min(o0 + lane, outs - 1), st, rr, t, row) && o0 + lane < outs;
    w4_mend<FMT, Z, G>(a, wanted, wanted ? out_row(t) * a.n + row : 0, int64_t(e) * a.n + row, wanted ? x_row(t) : 0, t,
                       nans);
  }
}

// ---- whole rows per wave -----------------------------------------------------
// Rings of codes and scales alone.
template <bool Z, int G, int R, int U>
struct W4StreamRing {
  using Scales = W4Scales<R, U * (128 / G)>;
  static constexpr int kCodeCopies = U * R;
  static constexpr int kCopies = kCodeCopies + (Scales::kPeriod == 1 ? Scales::kCopies * (Z ? 2 : 1) : 0);
  static constexpr int kBlock = kCodeCopies * 1024, kBlocks = 3;
  static constexpr int kScaleSlot = Scales::kBytes * (Z ? 2 : 1);
  static constexpr int kSlots = kBlocks + (Scales::kPeriod > 1);  // a short row begins a period with every block
  static constexpr int kScales = kBlocks * kBlock, kWave = kScales + kSlots * kScaleSlot;
};

// Where rows are plenty: every wave takes whole rows (16 R at a time, no split
// of k), one set after the other without a pause, and the workgroup's waves
// share the tile's activations, which stay in LDS.
//
// Grid: x groups of `reps` row sets per wave; y as in w4_kernel.
template <int FMT, bool Z, int G, int TX, int R, int U, bool ROUTED>
__global__ void __launch_bounds__(kW4Waves * kWave) w4_stream_kernel(W4Args a) {
  using L = W4StreamRing<Z, G, R, U>;
  using Block = W4Block<FMT, Z, G, TX, R, U>;
  using Scales = typename Block::Scales;
  constexpr int F = Block::F, A = Block::A, NB = L::kBlocks, kPieces = 4 * U, kUnits = 16 * U;
  constexpr int kRows = 16 * R;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid >> 6);
  const int quarter = lane >> 4, col = lane & 15;
  const unsigned half = unsigned(a.k) >> 1, groups = unsigned(a.k) / G;
  const int blocks = (unsigned(a.k) + 128 * U - 1) / (128 * U);
  const int sets = (a.n + kRows - 1) / kRows;
  const int first_set = blockIdx.x * (kW4Waves * a.reps), set0 = first_set + wave;  // then every kW4Waves-th
  const int total = max(0, min(a.reps, (sets - set0 + kW4Waves - 1) / kW4Waves)) * blocks;

  int e = 0, tt = min(TX, a.m - int(blockIdx.y) * TX);
  __shared__ W4Tile<TX> pairs;
  if constexpr (ROUTED) {
    e = w4_routed_tile<TX>(a, pairs, reinterpret_cast<int*>(lds), tt);
    const int row0 = first_set * kRows;
    if (e == a.experts) w4_store_zeros<TX>(a, row0, min(kW4Waves * a.reps * kRows, a.n - row0));
    if (e < 0 || e == a.experts) return;
  }
  const auto out_row = [&](int t) { return int64_t(w4_row<ROUTED, TX>(pairs, t)); };
  const auto x_row = [&](int t) { return int64_t(w4_row<ROUTED, TX>(pairs, t) / (ROUTED ? a.x_div : 1)); };
  const int64_t first_row = int64_t(e) * a.n;
  const uint32_t ring_at = lds_addr(lds) + wave * L::kWave, x_at = lds_addr(lds) + kW4Waves * L::kWave;
  const char* ring = lds + wave * L::kWave;
  const char* x_lds = lds + kW4Waves * L::kWave;
  const int x_row_bytes = (blocks * (kUnits * 16) + 1023) & ~1023;

  // ---- the copies' side of the stream: the next block to bring
  int c_block = 0, c_set = set0, c_slot = 0, c_scale_slot = 0;
  const uint8_t* wbase;
  const char* sbase;
  const uint8_t* zbase;
  unsigned cpos[L::kCodeCopies], cend[L::kCodeCopies], soff[R];
  auto start_set = [&]() {
    const int64_t row = first_row + int64_t(c_set) * kRows;
    wbase = a.w + row * half;
    sbase = static_cast<const char*>(a.scales) + ((row * groups) << (a.scales_bf16 ? 1 : 2));
    zbase = Z ? a.zeros + row * groups : nullptr;
    const int last = a.n - 1 - c_set * kRows;  // rows past the end are the last row again
#pragma unroll
    for (int c = 0; c < L::kCodeCopies; ++c) {
      const int r = (c * 64 + lane) / kPieces;
      const unsigned at = unsigned(min(r, last)) * half;
      cend[c] = at + half - 16;
      cpos[c] = at + ((lane % kPieces) ^ w4_swap<U>(r)) * 16;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) soff[r] = unsigned(min(r * 16 + (lane >> 2), last)) * groups;
  };
  auto copy_next = [&]() {
    const unsigned at = ring_at + unsigned(c_slot) * L::kBlock, blk = c_block;
    if (c_block % Scales::kPeriod == 0) {
      const unsigned to = ring_at + L::kScales + unsigned(c_scale_slot) * L::kScaleSlot;
      c_scale_slot = c_scale_slot + 1 == L::kSlots ? 0 : c_scale_slot + 1;
#pragma unroll
      for (int c = 0; c < Scales::kCopies; ++c) {
        const int h = c / R, r = c % R;
        const unsigned g = soff[r] + min(blk * F + 4 * h + (lane & 3), groups - 1);
        copy4_scale_to_lds(sbase, g, to + c * 256, a.scales_bf16);
        if constexpr (Z) copy1_zero_to_lds(zbase, g, to + Scales::kBytes + c * 256);
      }
    }
#pragma unroll
    for (int c = 0; c < L::kCodeCopies; ++c)
      copy16_to_lds(wbase, min(blk * (64 * U) + cpos[c], cend[c]), at + c * 1024);
    c_slot = c_slot + 1 == NB ? 0 : c_slot + 1;
    if (++c_block == blocks) {
      c_block = 0;
      c_set += kW4Waves;
      start_set();
    }
  };
  start_set();
#pragma unroll
  for (int b = 0; b < NB; ++b)
    if (b < total) copy_next();

  // the activations: token t's units, exchanged by t; units past the end are zero
  const int per = x_row_bytes >> 10;
  for (int c = wave; c < tt * per; c += kW4Waves) {
    const int t = c / per, unit = ((c % per) * 64 + lane) ^ (t & 15);
    const void* src = unit < a.k >> 3 ? static_cast<const void*>(a.x + x_row(t) * a.x_ld + unit * 8) : &kW4Zeros;
    copy16_scattered_to_lds(src, x_at + c * 1024);
  }
  copies_left<0>();
  lds_barrier();

  const int token = w4_token<TX>(col);
  const char* x_mine = x_lds + token * x_row_bytes;
  const unsigned scale_shift = a.scales_bf16 ? 16 : 0;
  float acc[R][A] = {};
  int block = 0, slot = 0, scale_slot = L::kSlots - 1, set = set0;
  bool past = false;  // of this lane's outputs one is not finite
  for (int b = 0; b < total; ++b) {
    const int newer = min(total - 1 - b, NB - 1);  // blocks in flight after this one
    if (newer == 2) copies_left<2 * L::kCopies>();
    else if (newer == 1) copies_left<L::kCopies>();
    else copies_left<0>();
    const char* at = ring + slot * L::kBlock;
    slot = slot + 1 == NB ? 0 : slot + 1;
    if (block % Scales::kPeriod == 0) scale_slot = scale_slot + 1 == L::kSlots ? 0 : scale_slot + 1;
    const char* scales = ring + L::kScales + scale_slot * L::kScaleSlot;
    Block o;
    o.s.read(scales, col, block % Scales::kPeriod);
    if constexpr (Z) o.z.read(scales + Scales::kBytes, col, block % Scales::kPeriod);
    o.read_codes(at, quarter, col);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the block has been read
    if (b + NB < total) copy_next();
    o.read_x(x_mine + block * (kUnits * 16), quarter, token);
    o.products(acc, unsigned(block) * F, groups, scale_shift);
    if (++block == blocks) {  // the rows are done
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = set * kRows + r * 16 + col;
#pragma unroll
        for (int v = 0; v < A; ++v) {
          const int t = quarter * A + v;
          if (row < a.n && t < tt) {
            w4_store(a, out_row(t) * a.n + row, acc[r][v]);
            past |= !w4_finite(acc[r][v]);
          }
          acc[r][v] = 0.f;
        }
      }
      block = 0;
      set += kW4Waves;
    }
  }
  if (__builtin_expect(__ballot(past) == 0, 1)) return;
  copies_left<0>();  // the stores are done
  W4Nans nans;
  for (int st = set0; st < set; st += kW4Waves)
#pragma unroll 1
    for (int t0 = 0; t0 < tt; t0 += kWave / kRows) {
      const int t = min(t0 + lane / kRows, TX - 1), row = st * kRows + lane % kRows;
      const bool wanted = row < a.n && t0 + lane / kRows < tt;
      w4_mend<FMT, Z, G>(a, wanted, wanted ? out_row(t) * a.n + row : 0, int64_t(e) * a.n + row, wanted ? x_row(t) : 0,
                         t, nans);
    }
}

}  // namespace fp8g
