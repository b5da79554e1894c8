// The step between two blocks of a model, and its gradients, for gfx950.
//
//   u = norm(x) post_weight   (or x),     h = residual_scale residual + gate u,
//   y = norm(h) pre_weight    -> y in x's type, and / or FP8 codes with a scale per 128 columns
//   norm(v) = (v - mean) / sqrt(var + eps)   or   v / sqrt(mean v^2 + eps)
// All of it in FP32, every output rounded once; y and the codes come from h
// before it is rounded.
//
// Gradients, with gy that of y and gh that of h from everything else that
// reads it; h as the forward pass stored it:
//   a = gy pre_weight,  dh = gh + D(a, h),    grad_residual = residual_scale dh
//   du = gate dh,       grad_gate = dh u  (summed over rows where rows share it)
//   grad_x = D(du post_weight, x)  (or du)
//   grad_pre_weight = sum over rows of gy n(h),  grad_post_weight = that of du n(x)
//   D(b, v) = (b - n mean(b n) [- mean b]) / sqrt(..),  n = norm(v)   [layer norms]
#pragma once

#include "cast_kernel.hpp"
#include "gemm_kernel.hpp"  // xcd_logical

namespace fp8g {

struct NormArgs {
  const void *x, *residual, *post_weight, *gate, *pre_weight;
  void *h, *y;
  uint8_t* q;
  float* q_scales;
  int64_t x_ld, residual_ld, q_ld;
  int rows, n;
  bool post_norm, gate_per_row, params_bf16, q_e5m2;
  float eps, residual_scale;
};

struct NormGradArgs {
  const void *grad_h, *grad_y, *x, *h, *post_weight, *gate, *pre_weight;
  void *grad_x, *grad_residual;
  float* grad_gate;  // [rows][n], of a gate per row
  float* partial;    // [slices][3][n]: pre_weight, post_weight, gate; null: no sums
  int64_t x_ld;
  int rows, n, rows_per_slice;
  bool post_norm, params_bf16;
  float eps, residual_scale;
};

// 8 consecutive elements as they are stored.
template <typename T>
struct Raw8 {
  static constexpr int kWords = sizeof(T) / 2;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at);
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = p[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  // What was made of the values is not to be kept: the compiler takes them to be new.
  __device__ __forceinline__ void renew() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i].x), "+v"(w[i].y), "+v"(w[i].z), "+v"(w[i].w));
  }
  __device__ __forceinline__ void get(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4& q = w[i * kWords / 8];
      const int at = kWords == 2 ? i & 3 : i >> 1;
      const uint32_t u = at == 0 ? q.x : at == 1 ? q.y : at == 2 ? q.z : q.w;
      v[i] = __uint_as_float(kWords == 2 ? u : i & 1 ? u & 0xffff0000u : u << 16);
    }
  }
};

template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t at, const float v[8]) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<T*>(base) + at);
  if constexpr (sizeof(T) == 4) {
    p[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    p[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    p[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
}

// 8 values of a parameter (FP32 or BF16), 1 where there is none.
__device__ __forceinline__ void param8(const void* p, bool bf16, int64_t at, float v[8]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.f;
  } else if (bf16) {
    load8(static_cast<const uint16_t*>(p) + at, v);
  } else {
    load8(static_cast<const float*>(p) + at, v);
  }
}

// The same, loaded early and used late.
struct RawParam {
  uint4 w[2];
  __device__ __forceinline__ void load(const void* p, bool bf16, int64_t at) {
    if (!p) return;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (bf16 ? 2 : 4));
    w[0] = q[0];
    if (!bf16) w[1] = q[1];
  }
  __device__ __forceinline__ void get(const void* p, bool bf16, float v[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4& f = w[i / 4];
      const uint32_t f32 = (i & 3) == 0 ? f.x : (i & 3) == 1 ? f.y : (i & 3) == 2 ? f.z : f.w;
      const uint32_t h = (i >> 1) == 0 ? w[0].x : (i >> 1) == 1 ? w[0].y : (i >> 1) == 2 ? w[0].z : w[0].w;
      v[i] = !p ? 1.f : __uint_as_float(!bf16 ? f32 : i & 1 ? h & 0xffff0000u : h << 16);
    }
  }
};

// v of the lane that a DPP pattern names, within rows of 16 lanes (a few cycles; a shuffle goes through LDS).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
constexpr int kSwapPairs = 0xB1, kSwapHalves = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

// f over the 16 lanes of a row, over the wave: in every lane.
template <typename F>
__device__ __forceinline__ float row16(float v, F&& f) {
  v = f(v, dpp<kSwapPairs>(v));
  v = f(v, dpp<kSwapHalves>(v));
  v = f(v, dpp<kMirror8>(v));
  return f(v, dpp<kMirror16>(v));
}
__device__ __forceinline__ float sum16(float v) {
  return row16(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float max16(float v) {
  return row16(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  const int a = __float_as_int(v);
  const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);  // the rows of each pair apart
  v = __int_as_float(r[0]) + __int_as_float(r[1]);
  const int b = __float_as_int(v);
  const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);  // the halves apart
  return __int_as_float(h[0]) + __int_as_float(h[1]);
}

// Sums of up to four values over the `waves` waves of a row (one wave: no barrier).  `part`: a place of LDS that no
// other call uses until every wave has passed another barrier.
constexpr int kNormMaxWaves = 16;
struct NormPart {
  float v[4][kNormMaxWaves];
};
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int waves, NormPart& part) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  const int lane = threadIdx.x & (kWave - 1);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) part.v[i][threadIdx.x >> 6] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = sum16((lane & 15) < waves ? part.v[i][lane & 15] : 0.f);
  }
}

// v = norm(v) over a row's n columns, of which this thread holds C pieces of 8; returns 1 / sqrt(..).  `in`: the piece
// is inside the row (the others hold zeros, before and after).
template <bool LAYER, int C>
__device__ __forceinline__ float normalise(float (&v)[C][8], const bool (&in)[C], int n, float eps, int waves,
                                           NormPart* parts) {
  float s[1] = {0.f};
  if constexpr (LAYER) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[c][i];
    row_sums(s, waves, parts[0]);
    const float mean = s[0] / n;
    s[0] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = in[c] ? v[c][i] - mean : 0.f;
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] = fmaf(v[c][i], v[c][i], s[0]);
  row_sums(s, waves, parts[1]);
  const float r = 1.f / sqrtf(s[0] / n + eps);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] *= r;
  return r;
}

// A thread holds C pieces of 8 columns, blockDim.x threads a row, blockDim.y rows a workgroup (more than one only
// where a row is one wave's).  Consecutive rows run on one XCD, so that its L2 gathers the lines of the scales.
//
// A row is read once and stays in registers.  Many rows are bound by memory: 16384 x 7168 with its codes 172 us, 4.8
// TB/s; 5003 x 2120 layer norms with an FP32 stream 34 us, 3.7 TB/s (four rounds of sums a row, whose waits the six rows
// of a CU do not cover quite).  One row of 7168 takes 4.4 us, a launch and the chain of two loads and two sums.
template <typename X, typename R, bool LAYER, int C>
__global__ void __launch_bounds__(C == 1 ? 1024 : 512) norm_residual_kernel(const NormArgs a) {
  __shared__ NormPart parts[4];
  const int row = xcd_logical(blockIdx.x, gridDim.x) * int(blockDim.y) + int(threadIdx.y);
  if (row >= a.rows) return;  // (whole waves: no barrier is left out)
  const int waves = blockDim.x >> 6;
  int col[C];
  bool in[C];
  float v[C][8];
  Raw8<X> xs[C];
  Raw8<R> rs[C];
  // Few rows, a piece each: the parameters are on their way with the row.  Else they are read where they are used (from
  // the cache; the registers are worth more to the rows that run beside this one).
  constexpr bool EARLY = C == 1;
  RawParam post = {}, gate = {}, pre = {};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = 8 * int(threadIdx.x + c * blockDim.x);
    in[c] = col[c] < a.n;
    xs[c].clear();
    rs[c].clear();
    if (in[c]) {
      xs[c].load(a.x, row * a.x_ld + col[c]);
      if (a.residual) rs[c].load(a.residual, row * a.residual_ld + col[c]);
      if (EARLY) {
        post.load(a.post_weight, a.params_bf16, col[c]);
        gate.load(a.gate, a.params_bf16, (a.gate_per_row ? int64_t(row) * a.n : 0) + col[c]);
        pre.load(a.pre_weight, a.params_bf16, col[c]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) xs[c].get(v[c]);
  if (a.post_norm) normalise<LAYER>(v, in, a.n, a.eps, waves, parts);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (!in[c]) continue;
    float w[8], r[8];
    if (a.post_norm && a.post_weight) {
      if (EARLY) post.get(a.post_weight, a.params_bf16, w);
      else param8(a.post_weight, a.params_bf16, col[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= w[i];
    }
    if (a.gate) {
      if (EARLY) gate.get(a.gate, a.params_bf16, w);
      else param8(a.gate, a.params_bf16, (a.gate_per_row ? int64_t(row) * a.n : 0) + col[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= w[i];
    }
    if (a.residual) {
      rs[c].get(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = fmaf(a.residual_scale, r[i], v[c][i]);
    }
    if (a.h) store8<R>(a.h, int64_t(row) * a.n + col[c], v[c]);
  }
  if (!a.y && !a.q) return;
  normalise<LAYER>(v, in, a.n, a.eps, waves, parts + 2);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (in[c]) {
      float w[8];
      if (EARLY) pre.get(a.pre_weight, a.params_bf16, w);
      else param8(a.pre_weight, a.params_bf16, col[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= w[i];
      if (a.y) store8<X>(a.y, int64_t(row) * a.n + col[c], v[c]);
    }
    if (a.q) {  // as the per-token-group cast: 16 lanes hold a group
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[c][i]));
      top = max16(top);
      const float s = a.q_e5m2 ? group_scale<kFmtE5M2>(top) : group_scale<kFmtE4M3>(top);
      float d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = __fdiv_rn(v[c][i], s);
      uint2 w;
      if (a.q_e5m2) {
        w.x = fp8x4<kFmtE5M2>(d[0], d[1], d[2], d[3]);
        w.y = fp8x4<kFmtE5M2>(d[4], d[5], d[6], d[7]);
      } else {
        w.x = fp8x4<kFmtE4M3>(d[0], d[1], d[2], d[3]);
        w.y = fp8x4<kFmtE4M3>(d[4], d[5], d[6], d[7]);
      }
      if (in[c]) {
        *reinterpret_cast<uint2*>(a.q + int64_t(row) * a.n + col[c]) = w;
        if ((threadIdx.x & 15) == 0) a.q_scales[(col[c] >> 7) * a.q_ld + row] = s;
      }
    }
  }
}

// Grid: slices of rows, which a workgroup takes blockDim.y at a time, each thread with its C pieces of 8 columns, whose
// sums over the rows stay in its registers and are added through LDS at the end where there are several rows at a time.
// What a row needs of itself takes two rounds of sums (three for layer norms, whose squares are of centred values):
//   sum h^2, sum a h, sum x^2  ->  dh  ->  sum b x,  b = du post_weight
// The next row is read while this one is worked on, which works because nothing else is read meanwhile: memory answers
// in order, so a wait for a parameter would be one for the next row.  The parameters therefore lie in LDS, as FP32
// (8192 x 4096 with its sums 95 us; 101 as they are stored, chosen and unpacked at every use; 107 from memory), but for a
// workgroup that has no next row (257 x 2048: 11.7 us, 12.5 with them there).
// Rows of more than 8192 columns (two pieces a thread) leave no registers for the next row: their threads keep only
// what is packed, d and one of the three sums, the other two lie in LDS, and the parameters come from the cache
// (2048 x 12288: 106 us; all in registers, which spilled, 219).
//
// Bound by memory, and nearly by vector instructions (some 300 for a thread's 8 columns): 8192 x 4096 at 4.5 TB/s in 90
// us, 16 waves a CU, and 5 for the sums of 256 or 512 slices.
constexpr int kNormGradRows = 8;  // rows at a time, at most
template <typename X, typename R, bool LAYER, bool ROW_GATE, int C, int MAX_THREADS, bool IN_LDS>
__global__ void __launch_bounds__(MAX_THREADS) norm_residual_backward_kernel(const NormGradArgs a) {
  constexpr bool SEVERAL = C == 1 && MAX_THREADS == 512;  // rows at a time, perhaps
  __shared__ NormPart parts[2][3][SEVERAL ? kNormGradRows : 1];
  const int ty = SEVERAL ? uniform(threadIdx.y) : 0, at_once = SEVERAL ? blockDim.y : 1;
  extern __shared__ __attribute__((aligned(16))) float params[];  // IN_LDS: pre_weight, post_weight, gate
  const int tid = ty * blockDim.x + threadIdx.x, threads = blockDim.x * at_once;
  constexpr bool KEEP = C == 1;  // what is unpacked, and the sums, stay in registers
  const void* const shared[3] = {a.pre_weight, a.post_weight, ROW_GATE ? nullptr : a.gate};
  auto param = [&](int k, unsigned c, float (&v)[8]) {
    if constexpr (IN_LDS) load8(params + k * a.n + c, v);
    else param8(shared[k], a.params_bf16, c, v);
  };
  const int waves = blockDim.x >> 6, n = a.n;
  const float inv_n = 1.f / n;
  unsigned col[C];  // beside addresses that are a wave's
  bool in[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = 8 * (threadIdx.x + c * blockDim.x);
    in[c] = int(col[c]) < n;
  }
  float s_pre[C][8] = {}, s_post[KEEP ? C : 1][8] = {}, s_gate[KEEP ? C : 1][8] = {};
  float* const long_sums = params;  // !KEEP: post_weight's, gate's
  if constexpr (!KEEP) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (in[c]) store8<float>(long_sums, col[c], s_post[0]), store8<float>(long_sums, n + col[c], s_post[0]);
  }
  const int first = blockIdx.x * a.rows_per_slice, last = min(a.rows, first + a.rows_per_slice);
  Raw8<X> xs[C], gys[C];
  Raw8<R> hs[C], ghs[C];
  auto load = [&](int row) {
    const int64_t at0 = int64_t(row) * n;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!in[c]) continue;
      if (a.x) xs[c].load(static_cast<const X*>(a.x) + row * a.x_ld, col[c]);
      if (a.grad_y) {
        gys[c].load(static_cast<const X*>(a.grad_y) + at0, col[c]);
        hs[c].load(static_cast<const R*>(a.h) + at0, col[c]);
      }
      if (a.grad_h) ghs[c].load(static_cast<const R*>(a.grad_h) + at0, col[c]);
    }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) xs[c].clear(), gys[c].clear(), hs[c].clear(), ghs[c].clear();
  if (first + ty < last) load(first + ty);
  if constexpr (IN_LDS) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      for (int i = tid * 8; i < n; i += threads * 8) {
        float v[8];
        param8(shared[k], a.params_bf16, i, v);
        store8<float>(params, k * n + i, v);
      }
    __syncthreads();
  }
  int turn = 0;
  for (int round = first; round < last; round += at_once, turn ^= 1) {  // every wave takes every round
    const int row = round + ty;
    const bool live = !SEVERAL || row < last;
    // A column that may be new every time keeps every tensor's address in scalar registers: kept per lane and advanced
    // from row to row, they spilled.
#pragma unroll
    for (int c = 0; c < C; ++c) asm volatile("" : "+v"(col[c]));
    const int64_t at0 = int64_t(row) * n;
    auto& part = parts[turn];
    float x_[C][8], h_[C][8], gy_[C][8], d[C][8], mean_h = 0.f, mean_x = 0.f;
    if constexpr (KEEP) xs[0].get(x_[0]), hs[0].get(h_[0]), gys[0].get(gy_[0]);
#pragma unroll
    for (int c = 0; c < C; ++c) ghs[c].get(d[c]);
    if constexpr (KEEP)  // unpacked here: put off past the next row's loads, it takes a copy of what is packed
#pragma unroll
      for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(x_[0][i]), "+v"(h_[0][i]), "+v"(gy_[0][i]), "+v"(d[0][i]));
    if (KEEP && row + at_once < last) load(row + at_once);
    auto get_x = [&](int c, float (&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8 && KEEP; ++i) v[i] = x_[c][i];
      if constexpr (!KEEP) {
        xs[c].get(v);
#pragma unroll
        for (int i = 0; i < 8 && LAYER; ++i) v[i] -= mean_x;
      }
    };
    auto get_h = [&](int c, float (&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8 && KEEP; ++i) v[i] = h_[c][i];
      if constexpr (!KEEP) {
        hs[c].get(v);
#pragma unroll
        for (int i = 0; i < 8 && LAYER; ++i) v[i] -= mean_h;
      }
    };
    auto get_gy = [&](int c, float (&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8 && KEEP; ++i) v[i] = gy_[c][i];
      if constexpr (!KEEP) gys[c].get(v);
    };
    auto next_piece = [&](int c) {
      if constexpr (!KEEP) {
        __builtin_amdgcn_sched_barrier(0);
        xs[c].renew(), hs[c].renew(), gys[c].renew();
      }
    };
    if constexpr (LAYER) {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float x[8], h[8];
        get_x(c, x), get_h(c, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[0] += h[i], m[1] += x[i];
        next_piece(c);
      }
      row_sums(m, waves, part[0][ty]);
      mean_h = m[0] * inv_n;
      if (a.post_norm) mean_x = m[1] * inv_n;
#pragma unroll
      for (int i = 0; i < 8 && KEEP; ++i) {
        h_[0][i] = in[0] ? h_[0][i] - mean_h : 0.f;
        x_[0][i] = in[0] ? x_[0][i] - mean_x : 0.f;
      }
    }
    float m[4] = {0.f, 0.f, 0.f, 0.f};  // of h^2, x^2, a h, a
    float rx = 1.f;
    if (a.grad_y || a.post_norm) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (!in[c]) continue;
        float w[8], x[8], h[8], gy[8];
        param(0, col[c], w);
        get_x(c, x), get_h(c, h), get_gy(c, gy);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float b = gy[i] * w[i];
          m[0] = fmaf(h[i], h[i], m[0]);
          m[1] = fmaf(x[i], x[i], m[1]);
          m[2] = fmaf(b, h[i], m[2]);
          m[3] += b;
        }
        next_piece(c);
      }
      row_sums(m, waves, part[1][ty]);
      if (a.post_norm) rx = 1.f / sqrtf(fmaf(m[1], inv_n, a.eps));
    }
    if (a.grad_y) {
      const float r = 1.f / sqrtf(fmaf(m[0], inv_n, a.eps));
      const float along = m[2] * inv_n * r * r, mean = LAYER ? m[3] * inv_n : 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (!in[c] || !live) continue;
        float w[8], h[8], gy[8];
        param(0, col[c], w);
        get_h(c, h), get_gy(c, gy);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s_pre[c][i] = fmaf(gy[i], h[i] * r, s_pre[c][i]);
          d[c][i] = fmaf(r, fmaf(-along, h[i], gy[i] * w[i]) - mean, d[c][i]);
        }
        next_piece(c);
      }
    }
    float b[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {  // d becomes the gradient of norm(x), or of x
      if (!in[c] || !live) continue;
      if (a.grad_residual) {
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = a.residual_scale * d[c][i];
        store8<R>(static_cast<R*>(a.grad_residual) + at0, col[c], g);
      }
      float w[8], x[8];
      param(1, col[c], w);
      get_x(c, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= rx;
      if (a.gate) {
        float u[8], g[8];
        if constexpr (ROW_GATE) param8(a.gate, a.params_bf16, at0 + col[c], g);
        else param(2, col[c], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = d[c][i] * (x[i] * w[i]);
        if constexpr (ROW_GATE) {
          if (a.grad_gate) store8<float>(a.grad_gate + at0, col[c], u);
        } else {
#pragma unroll
          for (int i = 0; i < 8 && KEEP; ++i) s_gate[c][i] += u[i];
          if constexpr (!KEEP) {
            float t[8];
            load8(long_sums + n + col[c], t);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] += u[i];
            store8<float>(long_sums, n + col[c], t);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] *= g[i];
      }
      if (a.post_norm) {
        float t[8];
        if constexpr (!KEEP) load8(long_sums + col[c], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& sum = KEEP ? s_post[c][i] : t[i];
          sum = fmaf(d[c][i], x[i], sum);
          d[c][i] *= w[i];
          b[0] = fmaf(d[c][i], x[i], b[0]);
          b[1] += d[c][i];
        }
        if constexpr (!KEEP) store8<float>(long_sums, col[c], t);
      }
      next_piece(c);
    }
    if (a.post_norm) {
      row_sums(b, waves, part[2][ty]);
      const float along = b[0] * inv_n, mean = LAYER ? b[1] * inv_n : 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float x[8];
        get_x(c, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] = rx * (fmaf(-along, x[i] * rx, d[c][i]) - mean);
        next_piece(c);
      }
    }
    if (a.grad_x) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (in[c] && live) store8<X>(static_cast<X*>(a.grad_x) + at0, col[c], d[c]);
    }
    if (!KEEP && row + at_once < last) load(row + at_once);
  }
  if (!a.partial) return;
  float* const out = a.partial + int64_t(blockIdx.x) * 3 * n;
  auto put = [&](float (&sum)[C][8], int64_t at) {
    if (SEVERAL && at_once > 1) {  // the rows' sums in order
      float* const mine = params + threadIdx.x * 8;
      static_assert(C == 1 || !SEVERAL, "several rows at a time have a piece a thread");
      __syncthreads();
      store8<float>(mine + ty * blockDim.x * 8, 0, sum[0]);
      __syncthreads();
      if (ty > 0) return;
      for (int y = 1; y < at_once; ++y) {
        float v[8];
        load8(mine + y * blockDim.x * 8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0][i] += v[i];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (in[c]) store8<float>(out, at + col[c], sum[c]);
  };
  put(s_pre, 0);
  if constexpr (KEEP) {
    put(s_post, n);
    put(s_gate, 2 * int64_t(n));
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!in[c]) continue;
      float t[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        load8(long_sums + k * n + col[c], t);
        store8<float>(out, (k + 1) * int64_t(n) + col[c], t);
      }
    }
  }
}

}  // namespace fp8g
