// Expert routing for gfx950: top-k experts and weights of every token from
// its router logits, and the gradient of the logits.
//
// What is computed, per token t, over experts e = 0 .. E - 1 in G groups of
// E / G consecutive experts:
//   eligible(e):  logit l_e > -inf (a NaN is not) and, with a bias, b_e > -inf;
//   score:        s_e = 1 / (1 + exp(-l_e)) or exp(l_e) / sum of exp(l) over
//                 the logits above -inf;
//   selection:    sigma_e = s_e + b_e for eligible experts, the others are
//                 never picked; a group's score is the largest sigma of its
//                 members or the sum of the two largest; the topk_groups best
//                 groups stay, and of their experts the topk best are picked,
//                 best first, ties to the lowest index everywhere;
//   weights:      w_j = scale * s_j, or scale * s_j / sum of the picked s.
// Picks that do not exist (fewer eligible experts than topk) have index -1
// and weight 0.  All arithmetic is FP32.
#pragma once

#include "device_common.hpp"

namespace fp8g {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxGroups = 64;
constexpr int kRouteMaxTopk = 32;
constexpr int kScoreSoftmax = 0, kScoreSigmoid = 1;
constexpr int kGroupMax = 0, kGroupTop2 = 1;
constexpr float kNegInf = -__builtin_inff();
constexpr float kMaxFinite = 3.402823466e38f;

struct RouteShape {
  int T, E, groups, topk_groups, topk;
  int score, group_score, renormalize;
  float scale;
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = uint16_t(pack_bf16x2(v, 0.f)); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// Orders a wave's LDS accesses: the lanes after it see what every lane wrote before it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// l - m, 0 where both are the same infinity.
__device__ __forceinline__ float below(float l, float m) { return l == m ? 0.f : l - m; }
__device__ __forceinline__ float sigmoid(float l) { return 1.f / (1.f + expf(-l)); }

// Index of the largest v (ties to the lowest i), -1 if no lane has one; every lane gets it.
__device__ __forceinline__ int wave_argmax(float v, int i) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const float u = __shfl_xor(v, d, kWave);
    const int j = __shfl_xor(i, d, kWave);
    if (u > v || (u == v && unsigned(j) < unsigned(i))) {
      v = u;
      i = j;
    }
  }
  return i;
}

// One wave per token, 4 tokens per workgroup; scores in LDS, picks one at a time.
template <typename L>
__global__ void __launch_bounds__(256) moe_route_kernel(const L* __restrict__ logits, int64_t ld,
                                                        const float* __restrict__ bias, RouteShape r,
                                                        int32_t* __restrict__ expert_idx,
                                                        float* __restrict__ weights) {
  __shared__ float sigma[4][kRouteMaxExperts];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= r.T) return;
  float* sel = sigma[wave];
  const L* row = logits + int64_t(t) * ld;
  float top = kNegInf;
  for (int e = lane; e < r.E; e += kWave) top = fmaxf(top, load_logit(row + e));
  top = wave_max(top);
  float sum = 0.f;
  if (r.score == kScoreSoftmax) {
    for (int e = lane; e < r.E; e += kWave) {
      const float l = load_logit(row + e);
      if (l > kNegInf) sum += expf(below(l, top));
    }
    sum = wave_sum(sum);
  }
  for (int e = lane; e < r.E; e += kWave) {
    const float l = load_logit(row + e), b = bias ? bias[e] : 0.f;
    const float s = r.score == kScoreSoftmax ? expf(below(l, top)) / sum : sigmoid(l);
    sel[e] = (l > kNegInf && b > kNegInf) ? fmaxf(s + b, -kMaxFinite) : kNegInf;
  }
  wave_sync();
  if (r.groups > 1) {
    const int size = r.E / r.groups;
    float best = kNegInf;
    if (lane < r.groups) {
      float m1 = kNegInf, m2 = kNegInf;
      for (int i = 0; i < size; ++i) {
        const float v = sel[lane * size + i];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
      best = (r.group_score == kGroupTop2 && m2 > kNegInf) ? fmaxf(m1 + m2, -kMaxFinite) : m1;
    }
    bool keep = false;
    for (int i = 0; i < r.topk_groups; ++i) {
      const int g = wave_argmax(best, best > kNegInf ? lane : -1);
      if (lane == g) {
        keep = true;
        best = kNegInf;
      }
    }
    if (lane < r.groups && !keep)
      for (int i = 0; i < size; ++i) sel[lane * size + i] = kNegInf;
    wave_sync();
  }
  int mine = -1;  // lane j: pick j
  for (int j = 0; j < r.topk; ++j) {
    float v = kNegInf;
    int at = -1;
    for (int e = lane; e < r.E; e += kWave)
      if (sel[e] > v) {
        v = sel[e];
        at = e;
      }
    at = wave_argmax(v, at);
    if (at >= 0) sel[at] = kNegInf;
    wave_sync();
    if (lane == j) mine = at;
  }
  const float l = mine >= 0 ? load_logit(row + mine) : kNegInf;
  float w = 0.f;
  if (r.renormalize) {
    const float m = wave_max(l);
    if (mine >= 0) {
      if (r.score == kScoreSoftmax) w = expf(below(l, m));
      else w = l >= 0.f ? sigmoid(l) : expf(below(l, fminf(m, 0.f))) / (1.f + expf(l));
    }
    const float total = wave_sum(w);
    w = total > 0.f ? w / total : 0.f;
  } else if (mine >= 0) {
    w = r.score == kScoreSoftmax ? expf(below(l, top)) / sum : sigmoid(l);
  }
  if (lane < r.topk) {
    expert_idx[int64_t(t) * r.topk + lane] = mine;
    weights[int64_t(t) * r.topk + lane] = w * r.scale;
  }
}

// Gradient of the logits, one wave per token.  With c_j the gradient of the
// unnormalised score of pick j (renormalised weights: c_j = scale * (g_j -
// sum of g_i s_i / S) / S, S the sum of the picked scores; else scale * g_j):
//   sigmoid:  dl_e = c_e s_e (1 - s_e) on the picked experts, 0 elsewhere;
//   softmax:  dl_e = s_e (c_e - sum over the picks of c_j s_j); renormalised,
//             the sum vanishes and only the picked experts have a gradient.
// In terms of the weights: dl_e = v_e * (1 - s_e) resp. v_e - s_e * sum v
// with v_j = c_j s_j = scale * w_j * (g_j - [renormalised] sum of g_i w_i),
// w the weights before the scale.
template <typename L>
__global__ void __launch_bounds__(256) moe_route_backward_kernel(const L* __restrict__ logits, int64_t ld,
                                                                 const int32_t* __restrict__ expert_idx,
                                                                 const float* __restrict__ grad_weights,
                                                                 RouteShape r, L* __restrict__ grad, int64_t grad_ld) {
  __shared__ float dense[4][kRouteMaxExperts];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= r.T) return;
  float* v = dense[wave];
  for (int e = lane; e < r.E; e += kWave) v[e] = 0.f;
  wave_sync();
  const L* row = logits + int64_t(t) * ld;
  int e = lane < r.topk ? expert_idx[int64_t(t) * r.topk + lane] : -1;
  if (e >= r.E) e = -1;
  const float g = e >= 0 ? grad_weights[int64_t(t) * r.topk + lane] : 0.f;
  const float l = e >= 0 ? load_logit(row + e) : kNegInf;
  float top = kNegInf, sum = 1.f, w = 0.f;
  const bool dense_softmax = r.score == kScoreSoftmax && !r.renormalize;
  if (r.renormalize) {
    const float m = wave_max(l);
    if (e >= 0) {
      if (r.score == kScoreSoftmax) w = expf(below(l, m));
      else w = l >= 0.f ? sigmoid(l) : expf(below(l, fminf(m, 0.f))) / (1.f + expf(l));
    }
    const float total = wave_sum(w);
    w = total > 0.f ? w / total : 0.f;
  } else if (dense_softmax) {
    for (int i = lane; i < r.E; i += kWave) top = fmaxf(top, load_logit(row + i));
    top = wave_max(top);
    sum = 0.f;
    for (int i = lane; i < r.E; i += kWave) {
      const float x = load_logit(row + i);
      if (x > kNegInf) sum += expf(below(x, top));
    }
    sum = wave_sum(sum);
    if (e >= 0) w = expf(below(l, top)) / sum;
  } else if (e >= 0) {
    w = sigmoid(l);
  }
  float d = w * g;
  if (r.renormalize) d = w * (g - wave_sum(d));
  if (e >= 0) v[e] = r.scale * (r.score == kScoreSigmoid ? d * (1.f / (1.f + expf(l))) : d);
  wave_sync();
  const float mean = dense_softmax ? r.scale * wave_sum(d) : 0.f;
  for (int i = lane; i < r.E; i += kWave) {
    float x = v[i];
    if (dense_softmax) {
      const float li = load_logit(row + i);
      if (li > kNegInf) x -= expf(below(li, top)) / sum * mean;
    }
    store_logit(grad + int64_t(t) * grad_ld + i, x);
  }
}

}  // namespace fp8g
