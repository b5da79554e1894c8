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
//
// What bounds it: long batches the vector instructions of ranking (239 a token
// of 256 experts; the logits alone would take 7 us at the rate of a large
// copy), short ones the chain of loads and exchanges.  32768 tokens of 256
// experts (FP32, sigmoid, bias, 4 of 8 groups, top 8) take 15.7 us a call, 92
// with one wave per token that picks one expert at a time; 8 tokens 4.5 us
// (13.5).
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
constexpr float kSigmoidOne = 17.328679f;  // 25 ln 2: the sigmoid of more rounds to 1

struct RouteShape {
  int T, E, groups, topk_groups, topk;
  int score, group_score, renormalize;
  float scale;
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = uint16_t(pack_bf16x2(v, 0.f)); }

// l - m, 0 where both are the same infinity.
__device__ __forceinline__ float below(float l, float m) { return l == m ? 0.f : l - m; }

// exp(x) for -104 <= x <= 88 (0 from the bottom of the range on): exp2 of t, the rounded product of x with log2(e), and
// r, what t lacks of the exact product (by a fused multiply-add, and log2(e) in two parts), put back to first order:
// exp2(t + r) = exp2(t) (1 + r ln 2).  Without r, |x| * 2^-24 of relative error.
__device__ __forceinline__ float exp_near(float x) {
  const float t = x * 1.44269502f;
  const float r = fmaf(x, 1.92596303e-8f, fmaf(x, 1.44269502f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * 0.693147181f, e);
}
// 1 / d, one step of Newton's method after the 1-ulp estimate.
__device__ __forceinline__ float reciprocal(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return fmaf(fmaf(-d, r, 1.f), r, r);
}
__device__ __forceinline__ float sigmoid_near(float l) {
  return reciprocal(1.f + exp_near(-__builtin_amdgcn_fmed3f(l, -88.f, 88.f)));
}
// The same for ranking, without the Newton step: within 2^-21.4 of its value (an ulp each, 2^-23, of the exponential and
// the reciprocal, half an ulp each of the exponential's correction and of the sum with 1); 0 below 2^-126.
__device__ __forceinline__ float sigmoid_rank(float l) {
  return __builtin_amdgcn_rcpf(1.f + exp_near(-__builtin_amdgcn_fmed3f(l, -88.f, 88.f)));
}
__device__ __forceinline__ float exp_below(float l, float m) { return exp_near(fmaxf(below(l, m), -104.f)); }

// ---- selection keys ----
// A selection score and its expert as one double: the score's FP32 value has
// 29 zero bits at the end of its double, the last 10 of which take the index
// so that of equal scores the lower index is larger.  One v_max_f64 and one
// v_min_f64 then order two (score, index) pairs exactly, ties included.
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ double key_max(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double key_min(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
// Experts that are not to be picked have the lowest score there is; any other is kept above it, by one step of FP32 (so
// that biases in the last thousandth of the range keep their order).  Logits that stand for a score above 0 are kept
// above that again.
constexpr float kNotAble = -kMaxFinite, kLeastAble = -0x1.fffffcp127f, kLeastLogit = -0x1.fffffap127f;
// rest = kRouteMaxExperts - 1 - expert; a score is no negative zero (it is a sum with a positive one, if of zeros).
__device__ __forceinline__ double make_key(float score, unsigned rest) {
  u32x2 k = __builtin_bit_cast(u32x2, double(score));
  k.x |= rest ^ (unsigned(__float_as_int(score) >> 31) & unsigned(kRouteMaxExperts - 1));
  return __builtin_bit_cast(double, k);
}
__device__ __forceinline__ int key_expert(double key) {
  const u32x2 k = __builtin_bit_cast(u32x2, key);
  const int i = int(k.x & unsigned(kRouteMaxExperts - 1));
  return key <= double(kNotAble) ? -1 : int(k.y) < 0 ? i : kRouteMaxExperts - 1 - i;
}

// The partner's value at level 0 .. 5 of an exchange in which after level n
// all 2^(n + 1) neighbouring lanes have met.
template <int LEVEL>
__device__ __forceinline__ unsigned partner(unsigned v) {
  if constexpr (LEVEL == 0) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);        // quad_perm 1 0 3 2
  else if constexpr (LEVEL == 1) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);   // quad_perm 2 3 0 1
  else if constexpr (LEVEL == 2) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);  // row_half_mirror
  else if constexpr (LEVEL == 3) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);  // row_mirror
  else return unsigned(__shfl_xor(int(v), 1 << LEVEL, kWave));
}
template <int LEVEL>
__device__ __forceinline__ float partner(float v) { return __uint_as_float(partner<LEVEL>(__float_as_uint(v))); }
template <int LEVEL>
__device__ __forceinline__ double partner(double v) {
  u32x2 k = __builtin_bit_cast(u32x2, v);
  k.x = partner<LEVEL>(k.x);
  k.y = partner<LEVEL>(k.y);
  return __builtin_bit_cast(double, k);
}
// f(std::integral_constant-like level) for every level of 2^log2_lanes lanes.
template <int LEVEL>
struct Level {
  static constexpr int value = LEVEL;
};
template <typename F>
__device__ __forceinline__ void for_levels(int log2_lanes, F&& f) {
  if (log2_lanes > 0) f(Level<0>{});
  if (log2_lanes > 1) f(Level<1>{});
  if (log2_lanes > 2) f(Level<2>{});
  if (log2_lanes > 3) f(Level<3>{});
  if (log2_lanes > 4) f(Level<4>{});
  if (log2_lanes > 5) f(Level<5>{});
}
__device__ __forceinline__ float lanes_max(float v, int log2_lanes) {
  for_levels(log2_lanes, [&](auto l) { v = fmaxf(v, partner<decltype(l)::value>(v)); });
  return v;
}
__device__ __forceinline__ float lanes_sum(float v, int log2_lanes) {
  for_levels(log2_lanes, [&](auto l) { v += partner<decltype(l)::value>(v); });
  return v;
}

// Descending sort of N (a power of two) keys: Batcher's odd-even merge sort.
template <int N>
__device__ __forceinline__ void sort_keys(double* k) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q > 0; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const double a = k[i + j], b = k[i + j + q];
            k[i + j] = key_max(a, b);
            k[i + j + q] = key_min(a, b);
          }
}
// Descending sort of a bitonic sequence.
template <int N>
__device__ __forceinline__ void sort_bitonic(double* k) {
#pragma unroll
  for (int q = N / 2; q > 0; q >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & q) == 0) {
        const double a = k[i], b = k[i + q];
        k[i] = key_max(a, b);
        k[i + q] = key_min(a, b);
      }
}
// a[0 .. N) = the N largest of two descending lists, descending.
template <int N>
__device__ __forceinline__ void merge_top(double* a, const double* b) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = key_max(a[i], b[N - 1 - i]);
  sort_bitonic<N>(a);
}

struct RouteLanes {
  int log2_lanes;        // of a token
  int log2_group_lanes;  // of a group
  int vector;            // a lane's logits are whole 16-byte pieces (or one smaller piece), aligned
};

// V consecutive logits of a lane.
template <int V>
__device__ __forceinline__ void load_vector(const float* p, float (&v)[V]) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const v4f t = *reinterpret_cast<const v4f*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = t[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[i];
  }
}
template <int V>
__device__ __forceinline__ void load_vector(const uint16_t* p, float (&v)[V]) {
  if constexpr (V >= 8) {
#pragma unroll
    for (int i = 0; i < V; i += 8) {
      const v4i t = *reinterpret_cast<const v4i*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i + 2 * j] = __int_as_float(t[j] << 16);
        v[i + 2 * j + 1] = __int_as_float(t[j] & 0xffff0000);
      }
    }
  } else if constexpr (V >= 2) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const unsigned t = *reinterpret_cast<const uint32_t*>(p + i);
      v[i] = __uint_as_float(t << 16);
      v[i + 1] = __uint_as_float(t & 0xffff0000u);
    }
  } else {
    v[0] = load_logit(p);
  }
}

template <int V>
__device__ __forceinline__ void store_vector(float* p, const float (&v)[V]) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<v4f*>(p + i) = v4f{v[i], v[i + 1], v[i + 2], v[i + 3]};
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = v[i];
  }
}
template <int V>
__device__ __forceinline__ void store_vector(uint16_t* p, const float (&v)[V]) {
  if constexpr (V >= 8) {
#pragma unroll
    for (int i = 0; i < V; i += 8) {
      v4i t;
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = int(pack_bf16x2(v[i + 2 * j], v[i + 2 * j + 1]));
      *reinterpret_cast<v4i*>(p + i) = t;
    }
  } else if constexpr (V >= 2) {
#pragma unroll
    for (int i = 0; i < V; i += 2) *reinterpret_cast<uint32_t*>(p + i) = pack_bf16x2(v[i], v[i + 1]);
  } else {
    store_logit(p, v[0]);
  }
}

// 2^log2_lanes lanes per token, V experts per lane, lists of KL >= topk keys.
// The groups get equal shares of the lanes (a power of two each; lanes past
// the last group, and places past a group's end, stay empty), so a lane's
// experts are consecutive and all of one group.  Each lane sorts its own
// keys; exchanges between lanes then merge sorted lists, keeping the KL
// largest, until every lane of the token has its list of picks.
template <typename L, int V, int KL>
__global__ void __launch_bounds__(256) moe_route_kernel(const L* __restrict__ logits, int64_t ld,
                                                        const float* __restrict__ bias, RouteShape r, RouteLanes lanes,
                                                        int32_t* __restrict__ expert_idx,
                                                        float* __restrict__ weights) {
  const int n = lanes.log2_lanes;
  const int64_t thread = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t token = thread >> n;
  const bool store = token < r.T;
  const int64_t t = store ? token : r.T - 1;
  const int mine = int(thread) & ((1 << n) - 1);  // lane of the token
  const int size = r.E / r.groups, group = mine >> lanes.log2_group_lanes;
  const int place = (mine & ((1 << lanes.log2_group_lanes) - 1)) * V;  // in the group
  const int e0 = group * size + place;
  const int count = group < r.groups ? max(0, min(V, size - place)) : 0;
  const L* row = logits + t * ld;

  float l[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = 0.f;
  if (lanes.vector) {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = kNegInf;
    if (count > 0) {
      load_vector<V>(row + e0, l);
      if (bias) load_vector<V>(bias + e0, b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = i < count ? load_logit(row + e0 + i) : kNegInf;
      if (bias) b[i] = i < count ? bias[e0 + i] : 0.f;
    }
  }

  // by the logits themselves where that is the same order (scores that round to 0 are equal, and so are sigmoids that
  // round to 1)
  const bool softmax = r.score == kScoreSoftmax;
  const bool by_logit = !bias && (r.groups == 1 || r.group_score == kGroupMax);
  float top = 0.f, sum = 1.f;
  if (softmax) {
    top = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
    top = lanes_max(top, n);
  }
  if (softmax && !(by_logit && r.renormalize)) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += l[i] > kNegInf ? exp_below(l[i], top) : 0.f;
    sum = lanes_sum(sum, n);
  }
  const float inv_sum = softmax ? reciprocal(fmaxf(sum, 1.f)) : 1.f;  // the largest term is 1

  float sel[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float s = softmax ? (!by_logit                      ? exp_below(l[i], top) * inv_sum
                               : below(l[i], top) >= -104.f ? fmaxf(l[i], kLeastLogit)
                                                              : kLeastAble)
                    : by_logit ? __builtin_amdgcn_fmed3f(l[i], -104.f, kSigmoidOne)
                               : sigmoid_rank(l[i]);
    sel[i] = l[i] > kNegInf && b[i] > kNegInf ? __builtin_amdgcn_fmed3f(s + b[i], kLeastAble, kMaxFinite) : kNotAble;
  }
  if (r.groups > 1) {
    float m1 = kNotAble, m2 = kNotAble;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      m2 = __builtin_amdgcn_fmed3f(m1, m2, sel[i]);
      m1 = fmaxf(m1, sel[i]);
    }
    for_levels(lanes.log2_group_lanes, [&](auto lv) {
      const float p1 = partner<decltype(lv)::value>(m1), p2 = partner<decltype(lv)::value>(m2);
      m2 = fmaxf(fminf(m1, p1), fmaxf(m2, p2));
      m1 = fmaxf(m1, p1);
    });
    // Halves: of two masked experts (biases of FP32's lowest value) the sum itself would pass the range, and so be no
    // lower than that of one.
    const float score = r.group_score == kGroupTop2 && m1 > kNotAble ? 0.5f * m1 + (m2 > kNotAble ? 0.5f * m2 : 0.f) : m1;
    int better = 0;  // groups before this one
    const int first = (threadIdx.x & (kWave - 1)) & ~((1 << n) - 1);
    for (int g = 0; g < r.groups; ++g) {
      const float other = __shfl(score, first + (g << lanes.log2_group_lanes), kWave);
      better += other > score || (other == score && g < group);
    }
    if (better >= r.topk_groups) {
#pragma unroll
      for (int i = 0; i < V; ++i) sel[i] = kNotAble;
    }
  }

  // ---- the KL best of the token
  constexpr int W = V > KL ? V : KL;
  double k[W];
#pragma unroll
  for (int i = 0; i < W; ++i)
    k[i] = make_key(i < V ? sel[i < V ? i : 0] : kNotAble, i < V ? kRouteMaxExperts - 1 - e0 - i : 0);
  if constexpr (V <= KL) {
    sort_keys<V>(k);
  } else {
#pragma unroll
    for (int c = 0; c < V; c += KL) sort_keys<KL>(k + c);
#pragma unroll
    for (int w = KL; w < V; w *= 2)
#pragma unroll
      for (int c = 0; c < V; c += 2 * w) merge_top<KL>(k + c, k + c + w);
  }
  for_levels(n, [&](auto lv) {
    constexpr int S = (V << decltype(lv)::value) < KL ? (V << decltype(lv)::value) : KL;  // keys of the lists now
    double other[S];
#pragma unroll
    for (int i = 0; i < S; ++i) other[i] = partner<decltype(lv)::value>(k[i]);
    if constexpr (S < KL) {
#pragma unroll
      for (int i = 0; i < S; ++i) k[S + i] = other[S - 1 - i];
      sort_bitonic<2 * S>(k);
    } else {
      merge_top<KL>(k, other);
    }
  });

  // ---- weights: pick j by lane j of the token, j + lanes, ...
  auto pick_of = [&](int j) {
    double key = -__builtin_inf();
#pragma unroll
    for (int i = 0; i < KL; ++i) key = i == j ? k[i] : key;
    return j < r.topk ? key_expert(key) : -1;
  };
  float high = kNegInf, total = 1.f;
  auto score_of = [&](float x) {  // renormalised: in proportion to the score, the largest about 1
    if (softmax) return r.renormalize ? exp_below(x, high) : exp_below(x, top) * inv_sum;
    if (x >= 0.f || !r.renormalize) return sigmoid_near(x);
    return exp_below(x, fminf(high, 0.f)) * reciprocal(1.f + exp_below(x, 0.f));
  };
  auto put = [&](int j, int e, float s) {
    if (!store || j >= r.topk) return;
    expert_idx[t * r.topk + j] = e;
    weights[t * r.topk + j] = e >= 0 ? s * (r.renormalize ? reciprocal(total) : 1.f) * r.scale : 0.f;
  };
  const int step = 1 << n;
  if (r.topk <= step) {
    const int e = pick_of(mine);
    const float x = e >= 0 ? load_logit(row + e) : kNegInf;
    if (r.renormalize) high = lanes_max(x, n);
    const float s = e >= 0 ? score_of(x) : 0.f;
    if (r.renormalize) total = lanes_sum(s, n);
    put(mine, e, s);
  } else {
    auto score_at = [&](int j) {
      const int e = pick_of(j);
      return e >= 0 ? score_of(load_logit(row + e)) : 0.f;
    };
    if (r.renormalize) {
      for (int j = mine; j < r.topk; j += step) {
        const int e = pick_of(j);
        if (e >= 0) high = fmaxf(high, load_logit(row + e));
      }
      high = lanes_max(high, n);
      total = 0.f;
      for (int j = mine; j < r.topk; j += step) total += score_at(j);
      total = lanes_sum(total, n);
    }
    for (int j = mine; j < r.topk; j += step) put(j, pick_of(j), score_at(j));
  }
}

// Gradient of the logits.  With c_j the gradient of the unnormalised score of
// pick j (renormalised weights: c_j = scale * (g_j - sum of g_i s_i / S) / S,
// S the sum of the picked scores; else scale * g_j):
//   sigmoid:  dl_e = c_e s_e (1 - s_e) on the picked experts, 0 elsewhere;
//   softmax:  dl_e = s_e (c_e - sum over the picks of c_j s_j); renormalised,
//             the sum vanishes and only the picked experts have a gradient.
// In terms of the weights: dl_e = v_e * (1 - s_e) resp. v_e - s_e * sum v
// with v_j = c_j s_j = scale * w_j * (g_j - [renormalised] sum of g_i w_i),
// w the weights before the scale.
//
// 2^log2_lanes (at least topk) lanes per token, V consecutive experts per
// lane; lane j computes v_j, which then goes round the lanes.  Bound by its
// writes and by the compares of every pick with every expert where the batch
// is long: 16384 tokens of 128 experts, 8 picks (BF16) take 6.1 us with a
// softmax over all, against 3.6 for the bytes at the rate of a large copy and
// the launch, and 5.0 with a sigmoid, against 2.8.
template <typename L, int V>
__global__ void __launch_bounds__(256) moe_route_backward_kernel(const L* __restrict__ logits, int64_t ld,
                                                                 const int32_t* __restrict__ expert_idx,
                                                                 const float* __restrict__ grad_weights,
                                                                 RouteShape r, RouteLanes lanes,
                                                                 L* __restrict__ grad, int64_t grad_ld) {
  const int n = lanes.log2_lanes;
  const int64_t thread = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const bool store = (thread >> n) < r.T;
  const int64_t t = store ? thread >> n : r.T - 1;
  const int mine = int(thread) & ((1 << n) - 1);
  const int e0 = mine * V, count = max(0, min(V, r.E - e0));
  const L* row = logits + t * ld;
  const bool softmax = r.score == kScoreSoftmax, dense = softmax && !r.renormalize;

  float l[V], top = 0.f, inv_sum = 1.f;
  if (dense) {  // read first, so that the picks' loads do not hold it up
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = kNegInf;
    if (!lanes.vector) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < count) l[i] = load_logit(row + e0 + i);
    } else if (count > 0) {
      load_vector<V>(row + e0, l);
    }
  }
  int e = -1;
  float g = 0.f;
  if (mine < r.topk) {
    e = expert_idx[t * r.topk + mine];
    g = grad_weights[t * r.topk + mine];
  }
  if (e < 0 || e >= r.E) e = -1, g = 0.f;
  const float x = e >= 0 ? load_logit(row + e) : kNegInf;
  if (dense) {
    top = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
    top = lanes_max(top, n);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = l[i] > kNegInf ? exp_below(l[i], top) : 0.f;
      sum += l[i];
    }
    inv_sum = reciprocal(fmaxf(lanes_sum(sum, n), 1.f));  // the largest term is 1
  }

  float w = 0.f;
  if (r.renormalize) {
    const float high = lanes_max(x, n);
    if (e >= 0) {
      if (softmax) w = exp_below(x, high);
      else w = x >= 0.f ? sigmoid_near(x) : exp_below(x, fminf(high, 0.f)) * reciprocal(1.f + exp_below(x, 0.f));
    }
    w *= reciprocal(fmaxf(lanes_sum(w, n), 0.5f));  // the largest term is 1/2 or more
  } else if (e >= 0) {
    w = softmax ? exp_below(x, top) * inv_sum : sigmoid_near(x);
  }
  float v = w * g;
  if (r.renormalize) v = w * (g - lanes_sum(v, n));
  const float mean = dense ? r.scale * inv_sum * lanes_sum(v, n) : 0.f;
  if (!softmax && e >= 0) v *= sigmoid_near(-x);
  v *= r.scale;

  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = dense ? -l[i] * mean : 0.f;
  const int first = (threadIdx.x & (kWave - 1)) & ~((1 << n) - 1);
  for (int j = 0; j < r.topk; ++j) {
    const int at = __shfl(e, first + j, kWave) - e0;
    const float add = __shfl(v, first + j, kWave);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] += at == i ? add : 0.f;
  }
  if (!store) return;
  L* out = grad + t * grad_ld + e0;
  if (lanes.vector) {
    if (count > 0) store_vector<V>(out, d);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < count) store_logit(out + i, d[i]);
  }
}

}  // namespace fp8g
