// A mixture-of-experts layer for a few tokens, in two kernels, for gfx950.
//
//   mid[p] = act(G_e x_t) * (U_e x_t)              p = t topk + j, e = expert_idx[p]
//   out[t] = bf16( sum over j of weights[p] D_e mid[p] )
// G_e, U_e: the first and the last `inter` rows of the expert's first matrix
// [2 inter][hidden], D_e its second [hidden][inter], FP8 E4M3 codes with an
// FP32 scale per 128 x 128 block, as the grouped GEMMs take them; x BF16.
//
// Both kernels stream matrices through the same code: blocks of up to 32 rows
// by 128 columns, with the 128 activations of up to 16 tokens, come by direct
// copies to a ring that every wave has for itself in LDS, several blocks ahead
// and across units (a unit is some rows of one expert's matrix), so that the
// matrices arrive without a pause.  The waves share the columns and meet where
// their partial sums are added, in the order of the waves.
//
// Codes become operands of the matrix instructions exactly.  The first kernel's
// are BF16, as x is, times 2^-16: then no sum of a block's 128 products passes
// FP32's range where its scaled value does not.  The second's are FP16: mid is
// kept as FP16 values with an exponent for each 16 of a pair's columns, which
// the first kernel finds where it forms them.  So mid is off by 2^-12 of its
// value (2^-24 of the largest of 128 neighbours where that is more), an eighth
// of what BF16 would cost in the same bytes: with BF16 the outputs' error was
// 1.41 times that of their own rounding, with this it is 1.01.  The block's
// scale and the largest exponent go onto the FP32 sum.
//
// What bounds it: the matrices are read once, a byte a weight.
#pragma once

#include "activation.hpp"
#include "gemm_kernel.hpp"  // the operand tiles' layout

namespace fp8g {

constexpr int kFewTokens = 64;  // of a launch, at most
constexpr int kFewMaxPairs = 1024;
constexpr int kFewMaxTopk = 32;
constexpr int kFewGroup = 16;  // columns of mid that share an exponent

struct MoeFewArgs {
  const uint16_t* x;
  int64_t x_ld;
  const int32_t* expert_idx;
  const float* weights;
  const uint8_t *up, *down;
  const float *up_scales, *down_scales;
  uint16_t* mid;      // [pairs][inter] FP16
  int8_t* exponents;  // [pairs][inter / 16]
  uint16_t* out;
  int tokens, topk, experts, hidden, inter, activation;
};

typedef __bf16 v8bf16_t __attribute__((ext_vector_type(8)));
typedef _Float16 v8f16_t __attribute__((ext_vector_type(8)));
typedef int v2i_t __attribute__((ext_vector_type(2)));

// Eight E4M3 codes (two dwords) -> eight BF16 values times 2^-16, or FP16 values; exact.
template <bool F16>
__device__ __forceinline__ v4i few_decode(int lo, int hi) {
  v4i f;
  if constexpr (F16) {
    f[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(unsigned(lo), 1.f, false));
    f[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(unsigned(lo), 1.f, true));
    f[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(unsigned(hi), 1.f, false));
    f[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(unsigned(hi), 1.f, true));
  } else {
    constexpr float s = 1.f / 65536.f;
    f[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(lo), s, false));
    f[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(lo), s, true));
    f[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(hi), s, false));
    f[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(hi), s, true));
  }
  return f;
}

// Workgroup barrier after this wave's LDS accesses; copies to LDS stay in flight.
__device__ __forceinline__ void few_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int N>
__device__ __forceinline__ void few_copies_left() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// As copy16_to_lds, every lane from an address of its own.
__device__ __forceinline__ void few_copy16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               ::"s"(uniform(int(lds))), "v"(src) : "memory");
}
__device__ __forceinline__ void few_copy4(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               ::"s"(uniform(int(lds))), "v"(src) : "memory");
}

// ---- which expert has which tokens ----------------------------------------------
// Pairs whose index is no expert's are in no plan.
//
// For up to TX tokens: a tile is one expert, in the order of the first pairs,
// and its column t is token t.  pair[tile][t]: the pair, or kFewNone where the
// token has not picked the expert.  A token that names an expert twice has the
// first of those pairs there, with the sum of their weights.
constexpr unsigned kFewNone = 0xffff;
template <int TX>
struct FewTokenPlan {
  static constexpr int kPairs = TX * kFewMaxTopk;
  uint16_t pair[kPairs][TX];
  uint16_t expert[kPairs];
  float weight[kPairs];
  int tiles;
};

// For any number of tokens: tiles of up to TX pairs of one expert, which follow
// one another; tiles in the order of their first pairs.
template <int TX>
struct FewPairPlan {
  static constexpr int kPairs = kFewMaxPairs;
  uint16_t pair[kPairs];       // by tile, in a tile in order
  uint16_t start[kPairs + 1];  // tile t's pairs are pair[start[t]] .. pair[start[t + 1] - 1]
  uint16_t expert[kPairs];
  int tiles;
};

constexpr int kFewMaxWaves = 8;
template <int PAIRS>
struct FewPlanScratch {
  __attribute__((aligned(16))) int expert[PAIRS];
  int count[PAIRS];
  int sums[kFewMaxWaves];
};

// The pairs' experts (-1: none), and four more.
template <int PAIRS>
__device__ __forceinline__ void few_load_experts(const MoeFewArgs& a, int pairs, FewPlanScratch<PAIRS>& s) {
  const int padded = (pairs + 3) & ~3;
  for (int p = threadIdx.x; p < padded; p += blockDim.x) {
    const int e = p < pairs ? a.expert_idx[p] : -1;
    s.expert[p] = e >= 0 && e < a.experts ? e : -1;
    s.count[p] = 0;
  }
}

// f(q, same) for the pairs q before p, and some after it in the same wave: whether q's expert is `mine`.
template <int PAIRS, typename F>
__device__ __forceinline__ void few_pairs_before(const FewPlanScratch<PAIRS>& s, int p, int mine, int pairs, F&& f) {
  const int end = min(pairs, uniform(p) + kWave);  // the wave's last pair
  for (int q0 = 0; q0 < end; q0 += 4) {
    const v4i e = *reinterpret_cast<const v4i*>(s.expert + q0);
#pragma unroll
    for (int i = 0; i < 4; ++i) f(q0 + i, e[i] == mine && q0 + i < p);
  }
}

template <int TX, int WAVES>
__device__ __forceinline__ void few_plan(const MoeFewArgs& a, FewTokenPlan<TX>& plan,
                                         FewPlanScratch<FewTokenPlan<TX>::kPairs>& s) {
  constexpr int THREADS = WAVES * kWave, ROUNDS = (FewTokenPlan<TX>::kPairs + THREADS - 1) / THREADS;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid >> 6), pairs = a.tokens * a.topk;
  for (int p = tid; p < pairs; p += THREADS) plan.weight[p] = a.weights ? a.weights[p] : 1.f;
  few_load_experts(a, pairs, s);
  for (int i = tid; i < pairs * (TX / 2); i += THREADS) reinterpret_cast<uint32_t*>(plan.pair)[i] = ~0u;
  __syncthreads();
  int head[ROUNDS], mine[ROUNDS], tiles = 0;
  float sum[ROUNDS];
  bool again[ROUNDS];
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    const int p = j * THREADS + tid;
    head[j] = p, mine[j] = -1, again[j] = false, sum[j] = 0.f;
    if (j * THREADS >= pairs) continue;
    mine[j] = p < pairs ? s.expert[p] : -1;
    const int token = p / a.topk, from = token * a.topk;
    few_pairs_before(s, p, mine[j], pairs, [&](int q, bool same) {
      head[j] = same && head[j] == p ? q : head[j];
      again[j] |= same && q >= from;
    });
    if (mine[j] >= 0 && !again[j]) {
      sum[j] = plan.weight[p];
      for (int q = p + 1; q < from + a.topk; ++q) sum[j] += s.expert[q] == mine[j] ? plan.weight[q] : 0.f;
    }
    // the tile of a pair that begins one: how many begin before
    const uint64_t first = __ballot(mine[j] >= 0 && head[j] == p);
    if (lane == 0) s.sums[wave] = __popcll(first);
    __syncthreads();
    int at = tiles + __popcll(first & ((uint64_t(1) << lane) - 1));
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      at += w < wave ? s.sums[w] : 0;
      tiles += s.sums[w];
    }
    if (mine[j] >= 0 && head[j] == p) {
      s.count[p] = at;
      plan.expert[at] = uint16_t(mine[j]);
    }
    __syncthreads();
  }
  if (tid == 0) plan.tiles = tiles;
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    const int p = j * THREADS + tid;
    if (mine[j] < 0 || again[j]) continue;
    plan.pair[s.count[head[j]]][p / a.topk] = uint16_t(p);
    plan.weight[p] = sum[j];
  }
  __syncthreads();
}

// Every pair finds its rank among its expert's and the pair that begins its
// tile; a scan over the tiles' first pairs then places the tiles.
template <int TX, int WAVES>
__device__ __forceinline__ void few_plan(const MoeFewArgs& a, FewPairPlan<TX>& plan,
                                         FewPlanScratch<FewPairPlan<TX>::kPairs>& s) {
  constexpr int THREADS = WAVES * kWave, ROUNDS = (FewPairPlan<TX>::kPairs + THREADS - 1) / THREADS;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid >> 6), pairs = a.tokens * a.topk;
  few_load_experts(a, pairs, s);
  __syncthreads();
  int rank[ROUNDS], head[ROUNDS], mine[ROUNDS];
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    const int p = j * THREADS + tid;
    rank[j] = 0, head[j] = p, mine[j] = -1;
    if (j * THREADS >= pairs) continue;
    mine[j] = p < pairs ? s.expert[p] : -1;
    few_pairs_before(s, p, mine[j], pairs, [&](int q, bool same) {
      head[j] = same && rank[j] % TX == 0 ? q : head[j];
      rank[j] += same;
    });
    if (rank[j] % TX == 0) head[j] = p;
    if (mine[j] >= 0) atomicAdd(&s.count[head[j]], 1);
  }
  __syncthreads();
  int before = 0;  // tiles << 16 | pairs of the rounds before
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    const int p = j * THREADS + tid;
    if (j * THREADS >= pairs) continue;
    const bool first = mine[j] >= 0 && head[j] == p;
    const int own = first ? 1 << 16 | s.count[p] : 0;
    int upto = own;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const int v = __shfl_up(upto, d, kWave);
      upto += lane >= d ? v : 0;
    }
    if (lane == kWave - 1) s.sums[wave] = upto;
    __syncthreads();
    int at = before + upto - own;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      at += w < wave ? s.sums[w] : 0;
      before += s.sums[w];
    }
    if (first) {
      plan.start[at >> 16] = uint16_t(at & 0xffff);
      plan.expert[at >> 16] = uint16_t(mine[j]);
      s.count[p] = at & 0xffff;
    }
    __syncthreads();
  }
  if (tid == 0) {
    plan.tiles = before >> 16;
    plan.start[before >> 16] = uint16_t(before & 0xffff);
  }
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j)
    if (mine[j] >= 0) plan.pair[s.count[head[j]] + rank[j] % TX] = uint16_t(j * THREADS + tid);
  __syncthreads();
}

// What the kernels ask a plan: the row of x or mid of column t of a tile (of a
// column without a pair: some other's), and its pair (kFewNone: none).
template <int TX>
__device__ __forceinline__ unsigned few_pair(const FewTokenPlan<TX>& p, int tile, int t) { return p.pair[tile][t]; }
template <int TX>
__device__ __forceinline__ unsigned few_pair(const FewPairPlan<TX>& p, int tile, int t) {
  const int at = p.start[tile] + t;
  return at < p.start[tile + 1] ? p.pair[at] : kFewNone;
}
template <int TX>
__device__ __forceinline__ const uint16_t* few_x(const MoeFewArgs& a, const FewTokenPlan<TX>&, int, int t) {
  return a.x + min(t, a.tokens - 1) * a.x_ld;
}
template <int TX>
__device__ __forceinline__ const uint16_t* few_x(const MoeFewArgs& a, const FewPairPlan<TX>& p, int tile, int t) {
  return a.x + p.pair[min(p.start[tile] + t, p.start[tile + 1] - 1)] / a.topk * a.x_ld;
}

// ---- the stream ------------------------------------------------------------------
// A block in LDS: 16 R rows of 128 codes (operand tiles, laid out as tile_byte
// says); TX rows of 128 activations (16-byte unit u of token t at u ^ (t & 15));
// 256 bytes more: the R row sets' scales in turn, or (MID) the tokens' eight
// exponents, and from byte 128 on the scale.
template <int TX, int R, int WAVES, int LDS_BYTES, bool MID>
struct FewRing {
  static constexpr int kX = R * 2048, kMore = kX + TX * 256, kSlot = kMore + 256;
  static constexpr int kXCopies = TX * 256 / 1024, kCopies = 2 * R + kXCopies + 1;
  static constexpr int kFit = LDS_BYTES / (WAVES * kSlot), kBlocks = kFit > 6 ? 6 : kFit;
  static constexpr int kWaveBytes = kBlocks * kSlot, kBytes = WAVES * kWaveBytes;
  static_assert(kBlocks >= 2 && (kBlocks - 1) * kCopies < 64, "LDS and vmcnt");
};

// Where a unit's data lies.
template <int R>
struct FewSource {
  const uint8_t* codes[R];  // 16 rows each
  const void* more;         // of this lane: the scales of the row set's blocks, or the exponents of its token
};

// A block as it comes out of the stream: the sums of its products before the scale, and what that is.
template <int R>
struct FewBlock {
  v4f part[R];      // of token `lane & 15` and rows 4 (lane >> 4) ..
  float scale[R];
  int exponent;     // MID: the token's
};

template <typename L, int TX, int R, int WAVES, bool MID>
struct FewStream {
  const char* ring;
  uint32_t ring_at;
  int lane, groups, g, g_restart, g_step, unit, total, issued = 0, taken = 0, issue_slot = 0, read_slot = 0;
  FewSource<R> src;
  const uint16_t* xsrc[L::kXCopies];
  unsigned row_off[2];

  // `source(unit)`: the data of a unit; `x_row(unit, t)`: its t-th token's activations.
  template <typename S, typename X>
  __device__ __forceinline__ void begin_unit(S&& source, X&& x_row) {
    src = source(unit);
#pragma unroll
    for (int c = 0; c < L::kXCopies; ++c) {
      const int t = (c * 64 + lane) / 16;
      xsrc[c] = x_row(unit, t) + (((lane & 15) ^ t) & 15) * 8;
    }
  }
  // Blocks of this wave: `total` of them, from block g_ of unit `unit_` on every step-th, in further units from block
  // `restart` on.
  template <typename S, typename X>
  __device__ __forceinline__ void start(char* lds, int k, int unit_, int g_, int restart, int step, int total_,
                                        S&& source, X&& x_row) {
    const int wave = uniform(threadIdx.x >> 6);
    lane = threadIdx.x & (kWave - 1);
    ring = lds + wave * L::kWaveBytes;
    ring_at = lds_addr(lds) + wave * L::kWaveBytes;
    groups = k / kGroupK;
    unit = unit_, g = g_, g_restart = restart, g_step = step, total = total_;
#pragma unroll
    for (int h = 0; h < 2; ++h) row_off[h] = unsigned(tile_row(h, lane)) * unsigned(k) + 16u * tile_chunk(h, lane);
    if (total > 0) begin_unit(source, x_row);
    for (int i = 0; i < L::kBlocks && i < total; ++i) copy_next(source, x_row);
  }
  template <typename S, typename X>
  __device__ __forceinline__ void copy_next(S&& source, X&& x_row) {
    const uint32_t at = ring_at + unsigned(issue_slot) * L::kSlot;
#pragma unroll
    for (int s = 0; s < R; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        copy16_to_lds(src.codes[s] + g * kGroupK, row_off[h], at + s * 2048 + h * 1024);
#pragma unroll
    for (int c = 0; c < L::kXCopies; ++c) few_copy16(xsrc[c] + g * kGroupK, at + L::kX + c * 1024);
    const int step = MID && lane < 32 ? kGroupK / kFewGroup : 4;
    few_copy4(static_cast<const char*>(src.more) + g * step, at + L::kMore);
    issue_slot = issue_slot + 1 == L::kBlocks ? 0 : issue_slot + 1;
    g += g_step;
    if (++issued < total && g >= groups) {
      g = g_restart;
      ++unit;
      begin_unit(source, x_row);
    }
  }
  template <int N = L::kBlocks - 1>
  __device__ __forceinline__ void wait(int newer) {
    if (N == 0 || newer >= N) few_copies_left<N * L::kCopies>();
    else if constexpr (N > 0) wait<N - 1>(newer);
  }
  template <typename S, typename X>
  __device__ __forceinline__ FewBlock<R> next(S&& source, X&& x_row) {
    wait(min(total - 1 - taken, L::kBlocks - 1));  // blocks in flight after this one
    ++taken;
    const char* at = ring + read_slot * L::kSlot;
    read_slot = read_slot + 1 == L::kBlocks ? 0 : read_slot + 1;
    const int lr = lane & 15, q = lane >> 4, t = lr & (TX - 1);
    v4i codes[R][2], x[4];
#pragma unroll
    for (int s = 0; s < R; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        codes[s][h] = *reinterpret_cast<const v4i*>(at + s * 2048 + tile_byte(lr, 2 * q + h));
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const v4i*>(at + L::kX + t * 256 + ((4 * q + j) ^ t) * 16);
    FewBlock<R> b;
    v2i_t exponents = {0, 0};
    if constexpr (MID) {
      const float scale = *reinterpret_cast<const float*>(at + L::kMore + 128);
#pragma unroll
      for (int s = 0; s < R; ++s) b.scale[s] = scale;
      exponents = *reinterpret_cast<const v2i_t*>(at + L::kMore + t * 8);
    } else {
#pragma unroll
      for (int s = 0; s < R; ++s) b.scale[s] = *reinterpret_cast<const float*>(at + L::kMore + 4 * s) * 65536.f;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the block has been read
    if (issued < total) copy_next(source, x_row);
    b.exponent = 0;
    if constexpr (MID) {
      // The lane's activations, 32 columns from 32 q on, are of the groups 2 q and 2 q + 1: brought to the token's
      // largest exponent.  (Under 2^-14 of it: 0.)
      int top = -128, own[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, int(exponents[i / 4] << (24 - 8 * (i & 3))) >> 24);
      const int word = q & 2 ? exponents[1] : exponents[0], half = q & 1 ? word >> 16 : word;
      own[0] = int(unsigned(half) << 24) >> 24, own[1] = int(unsigned(half) << 16) >> 24;
      b.exponent = top;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = own[j / 2] - top;
        const uint16_t by = d < -14 ? 0 : uint16_t((d + 15) << 10);  // 2^d
        x[j] = __builtin_bit_cast(v4i, __builtin_bit_cast(v8f16_t, x[j]) * __builtin_bit_cast(_Float16, by));
      }
    }
#pragma unroll
    for (int s = 0; s < R; ++s) b.part[s] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < R; ++s) {
        const v4i w = few_decode<MID>(codes[s][j / 2][2 * (j & 1)], codes[s][j / 2][2 * (j & 1) + 1]);
        if constexpr (MID)
          b.part[s] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8f16_t, w),
                                                             __builtin_bit_cast(v8f16_t, x[j]), b.part[s], 0, 0, 0);
        else
          b.part[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf16_t, w),
                                                              __builtin_bit_cast(v8bf16_t, x[j]), b.part[s], 0, 0, 0);
      }
    return b;
  }
};

// The waves' sums of 16 R rows: [wave][token][rows], 16-byte piece c of token t at c ^ (t & (4 R - 1)).
template <int TX, int R, int WAVES>
struct FewSums {
  float v[WAVES][TX][16 * R];
  __device__ __forceinline__ void put(const v4f (&acc)[R]) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6, t = lane & 15, q = lane >> 4;
    if (t >= TX) return;
#pragma unroll
    for (int s = 0; s < R; ++s)
      *reinterpret_cast<v4f*>(&v[wave][t][((4 * s + q) ^ (t & (4 * R - 1))) * 4]) = acc[s];
  }
  __device__ __forceinline__ float get(int t, int row) const {
    const int at = ((row >> 2) ^ (t & (4 * R - 1))) * 4 + (row & 3);
    float sum = v[0][t][at];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += v[w][t][at];
    return sum;
  }
};

// ---- first kernel ------------------------------------------------------------------
// A unit is 16 rows of G and the 16 of U of one tile; a workgroup takes a run of
// units, its waves every fourth block of each.  Grid: any number of workgroups.
constexpr int kFewUpWaves = 4;
template <int TX, typename Plan>
struct FewUp {
  static constexpr int kLds = 160 * 1024 - int(sizeof(Plan) + sizeof(FewSums<TX, 2, kFewUpWaves>)) - 256;
  // Two workgroups fit a CU with a few tokens (their waits then overlap), one with more.
  using Ring = FewRing<TX, 2, kFewUpWaves, (TX == 4 ? 64 * 1024 : kLds), false>;
  __attribute__((aligned(1024))) char ring[Ring::kBytes];
  FewSums<TX, 2, kFewUpWaves> sums;
  Plan plan;
  static_assert(sizeof(FewPlanScratch<Plan::kPairs>) <= Ring::kBytes, "the plan's scratch takes the ring's place");
};

template <int TX, typename Plan>
__global__ void __launch_bounds__(kFewUpWaves* kWave) moe_few_up_kernel(const MoeFewArgs a) {
  using Lds = FewUp<TX, Plan>;
  __shared__ Lds lds;
  const Plan& plan = lds.plan;
  few_plan<TX, kFewUpWaves>(a, lds.plan, *reinterpret_cast<FewPlanScratch<Plan::kPairs>*>(lds.ring));
  const int sets = a.inter / kFewGroup, kg = a.hidden / kGroupK, tid = threadIdx.x, wave = uniform(tid >> 6);
  const int64_t units = int64_t(uniform(plan.tiles)) * sets;
  const int u0 = int(units * blockIdx.x / gridDim.x), u1 = int(units * (blockIdx.x + 1) / gridDim.x);
  if (u0 == u1) return;
  auto source = [&](int u) {
    const int e = uniform(plan.expert[u / sets]), row = u % sets * kFewGroup;
    FewSource<2> s;
    s.codes[0] = a.up + (int64_t(e) * 2 * a.inter + row) * a.hidden;
    s.codes[1] = s.codes[0] + int64_t(a.inter) * a.hidden;
    s.more = a.up_scales + (int64_t(e) * 2 * (a.inter / kGroupK) + row / kGroupK +
                            ((tid & 1) ? a.inter / kGroupK : 0)) * kg;
    return s;
  };
  auto x_row = [&](int u, int t) { return few_x(a, plan, u / sets, t); };
  FewStream<typename Lds::Ring, TX, 2, kFewUpWaves, false> stream;
  const int blocks = (kg - wave + kFewUpWaves - 1) / kFewUpWaves;
  stream.start(lds.ring, a.hidden, u0, wave, wave, kFewUpWaves, (u1 - u0) * blocks, source, x_row);
  for (int u = u0; u < u1; ++u) {
    v4f acc[2] = {};
    for (int i = 0; i < blocks; ++i) {
      const FewBlock<2> b = stream.next(source, x_row);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[s][r] = fmaf(b.scale[s], b.part[s][r], acc[s][r]);
    }
    few_barrier();  // the sums of the unit before are read
    lds.sums.put(acc);
    few_barrier();
    const int tile = u / sets, set = u % sets, row = tid & 15, t = tid >> 4;
    const unsigned p = t < TX ? few_pair(plan, tile, t) : kFewNone;
    if (p == kFewNone) continue;  // (16 lanes together)
    const float v = activate(a.activation, lds.sums.get(t, row)) * lds.sums.get(t, 16 + row);
    // FP16 with the exponent that takes the largest of the 16 to 2^14 .. 2^15; with an infinity or a NaN the largest
    // exponent, which leaves it what it is.
    float top = fabsf(v);
#pragma unroll
    for (int d = 1; d < 16; d *= 2) {
      const float o = __shfl_xor(top, d, 16);
      top = o > top || o != o ? o : top;
    }
    const int e = top < __builtin_inff() ? max(-128, (top > 0.f ? ilogbf(top) : -128) - 14) : 113;
    const _Float16 h = _Float16(ldexpf(v, -e));
    a.mid[int64_t(p) * a.inter + set * kFewGroup + row] = __builtin_bit_cast(uint16_t, h);
    if (row == 0) a.exponents[int64_t(p) * sets + set] = int8_t(e);
  }
}

// ---- second kernel, any number of tokens -------------------------------------------
// A workgroup has 32 rows of the output, of all tokens, in LDS and takes the tiles
// one after the other, its waves every fourth block of each.  Grid: hidden / 32.
template <int TX>
struct FewDownPairs {
  static constexpr int kWaves = 4;
  using Plan = FewPairPlan<TX>;
  using Ring = FewRing<TX, 2, kWaves, 132 * 1024, true>;
  __attribute__((aligned(1024))) char ring[Ring::kBytes];
  FewSums<TX, 2, kWaves> sums;
  float out[kFewTokens][32];
  float weight[kFewMaxPairs];
  Plan plan;
};

template <int TX>
__global__ void __launch_bounds__(FewDownPairs<TX>::kWaves* kWave) moe_few_down_pairs_kernel(const MoeFewArgs a) {
  using Lds = FewDownPairs<TX>;
  constexpr int kWaves = Lds::kWaves, kThreads = kWaves * kWave, kRows = 32;
  __shared__ Lds lds;
  const auto& plan = lds.plan;
  const int tid = threadIdx.x, wave = uniform(tid >> 6), row0 = blockIdx.x * kRows, kg = a.inter / kGroupK;
  for (int p = tid; p < a.tokens * a.topk; p += kThreads) lds.weight[p] = a.weights ? a.weights[p] : 1.f;
  for (int o = tid; o < a.tokens * kRows; o += kThreads) lds.out[o / kRows][o % kRows] = 0.f;
  few_plan<TX, kWaves>(a, lds.plan, *reinterpret_cast<FewPlanScratch<kFewMaxPairs>*>(lds.ring));
  const int tiles = uniform(plan.tiles);
  const auto row_pair = [&](int u, int t) { return plan.pair[min(plan.start[u] + t, plan.start[u + 1] - 1)]; };
  auto source = [&](int u) {
    const int e = uniform(plan.expert[u]), lane = tid & (kWave - 1);
    FewSource<2> s;
    s.codes[0] = a.down + (int64_t(e) * a.hidden + row0) * a.inter;
    s.codes[1] = s.codes[0] + int64_t(16) * a.inter;
    const float* scales = a.down_scales + (int64_t(e) * (a.hidden / kGroupK) + row0 / kGroupK) * kg;
    s.more = lane < 32 ? static_cast<const void*>(a.exponents + int64_t(row_pair(u, lane >> 1 & (TX - 1))) *
                                                                    (a.inter / kFewGroup) + 4 * (lane & 1))
                       : scales;
    return s;
  };
  auto x_row = [&](int u, int t) { return a.mid + int64_t(row_pair(u, t)) * a.inter; };
  FewStream<typename Lds::Ring, TX, 2, kWaves, true> stream;
  const int blocks = (kg - wave + kWaves - 1) / kWaves;
  stream.start(lds.ring, a.inter, 0, wave, wave, kWaves, tiles * blocks, source, x_row);
  for (int u = 0; u < tiles; ++u) {
    v4f acc[2] = {};
    for (int i = 0; i < blocks; ++i) {
      const FewBlock<2> b = stream.next(source, x_row);
      const float scale = ldexpf(b.scale[0], b.exponent);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[s][r] = fmaf(scale, b.part[s][r], acc[s][r]);
    }
    few_barrier();  // the sums of the unit before are read
    lds.sums.put(acc);
    few_barrier();
    const int first = plan.start[u], count = plan.start[u + 1] - first;
    for (int o = tid; o < count * kRows; o += kThreads) {
      const int row = o % kRows;
      int t = o / kRows;
      const int token = plan.pair[first + t] / a.topk;
      // pairs of one token (an expert picked twice) follow one another; the first one's thread adds them all
      if (t > 0 && plan.pair[first + t - 1] / a.topk == token) continue;
      float sum = lds.out[token][row];
      for (; t < count && plan.pair[first + t] / a.topk == token; ++t)
        sum = fmaf(lds.weight[plan.pair[first + t]], lds.sums.get(t, row), sum);
      lds.out[token][row] = sum;
    }
  }
  __syncthreads();
  for (int o = tid; o < a.tokens * (kRows / 2); o += kThreads) {
    const int t = o / (kRows / 2), c = 2 * (o % (kRows / 2));
    *reinterpret_cast<uint32_t*>(a.out + int64_t(t) * a.hidden + row0 + c) =
        pack_bf16x2(lds.out[t][c], lds.out[t][c + 1]);
  }
}

// ---- second kernel, up to TX tokens ------------------------------------------------
// A lane's column is a token, so its sums over all experts, weighted, stay in
// its registers.  A workgroup has 16 R rows of the output; its waves take equal
// runs of the experts' blocks and meet once, at the end.  Grid: hidden / (16 R).
constexpr int kFewDownWaves = 8;
template <int TX, int R>
struct FewDownTokens {
  static constexpr int kWaves = kFewDownWaves;
  using Plan = FewTokenPlan<TX>;
  using Ring = FewRing<TX, R, kWaves, 160 * 1024 - int(sizeof(Plan)) - 1024, true>;
  __attribute__((aligned(1024))) char ring[Ring::kBytes];
  Plan plan;
  static_assert(sizeof(FewSums<TX, R, kWaves>) <= Ring::kBytes, "the sums take the ring's place");
  static_assert(sizeof(FewPlanScratch<Plan::kPairs>) <= Ring::kBytes, "the plan's scratch takes the ring's place");
};

template <int TX, int R>
__global__ void __launch_bounds__(kFewDownWaves* kWave) moe_few_down_kernel(const MoeFewArgs a) {
  using Lds = FewDownTokens<TX, R>;
  constexpr int kWaves = Lds::kWaves, kRows = 16 * R;
  __shared__ Lds lds;
  const auto& plan = lds.plan;
  few_plan<TX, kWaves>(a, lds.plan, *reinterpret_cast<FewPlanScratch<Lds::Plan::kPairs>*>(lds.ring));
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid >> 6);
  const int row0 = blockIdx.x * kRows, kg = a.inter / kGroupK, sets = a.inter / kFewGroup;
  const int all = uniform(plan.tiles) * kg;  // (at most 512 experts' 512 blocks)
  const int f0 = all * wave / kWaves, f1 = all * (wave + 1) / kWaves;
  // a column without a pair: the tile's first one's (there is one)
  auto row_pair = [&](int u, int t) {
    unsigned p = plan.pair[u][t];
    for (int i = 0; p == kFewNone; ++i) p = plan.pair[u][i];
    return p;
  };
  auto source = [&](int u) {
    const int e = uniform(plan.expert[u]);
    FewSource<R> s;
#pragma unroll
    for (int r = 0; r < R; ++r) s.codes[r] = a.down + (int64_t(e) * a.hidden + row0 + 16 * r) * a.inter;
    const float* scales = a.down_scales + (int64_t(e) * (a.hidden / kGroupK) + row0 / kGroupK) * kg;
    s.more = lane < 32 ? static_cast<const void*>(a.exponents + int64_t(row_pair(u, lane >> 1 & (TX - 1))) * sets +
                                                  4 * (lane & 1))
                       : scales;
    return s;
  };
  auto x_row = [&](int u, int t) { return a.mid + int64_t(row_pair(u, t)) * a.inter; };
  FewStream<typename Lds::Ring, TX, R, kWaves, true> stream;
  stream.start(lds.ring, a.inter, f0 / kg, f0 % kg, 0, 1, f1 - f0, source, x_row);
  v4f acc[R] = {};
  int unit = -1;
  bool live = false;
  float weight = 0.f;
  for (int f = f0; f < f1; ++f) {
    if (f / kg != unit) {
      unit = f / kg;
      const unsigned p = plan.pair[unit][lane & (TX - 1)];
      live = p != kFewNone;
      weight = live ? plan.weight[p] : 0.f;
    }
    const FewBlock<R> b = stream.next(source, x_row);
    const float scale = weight * ldexpf(b.scale[0], b.exponent);
#pragma unroll
    for (int s = 0; s < R; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[s][r] = live ? fmaf(scale, b.part[s][r], acc[s][r]) : acc[s][r];
  }
  auto& sums = *reinterpret_cast<FewSums<TX, R, kWaves>*>(lds.ring);
  __syncthreads();  // every wave is done with its ring
  sums.put(acc);
  __syncthreads();
  for (int o = tid; o < a.tokens * (kRows / 2); o += kWaves * kWave) {
    const int t = o / (kRows / 2), c = 2 * (o % (kRows / 2));
    *reinterpret_cast<uint32_t*>(a.out + int64_t(t) * a.hidden + row0 + c) =
        pack_bf16x2(sums.get(t, c), sums.get(t, c + 1));
  }
}

}  // namespace fp8g
