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
// the first kernel finds where it forms them, and brought to the largest exponent
// of a block where it is read.  So mid is off by 2^-11 of its value, an eighth of
// what BF16 would cost in the same bytes, and by 2^-37 of the largest of 128
// neighbours where that is more: a single large channel, as gated feed-forward
// networks have them, leaves its neighbours as they are even where the second
// matrix has nothing for it.  With BF16 the outputs' error was 1.41 times that of
// their own rounding, with this it is 1.01.  The block's scale and the largest
// exponent go onto the FP32 sum.
//
// What bounds it: the matrices are read once, a byte a weight.  64 tokens, 128
// experts of 7168 x 2048: 626 us for the first kernel (6.0 TB/s) and 278 for the
// second (6.8); 7 tokens, 16 of 4096 x 2048: 37 and 20.  One token, 8 experts of
// 2048 x 768: 8.4 and 7.0, of which a launch and the chain of loads up to the
// first block (the indices, then what they name) are 2.8 and 3.6.
#pragma once

#include <type_traits>

#include "activation.hpp"
#include "gemm_kernel.hpp"  // the operand tiles' layout

namespace fp8g {

constexpr int kFewTokens = 64;  // of a launch, at most
constexpr int kFewMaxPairs = 512;
constexpr int kFewMaxTopk = 32;
constexpr int kFewMaxExperts = 4096;  // a table of them takes the rings' place in LDS
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
  float* partial;     // [slices][tokens][hidden], where the second kernel has slices
  unsigned long long* counters;  // arrivals, one for each workgroup of a slice
  uint16_t* out;
  unsigned tag;  // of the counters
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

// 2^d for d <= 0 as FP16: below 2^-14 one of its subnormal numbers, below 2^-24 0.
__device__ __forceinline__ _Float16 few_power(int d) {
  const int bits = d >= -14 ? (d + 15) << 10 : d >= -24 ? 1 << (d + 24) : 0;
  return __builtin_bit_cast(_Float16, uint16_t(bits));
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
// A pair whose index is no expert's is in no plan, and of a token's pairs with
// one expert only the first, which has the sum of their weights.
//
// For up to TX tokens: a tile is one expert, in the order of the first pairs,
// and its column t is token t.  pair[tile][t]: the pair, or kFewNone where the
// token has not picked the expert.
constexpr unsigned kFewNone = 0xffff;
template <int TX>
struct FewTokenPlan {
  static constexpr int kPairs = TX * kFewMaxTopk;
  uint16_t pair[kPairs][TX];
  uint16_t expert[kPairs];
  float weight[kPairs];
  int tiles;
};

// For any number of tokens: a tile is up to TX pairs of one expert; an expert's
// tiles follow one another, the experts in the order of their first pairs, and
// an expert's pairs go to its tiles in order.  (Which column of its tile a pair
// has may change from run to run; nothing that is computed depends on it.)
template <int TX>
struct FewPairPlan {
  static constexpr int kPairs = kFewMaxPairs;
  uint16_t pair[kPairs];       // by tile
  uint16_t start[kPairs + 1];  // tile t's pairs are pair[start[t]] .. pair[start[t + 1] - 1]
  uint16_t expert[kPairs];
  uint16_t first[kPairs], number[kPairs];  // the first of its expert's tiles, and how many there are
  uint16_t token[kPairs];                  // of a pair
  float weight[kPairs];
  int tiles;
};

constexpr int kFewMaxWaves = 8;
template <int PAIRS>
struct FewPlanScratch {
  __attribute__((aligned(16))) int first[kFewMaxExperts];  // an expert's first pair
  int count[kFewMaxExperts];  // and its pairs; then where its tile, or its first pair, is
  int expert[PAIRS];
  int sums[kFewMaxWaves];
};

// What a plan begins with: the table of the experts; for every pair p = j THREADS + tid its expert (-1: it is in no
// plan), its place among the expert's, and in plan.weight its weight.
template <int WAVES, int ROUNDS, typename Plan>
__device__ __forceinline__ void few_count(const MoeFewArgs& a, Plan& plan, FewPlanScratch<Plan::kPairs>& s,
                                          int (&mine)[ROUNDS], int (&rank)[ROUNDS]) {
  constexpr int THREADS = WAVES * kWave;
  const int tid = threadIdx.x, pairs = a.tokens * a.topk;
  for (int p = tid; p < pairs; p += THREADS) {
    const int e = a.expert_idx[p];
    const float w = a.weights ? a.weights[p] : 1.f;
    s.expert[p] = e >= 0 && e < a.experts ? e : -1;
    plan.weight[p] = w;
  }
  for (int e = tid; e < a.experts; e += THREADS) s.first[e] = INT32_MAX, s.count[e] = 0;
  __syncthreads();
  float sum[ROUNDS];
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    const int p = j * THREADS + tid;
    mine[j] = -1, rank[j] = 0, sum[j] = 0.f;
    if (p >= pairs) continue;
    mine[j] = s.expert[p];
    const int from = p / a.topk * a.topk;
    bool again = false;
    sum[j] = plan.weight[p];
    for (int q = from; q < from + a.topk; ++q) {
      const bool same = s.expert[q] == mine[j];
      again |= same && q < p;
      sum[j] += same && q > p ? plan.weight[q] : 0.f;
    }
    if (again) mine[j] = -1;
    if (mine[j] < 0) continue;
    atomicMin(&s.first[mine[j]], p);
    rank[j] = atomicAdd(&s.count[mine[j]], 1);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j)
    if (mine[j] >= 0) plan.weight[j * THREADS + tid] = sum[j];
}

// Sums of v over the lanes and waves before this one, and (`all` added to) over all.
template <int WAVES>
__device__ __forceinline__ int few_sum_before(int v, int& all, int (&sums)[kFewMaxWaves]) {
  const int lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x >> 6);
  int upto = v;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int o = __shfl_up(upto, d, kWave);
    upto += lane >= d ? o : 0;
  }
  if (lane == kWave - 1) sums[wave] = upto;
  __syncthreads();
  int before = all + upto - v;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    before += w < wave ? sums[w] : 0;
    all += sums[w];
  }
  __syncthreads();
  return before;
}

template <int TX, int WAVES>
__device__ __forceinline__ void few_plan(const MoeFewArgs& a, FewTokenPlan<TX>& plan,
                                         FewPlanScratch<FewTokenPlan<TX>::kPairs>& s) {
  static_assert(FewTokenPlan<TX>::kPairs <= WAVES * kWave, "a thread for every pair");
  const int p = threadIdx.x, pairs = a.tokens * a.topk;
  if (pairs <= kWave) {
    // A lane for every pair: the first wave does it in registers, the others meet it once (one token, 64 experts of
    // 2048 x 768: a microsecond of 17.6).
    if (p < kWave) {
      int e = -1;
      float w = 0.f;
      if (p < pairs) {
        e = a.expert_idx[p];
        w = a.weights ? a.weights[p] : 1.f;
        if (e >= a.experts) e = -1;
      }
      for (int i = p; i < pairs * TX; i += kWave) plan.pair[i / TX][i % TX] = uint16_t(kFewNone);
      const int token = p / a.topk, from = token * a.topk;
      int head = p;
      bool again = false;
      float sum = w;
      for (int q = 0; q < pairs; ++q) {
        const bool same = __builtin_amdgcn_readlane(e, q) == e;
        const float wq = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), q));
        head = same && q < head ? q : head;
        again |= same && q >= from && q < p;
        sum += same && q > p && q < from + a.topk ? wq : 0.f;
      }
      const uint64_t heads = __ballot(e >= 0 && head == p);
      const int tile = __popcll(heads & ((uint64_t(1) << head) - 1));
      if (e >= 0 && !again) {
        plan.pair[tile][token] = uint16_t(p);
        plan.weight[p] = sum;
        if (head == p) plan.expert[tile] = uint16_t(e);
      }
      if (p == 0) plan.tiles = __popcll(heads);
    }
    __syncthreads();
    return;
  }
  for (int i = p; i < pairs * TX; i += WAVES * kWave) plan.pair[i / TX][i % TX] = uint16_t(kFewNone);
  int mine[1], rank[1], tiles = 0;
  few_count<WAVES>(a, plan, s, mine, rank);
  const bool head = mine[0] >= 0 && s.first[mine[0]] == p;
  const int at = few_sum_before<WAVES>(head, tiles, s.sums);
  if (head) {
    s.count[mine[0]] = at;
    plan.expert[at] = uint16_t(mine[0]);
  }
  if (p == 0) plan.tiles = tiles;
  __syncthreads();
  if (mine[0] >= 0) plan.pair[s.count[mine[0]]][p / a.topk] = uint16_t(p);
  __syncthreads();
}

template <int TX, int WAVES>
__device__ __forceinline__ void few_plan(const MoeFewArgs& a, FewPairPlan<TX>& plan,
                                         FewPlanScratch<FewPairPlan<TX>::kPairs>& s) {
  constexpr int THREADS = WAVES * kWave, ROUNDS = FewPairPlan<TX>::kPairs / THREADS;
  const int tid = threadIdx.x, pairs = a.tokens * a.topk;
  int mine[ROUNDS], rank[ROUNDS], heads[ROUNDS] = {}, all = 0;  // tiles << 16 | pairs
  few_count<WAVES>(a, plan, s, mine, rank);
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    if (j * THREADS >= pairs) continue;
    const bool head = mine[j] >= 0 && s.first[mine[j]] == j * THREADS + tid;
    const int count = head ? s.count[mine[j]] : 0, number = (count + TX - 1) / TX;
    const int at = few_sum_before<WAVES>(number << 16 | count, all, s.sums), tile = at >> 16, pos = at & 0xffff;
    for (int i = 0; i < number; ++i) {
      plan.start[tile + i] = uint16_t(pos + i * TX);
      plan.expert[tile + i] = uint16_t(mine[j]);
      plan.first[tile + i] = uint16_t(tile);
      plan.number[tile + i] = uint16_t(number);
    }
    if (head) s.count[mine[j]] = pos, heads[j] = count;
  }
  if (tid == 0) {
    plan.tiles = all >> 16;
    plan.start[all >> 16] = uint16_t(all & 0xffff);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    if (mine[j] >= 0) s.expert[s.count[mine[j]] + rank[j]] = j * THREADS + tid;  // the pairs by expert, in any order
    if (heads[j]) s.first[mine[j]] = heads[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    if (mine[j] < 0) continue;
    const int pos = s.count[mine[j]], count = s.first[mine[j]], p = j * THREADS + tid;
    if (count > TX) {  // by tile: in order
      rank[j] = 0;
      for (int i = 0; i < count; ++i) rank[j] += s.expert[pos + i] < p;
    }
    plan.pair[pos + rank[j]] = uint16_t(p);
    plan.token[p] = uint16_t(p / a.topk);
  }
  __syncthreads();
}

// What the kernels ask a plan: the pair of column t of a tile (kFewNone: none) and, for a column that has none, a pair
// to read in its place; the row of x for column t; and how many tiles of the same expert there are from a tile on that
// is its first.
template <int TX>
__device__ __forceinline__ unsigned few_pair(const FewTokenPlan<TX>& p, int tile, int t) { return p.pair[tile][t]; }
template <int TX>
__device__ __forceinline__ unsigned few_any_pair(const FewTokenPlan<TX>& p, int tile, int t) {
  unsigned pair = p.pair[tile][t];
  for (int i = 0; pair == kFewNone; ++i) pair = p.pair[tile][i];  // (a tile has one)
  return pair;
}
template <int TX>
__device__ __forceinline__ const uint16_t* few_x(const MoeFewArgs& a, const FewTokenPlan<TX>&, int, int t) {
  return a.x + min(t, a.tokens - 1) * a.x_ld;
}
template <int TX>
__device__ __forceinline__ int few_first(const FewTokenPlan<TX>&, int tile) { return tile; }
template <int TX>
__device__ __forceinline__ int few_number(const FewTokenPlan<TX>&, int) { return 1; }
template <int TX>
__device__ __forceinline__ unsigned few_pair(const FewPairPlan<TX>& p, int tile, int t) {
  const int at = p.start[tile] + t;
  return at < p.start[tile + 1] ? p.pair[at] : kFewNone;
}
template <int TX>
__device__ __forceinline__ unsigned few_any_pair(const FewPairPlan<TX>& p, int tile, int t) {
  return p.pair[min(p.start[tile] + t, p.start[tile + 1] - 1)];
}
template <int TX>
__device__ __forceinline__ const uint16_t* few_x(const MoeFewArgs& a, const FewPairPlan<TX>& p, int tile, int t) {
  return a.x + p.token[few_any_pair(p, tile, t)] * a.x_ld;
}
template <int TX>
__device__ __forceinline__ int few_first(const FewPairPlan<TX>& p, int tile) { return uniform(p.first[tile]); }
template <int TX>
__device__ __forceinline__ int few_number(const FewPairPlan<TX>& p, int tile) { return uniform(p.number[tile]); }

// The first kernel's units in order: experts, row sets of each, and next to one another the tiles of the expert, of
// which the second then finds the rows in the cache.
template <typename Plan>
struct FewUnits {
  const Plan& plan;
  int sets, first, number, set, i;
  __device__ __forceinline__ FewUnits(const Plan& plan_, int sets_, int u) : plan(plan_), sets(sets_) {
    first = few_first(plan, u / sets), number = few_number(plan, first);
    const int r = u - first * sets;
    set = r / number, i = r % number;
  }
  __device__ __forceinline__ int tile() const { return first + i; }
  __device__ __forceinline__ void next() {
    if (++i < number) return;
    i = 0;
    if (++set < sets) return;
    set = 0, first += number;
    number = few_number(plan, min(first, plan.tiles - 1));
  }
};

// ---- the stream ------------------------------------------------------------------
// A block in LDS: 16 R rows of 128 codes (operand tiles, laid out as tile_byte
// says); TX rows of 128 activations (16-byte unit u of token t at u ^ (t & 15));
// 256 bytes more: the R row sets' scales in turn, or (MID) the tokens' eight
// exponents, and from byte 128 on the scale.
template <int TX, int R, int WAVES, int LDS_BYTES, bool MID>
struct FewRing {
  static constexpr int kX = R * 2048, kMore = kX + TX * 256, kSlot = kMore + 256;
  static constexpr int kXCopies = (TX * 256 + 1023) / 1024, kCopies = 2 * R + kXCopies + 1;
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
  int lane, groups, g, g_restart, g_step, total, issued = 0, taken = 0, issue_slot = 0, read_slot = 0;
  FewSource<R> src;
  const uint16_t* xsrc[L::kXCopies];
  unsigned row_off[2];

  // `units`: source() the data of the unit it is at, x_row(t) its t-th token's activations, next() goes on.
  template <typename U>
  __device__ __forceinline__ void begin_unit(U& units) {
    src = units.source();
#pragma unroll
    for (int c = 0; c < L::kXCopies; ++c) {
      const int t = (c * 64 + lane) / 16;
      xsrc[c] = units.x_row(t & (TX - 1)) + (((lane & 15) ^ t) & 15) * 8;
    }
  }
  // Blocks of this wave: `total` of them, from block g_ of the first unit on every step-th, in further units from block
  // `restart` on.
  template <typename U>
  __device__ __forceinline__ void start(char* lds, int k, int g_, int restart, int step, int total_, U& units) {
    const int wave = uniform(threadIdx.x >> 6);
    lane = threadIdx.x & (kWave - 1);
    ring = lds + wave * L::kWaveBytes;
    ring_at = lds_addr(lds) + wave * L::kWaveBytes;
    groups = k / kGroupK;
    g = g_, g_restart = restart, g_step = step, total = total_;
#pragma unroll
    for (int h = 0; h < 2; ++h) row_off[h] = unsigned(tile_row(h, lane)) * unsigned(k) + 16u * tile_chunk(h, lane);
    if (total > 0) begin_unit(units);
    for (int i = 0; i < L::kBlocks && i < total; ++i) copy_next(units);
  }
  template <typename U>
  __device__ __forceinline__ void copy_next(U& units) {
    const uint32_t at = ring_at + unsigned(issue_slot) * L::kSlot;
#pragma unroll
    for (int s = 0; s < R; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        copy16_to_lds(src.codes[s] + g * kGroupK, row_off[h], at + s * 2048 + h * 1024);
#pragma unroll
    for (int c = 0; c < L::kXCopies; ++c)
      if (TX >= 4 || lane < TX * 16) few_copy16(xsrc[c] + g * kGroupK, at + L::kX + c * 1024);
    const int step = MID && lane < 32 ? kGroupK / kFewGroup : 4;
    few_copy4(static_cast<const char*>(src.more) + g * step, at + L::kMore);
    issue_slot = issue_slot + 1 == L::kBlocks ? 0 : issue_slot + 1;
    g += g_step;
    if (++issued < total && g >= groups) {
      g = g_restart;
      units.next();
      begin_unit(units);
    }
  }
  template <int N = L::kBlocks - 1>
  __device__ __forceinline__ void wait(int newer) {
    if (N == 0 || newer >= N) few_copies_left<N * L::kCopies>();
    else if constexpr (N > 0) wait<N - 1>(newer);
  }
  template <typename U>
  __device__ __forceinline__ FewBlock<R> next(U& units) {
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
    if (issued < total) copy_next(units);
    b.exponent = 0;
    if constexpr (MID) {
      // The lane's activations, 32 columns from 32 q on, are of the groups 2 q and 2 q + 1: brought to the token's
      // largest exponent.  One power of two takes a group down by 2^-14 and, where a lane has one farther down, another by
      // 2^-24 more (under that: 0).  (Both for every block: 64 tokens, 128 experts of 7168 x 2048 965 us, 918 so.)
      int top = -128, own[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, int(exponents[i / 4] << (24 - 8 * (i & 3))) >> 24);
      const int word = q & 2 ? exponents[1] : exponents[0], half = q & 1 ? word >> 16 : word;
      own[0] = int(unsigned(half) << 24) >> 24, own[1] = int(unsigned(half) << 16) >> 24;
      b.exponent = top;
      auto times = [&](int j, _Float16 by) {
        x[j] = __builtin_bit_cast(v4i, __builtin_bit_cast(v8f16_t, x[j]) * by);
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) times(j, few_power(max(own[j / 2] - top, -14)));
      if (__any(min(own[0], own[1]) - top < -14)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) times(j, few_power(min(own[j / 2] - top + 14, 0)));
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
  // This lane's four rows of row set s.
  __device__ __forceinline__ v4f* at(int wave, int t, int s) {
    return reinterpret_cast<v4f*>(&v[wave][t][((4 * s + (threadIdx.x >> 4 & 3)) ^ (t & (4 * R - 1))) * 4]);
  }
  __device__ __forceinline__ void put(const v4f (&acc)[R]) {
    const int t = threadIdx.x & 15;
    if (t >= TX) return;
#pragma unroll
    for (int s = 0; s < R; ++s) *at(threadIdx.x >> 6, t, s) = acc[s];
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
// A unit is 8 R rows of G and the 8 R of U of one tile; a workgroup takes a run of
// units, its waves every fourth block of each.  Grid: any number of workgroups.
constexpr int kFewUpWaves = 4;
constexpr int kFewLds = 160 * 1024;
// Two workgroups fit a CU with a few tokens (their waits then overlap), one with more.
template <int TX>
constexpr int kFewUpPerCu = TX <= 4 ? 2 : 1;
template <int TX, int R, typename Plan>
struct FewUp {
  static constexpr int kRest = int(sizeof(Plan) + sizeof(FewSums<TX, R, kFewUpWaves>)) + 1024;
  using Ring = FewRing<TX, R, kFewUpWaves, kFewLds / kFewUpPerCu<TX> - kRest, false>;
  __attribute__((aligned(1024))) char ring[Ring::kBytes];
  FewSums<TX, R, kFewUpWaves> sums;
  Plan plan;
  static_assert(sizeof(FewPlanScratch<Plan::kPairs>) <= Ring::kBytes, "the plan's scratch takes the ring's place");
};

template <int TX, int R, typename Plan>
__global__ void __launch_bounds__(kFewUpWaves* kWave) moe_few_up_kernel(const MoeFewArgs a) {
  using Lds = FewUp<TX, R, Plan>;
  constexpr int kRows = 8 * R;  // of G, and of U
  __shared__ Lds lds;
  const Plan& plan = lds.plan;
  few_plan<TX, kFewUpWaves>(a, lds.plan, *reinterpret_cast<FewPlanScratch<Plan::kPairs>*>(lds.ring));
  const int sets = a.inter / kRows, tid = threadIdx.x, wave = uniform(tid >> 6);
  const int64_t units = int64_t(uniform(plan.tiles)) * sets;
  const int u0 = int(units * blockIdx.x / gridDim.x), u1 = int(units * (blockIdx.x + 1) / gridDim.x);
  if (u0 == u1) return;
  struct Units : FewUnits<Plan> {
    const MoeFewArgs& a;
    int kg;
    __device__ __forceinline__ Units(const MoeFewArgs& a_, const Plan& plan_, int sets_, int u)
        : FewUnits<Plan>(plan_, sets_, u), a(a_), kg(a_.hidden / kGroupK) {}
    __device__ __forceinline__ FewSource<R> source() const {
      const int e = uniform(this->plan.expert[this->tile()]), row = this->set * kRows;
      FewSource<R> s;
#pragma unroll
      for (int r = 0; r < R; ++r)
        s.codes[r] = a.up + (int64_t(e) * 2 * a.inter + (r < R / 2 ? 0 : a.inter) + row + 16 * (r % (R / 2))) * a.hidden;
      s.more = a.up_scales + (int64_t(e) * 2 * (a.inter / kGroupK) + row / kGroupK +
                              ((threadIdx.x & (R - 1)) < R / 2 ? 0 : a.inter / kGroupK)) * kg;
      return s;
    }
    __device__ __forceinline__ const uint16_t* x_row(int t) const { return few_x(a, this->plan, this->tile(), t); }
  };
  Units copied(a, plan, sets, u0);
  FewUnits<Plan> at(plan, sets, u0);
  FewStream<typename Lds::Ring, TX, R, kFewUpWaves, false> stream;
  const int blocks = (a.hidden / kGroupK - wave + kFewUpWaves - 1) / kFewUpWaves;
  stream.start(lds.ring, a.hidden, wave, wave, kFewUpWaves, (u1 - u0) * blocks, copied);
  for (int u = u0; u < u1; ++u, at.next()) {
    v4f acc[R] = {};
    for (int i = 0; i < blocks; ++i) {
      const FewBlock<R> b = stream.next(copied);
#pragma unroll
      for (int s = 0; s < R; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[s][r] = fmaf(b.scale[s], b.part[s][r], acc[s][r]);
    }
    few_barrier();  // the sums of the unit before are read
    lds.sums.put(acc);
    few_barrier();
    for (int o = tid; o < TX * kRows; o += kFewUpWaves * kWave) {
      const int row = o % kRows, t = o / kRows;
      const unsigned p = few_pair(plan, at.tile(), t);
      if (p == kFewNone) continue;  // (16 lanes together)
      const float v = activate(a.activation, lds.sums.get(t, row)) * lds.sums.get(t, kRows + row);
      // FP16 with the exponent that takes the largest of the 16 to 2^14 .. 2^15; with an infinity or a NaN the largest
      // exponent, which leaves it what it is.
      float top = fabsf(v);
#pragma unroll
      for (int d = 1; d < 16; d *= 2) {
        const float other = __shfl_xor(top, d, 16);
        top = other > top || other != other ? other : top;
      }
      const int e = top < __builtin_inff() ? max(-128, (top > 0.f ? ilogbf(top) : -128) - 14) : 113;
      const _Float16 h = _Float16(ldexpf(v, -e));
      const int64_t to = int64_t(p) * a.inter + at.set * kRows + row;
      a.mid[to] = __builtin_bit_cast(uint16_t, h);
      if (row % kFewGroup == 0) a.exponents[to / kFewGroup] = int8_t(e);
    }
  }
}

// ---- second kernel -----------------------------------------------------------------
// A workgroup has 16 R rows of the output; its waves take equal runs of the
// tiles' blocks and meet once, at the end.  With a column for each token (a
// FewTokenPlan) a wave's sums over all experts, weighted, stay in registers;
// else they are added, at the end of each of its tiles, to the wave's own sums
// of every token in LDS.  Where there are few rows, slices of the tiles' blocks
// have workgroups of their own; their sums go past the caches to `partial`, and the
// last of them to arrive adds them in order (the counters are those of the
// split-K GEMM: a word that does not carry the call's tag is restarted, and the
// last arrival leaves it at zero).  Grid: x hidden / (16 R), y slices.
constexpr int kFewMaxSlices = 8;

// Counts an arrival; whether it is the last of `all`.
__device__ __forceinline__ bool few_arrive(unsigned long long* counter, unsigned tag, int all) {
  unsigned long long old = __hip_atomic_load(counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), now;
  for (;;) {
    if (unsigned(old >> 32) == tag) {
      now = __hip_atomic_fetch_add(counter, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1;
      break;
    }
    now = (unsigned long long)tag << 32 | 1ull;
    if (__hip_atomic_compare_exchange_strong(counter, &old, now, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT))
      break;
  }
  const bool last = unsigned(now) == unsigned(all);
  if (last) __hip_atomic_store(counter, (unsigned long long)tag << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return last;
}

// The sum of S slices' partial sums, in order.
template <int S>
__device__ __forceinline__ v4f few_add(const float* partial, int64_t size) {
  const float* at[S];
  v4f v[S];
#pragma unroll
  for (int s = 0; s < S; ++s) at[s] = partial + s * size;
  load16_coherent<S>(at, v);
#pragma unroll
  for (int s = 1; s < S; ++s) v[0] += v[s];
  return v[0];
}

template <int TX, int R, int WAVES, typename Plan>
struct FewDown {
  static constexpr bool kTokens = std::is_same_v<Plan, FewTokenPlan<TX>>;
  static constexpr int kSums = kTokens ? TX : kFewTokens;  // tokens
  static constexpr int kApart = kTokens ? 0 : int(sizeof(FewSums<kSums, R, WAVES>));
  using Ring = FewRing<TX, R, WAVES, kFewLds - int(sizeof(Plan)) - kApart - 1024, true>;
  using Sums = FewSums<kSums, R, WAVES>;
  __attribute__((aligned(1024))) char ring[Ring::kBytes + kApart];  // the tokens' sums lie behind it, or take its place
  Plan plan;
  static_assert(sizeof(Sums) <= sizeof(ring) && sizeof(FewPlanScratch<Plan::kPairs>) <= Ring::kBytes, "places");
};

template <int TX, int R, int WAVES, typename Plan>
__global__ void __launch_bounds__(WAVES* kWave) moe_few_down_kernel(const MoeFewArgs a) {
  using Lds = FewDown<TX, R, WAVES, Plan>;
  constexpr int kRows = 16 * R;
  __shared__ Lds lds;
  const Plan& plan = lds.plan;
  auto& sums = *reinterpret_cast<typename Lds::Sums*>(lds.ring + (Lds::kTokens ? 0 : Lds::Ring::kBytes));
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid >> 6);
  if constexpr (!Lds::kTokens)
    for (int i = lane; i < a.tokens * kRows; i += kWave) sums.v[wave][i / kRows][i % kRows] = 0.f;
  few_plan<TX, WAVES>(a, lds.plan, *reinterpret_cast<FewPlanScratch<Plan::kPairs>*>(lds.ring));
  const int row0 = blockIdx.x * kRows, kg = a.inter / kGroupK, sets = a.inter / kFewGroup;
  const int all = uniform(plan.tiles) * kg;  // (at most 512 tiles of 512 blocks)
  const int slices = gridDim.y, run = blockIdx.y * WAVES + wave;
  const int f0 = int(int64_t(all) * run / (slices * WAVES)), f1 = int(int64_t(all) * (run + 1) / (slices * WAVES));
  struct Units {
    const MoeFewArgs& a;
    const Plan& plan;
    int tile, row0, kg, sets;
    __device__ __forceinline__ void next() { ++tile; }
    __device__ __forceinline__ FewSource<R> source() const {
      const int e = uniform(plan.expert[tile]), lane = threadIdx.x & (kWave - 1);
      FewSource<R> s;
#pragma unroll
      for (int r = 0; r < R; ++r) s.codes[r] = a.down + (int64_t(e) * a.hidden + row0 + 16 * r) * a.inter;
      const float* scales = a.down_scales + (int64_t(e) * (a.hidden / kGroupK) + row0 / kGroupK) * kg;
      const int64_t p = few_any_pair(plan, tile, (lane >> 1) & (TX - 1));
      s.more = lane < 32 ? static_cast<const void*>(a.exponents + p * sets + 4 * (lane & 1)) : scales;
      return s;
    }
    __device__ __forceinline__ const uint16_t* x_row(int t) const {
      return a.mid + int64_t(few_any_pair(plan, tile, t)) * a.inter;
    }
  };
  Units copied{a, plan, f0 / kg, row0, kg, sets};
  FewStream<typename Lds::Ring, TX, R, WAVES, true> stream;
  stream.start(lds.ring, a.inter, f0 % kg, 0, 1, f1 - f0, copied);
  v4f acc[R] = {};
  for (int f = f0, unit = f0 / kg; f < f1; ++unit) {
    const unsigned p = few_pair(plan, unit, lane & (TX - 1));
    const bool live = p != kFewNone;
    const float weight = live ? plan.weight[p] : 0.f;
    for (const int end = min(f1, (unit + 1) * kg); f < end; ++f) {
      const FewBlock<R> b = stream.next(copied);
      float scale = ldexpf(b.scale[0], b.exponent);
      if constexpr (Lds::kTokens) scale *= weight;
#pragma unroll
      for (int s = 0; s < R; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[s][r] = live ? fmaf(scale, b.part[s][r], acc[s][r]) : acc[s][r];
    }
    if constexpr (!Lds::kTokens) {
      const int token = live ? plan.token[p] : 0;
#pragma unroll
      for (int s = 0; s < R; ++s) {
        v4f* to = sums.at(wave, token, s);
        if (live && (lane & 15) < TX) {  // a tile has a token once
          v4f v = *to;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = fmaf(weight, acc[s][r], v[r]);
          *to = v;
        }
        acc[s] = v4f{0.f, 0.f, 0.f, 0.f};
      }
    }
  }
  __syncthreads();  // every wave is done with its ring
  if constexpr (Lds::kTokens) {
    sums.put(acc);
    __syncthreads();
  }
  if (slices > 1) {
    const int64_t size = int64_t(a.tokens) * a.hidden;
    constexpr int kPieces = kRows / 4;
    for (int o = tid; o < a.tokens * kPieces; o += WAVES * kWave) {
      const int t = o / kPieces, c = 4 * (o % kPieces);
      store16_coherent(a.partial + blockIdx.y * size + int64_t(t) * a.hidden + row0 + c,
                       v4f{sums.get(t, c), sums.get(t, c + 1), sums.get(t, c + 2), sums.get(t, c + 3)});
    }
    __shared__ int last;
    wait_vmcnt<0>();
    __syncthreads();
    if (tid == 0) last = few_arrive(a.counters + blockIdx.x, a.tag, slices);
    __syncthreads();
    if (!last) return;
    for (int o = tid; o < a.tokens * kPieces; o += WAVES * kWave) {
      const int64_t at = int64_t(o / kPieces) * a.hidden + row0 + 4 * (o % kPieces);
      v4f sum;
      if (slices == 2) sum = few_add<2>(a.partial + at, size);
      else if (slices == 4) sum = few_add<4>(a.partial + at, size);
      else sum = few_add<8>(a.partial + at, size);
      *reinterpret_cast<uint2*>(a.out + at) = make_uint2(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]));
    }
    return;
  }
  for (int o = tid; o < a.tokens * (kRows / 2); o += WAVES * kWave) {
    const int t = o / (kRows / 2), c = 2 * (o % (kRows / 2));
    *reinterpret_cast<uint32_t*>(a.out + int64_t(t) * a.hidden + row0 + c) =
        pack_bf16x2(sums.get(t, c), sums.get(t, c + 1));
  }
}

}  // namespace fp8g
