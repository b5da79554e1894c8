// A mixture-of-experts layer for a few tokens, in two kernels, for gfx950.
//
//   mid[p] = bf16( act(G_e x_t) * (U_e x_t) )          p = t topk + j, e = expert_idx[p]
//   out[t] = bf16( sum over j of weights[p] D_e mid[p] )
// G_e, U_e: the first and the last `inter` rows of the expert's first matrix
// [2 inter][hidden], D_e its second [hidden][inter], FP8 E4M3 codes with an
// FP32 scale per 128 x 128 block, as the grouped GEMMs take them; x, mid BF16.
// (mid is rounded to BF16 because that is what the matrix instruction takes;
// it costs as much as the output's own rounding does.)
//
// Both kernels stream matrices through the same code.  A unit is 32 rows of an
// expert's matrix (16 of G and 16 of U, or 32 of D) times up to TX of its
// pairs; a workgroup takes units one after the other.  Its waves share a unit's
// k: wave w takes the 128-column blocks w, w + 4, ..., each with a ring of its
// own in LDS that direct copies fill several blocks ahead, across units, so the
// matrices arrive without a pause and the waves meet only at a unit's end, where
// their partial sums are added in the order of the waves.
//
// Codes become BF16 operands exactly, times 2^-16: then no sum of a block's 128
// products passes FP32's range where its scaled value does not.  The block's
// scale, times 2^16, is applied to the FP32 sum.
//
// What bounds it: the matrices are read once, a byte a weight.
#pragma once

#include "activation.hpp"
#include "gemm_kernel.hpp"  // lds_frag's layout helpers

namespace fp8g {

constexpr int kFewWaves = 4, kFewThreads = kFewWaves * kWave;
constexpr int kFewRows = 32;     // of a unit
constexpr int kFewTokens = 64;   // of a launch, at most
constexpr int kFewMaxPairs = 1024;

struct MoeFewArgs {
  const uint16_t* x;
  int64_t x_ld;
  const int32_t* expert_idx;
  const float* weights;
  const uint8_t *up, *down;
  const float *up_scales, *down_scales;
  uint16_t *mid, *out;
  int tokens, topk, experts, hidden, inter, activation;
};

typedef __bf16 v8bf16_t __attribute__((ext_vector_type(8)));
typedef float v2f_t __attribute__((ext_vector_type(2)));

// Eight E4M3 codes (two dwords) -> eight BF16 values times 2^-16, exact.
__device__ __forceinline__ v4i few_decode(int lo, int hi) {
  constexpr float s = 1.f / 65536.f;
  v4i f;
  f[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(lo), s, false));
  f[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(lo), s, true));
  f[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(hi), s, false));
  f[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(hi), s, true));
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

// ---- which expert has which pairs ---------------------------------------------
// Pairs of one expert that follow one another form tiles of TX; tiles stand in
// the order of their first pairs.  Pairs whose index is no expert's are in none.
template <int MAXP>
struct FewPlan {
  uint16_t pair[MAXP];       // by tile, in a tile in order
  uint16_t start[MAXP + 1];  // tile t's pairs are pair[start[t]] .. pair[start[t + 1] - 1]
  uint16_t expert[MAXP];
  int tiles;
};
template <int MAXP>
struct FewPlanScratch {
  __attribute__((aligned(16))) int expert[MAXP];
  int count[MAXP];
  int sums[kFewWaves];
};

// Every pair compares its expert with those of the pairs before it: rank = how
// many are the same, and the pair that begins its tile.  A scan over the tiles'
// first pairs then places the tiles.
template <int TX, int MAXP>
__device__ __forceinline__ void few_plan(const MoeFewArgs& a, FewPlan<MAXP>& plan, FewPlanScratch<MAXP>& s) {
  constexpr int ROUNDS = (MAXP + kFewThreads - 1) / kFewThreads;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6, pairs = a.tokens * a.topk;
  const int padded = (pairs + 3) & ~3;
  for (int p = tid; p < MAXP && p < padded; p += kFewThreads) {
    const int e = p < pairs ? a.expert_idx[p] : -1;
    s.expert[p] = e >= 0 && e < a.experts ? e : -1;
    s.count[p] = 0;
  }
  __syncthreads();
  int rank[ROUNDS], head[ROUNDS], mine[ROUNDS];
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    const int p = j * kFewThreads + tid;
    rank[j] = 0, head[j] = p, mine[j] = -1;
    if (j * kFewThreads >= pairs) continue;
    mine[j] = p < pairs ? s.expert[p] : -1;
    const int end = min(pairs, uniform(p) + kWave);  // the wave's last pair
    for (int q0 = 0; q0 < end; q0 += 4) {
      const v4i e = *reinterpret_cast<const v4i*>(s.expert + q0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool same = e[i] == mine[j] && q0 + i < p;
        head[j] = same && rank[j] % TX == 0 ? q0 + i : head[j];
        rank[j] += same;
      }
    }
    if (rank[j] % TX == 0) head[j] = p;
    if (mine[j] >= 0) atomicAdd(&s.count[head[j]], 1);
  }
  __syncthreads();
  int before = 0;  // tiles << 16 | pairs of the rounds before
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    const int p = j * kFewThreads + tid;
    if (j * kFewThreads >= pairs) continue;
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
    for (int w = 0; w < kFewWaves; ++w) {
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
    if (mine[j] >= 0) plan.pair[s.count[head[j]] + rank[j] % TX] = uint16_t(j * kFewThreads + tid);
  __syncthreads();
}

// ---- the stream ------------------------------------------------------------------
// A block in LDS: 32 rows of 128 codes (two operand tiles, laid out as
// tile_byte says), TX rows of 128 BF16 activations (16-byte unit u of token t
// at u ^ (t & 15)), the two row sets' scales in turn.
template <int TX>
struct FewRing {
  static constexpr int kX = 4096, kScales = kX + TX * 256, kSlot = kScales + 256;
  static constexpr int kXCopies = TX * 256 / 1024, kCopies = 4 + kXCopies + 1;
  static constexpr int kBlocks = TX == 16 ? 4 : 3, kWave = kBlocks * kSlot;
  static constexpr int kMaxPairs = TX == 16 ? kFewMaxPairs : 128;
};

// Where a unit's data lies.
struct FewSource {
  const uint8_t* codes[2];  // 16 rows each
  const float* scales[2];   // of the row sets' blocks, one after another
};

template <int TX>
struct FewStream {
  using L = FewRing<TX>;
  const char* ring;
  uint32_t ring_at;
  int k, blocks, wave, lane;  // blocks: of this wave in a unit
  int issued = 0, copied_unit, copied_block = 0, issue_slot = 0, read_slot = 0, total;
  FewSource src;
  const uint16_t* xsrc[L::kXCopies];
  unsigned row_off[2];

  // `source(unit)`, `x_row(unit, t)`: the data of a unit and of its t-th pair.
  template <typename S, typename X>
  __device__ __forceinline__ void begin_unit(int unit, S&& source, X&& x_row) {
    src = source(unit);
#pragma unroll
    for (int c = 0; c < L::kXCopies; ++c) {
      const int t = (c * 64 + lane) / 16;
      xsrc[c] = x_row(unit, t) + (((lane & 15) ^ t) & 15) * 8;
    }
  }
  template <typename S, typename X>
  __device__ __forceinline__ void start(char* lds, int k_, int unit0, int units, S&& source, X&& x_row) {
    lane = threadIdx.x & (kWave - 1), wave = uniform(threadIdx.x >> 6);
    ring = lds + wave * L::kWave;
    ring_at = lds_addr(lds) + wave * L::kWave;
    k = k_;
    blocks = (k / kGroupK - wave + kFewWaves - 1) / kFewWaves;
    total = units * blocks;
    copied_unit = unit0;
#pragma unroll
    for (int h = 0; h < 2; ++h) row_off[h] = unsigned(tile_row(h, lane)) * unsigned(k) + 16u * tile_chunk(h, lane);
    if (total > 0) begin_unit(unit0, source, x_row);
    for (int i = 0; i < L::kBlocks && i < total; ++i) copy_next(source, x_row);
  }
  template <typename S, typename X>
  __device__ __forceinline__ void copy_next(S&& source, X&& x_row) {
    const int g = wave + copied_block * kFewWaves;
    const uint32_t at = ring_at + unsigned(issue_slot) * L::kSlot;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        copy16_to_lds(src.codes[s] + g * kGroupK, row_off[h], at + s * 2048 + h * 1024);
#pragma unroll
    for (int c = 0; c < L::kXCopies; ++c) few_copy16(xsrc[c] + g * kGroupK, at + L::kX + c * 1024);
    few_copy4((lane & 1 ? src.scales[1] : src.scales[0]) + g, at + L::kScales);
    issue_slot = issue_slot + 1 == L::kBlocks ? 0 : issue_slot + 1;
    if (++issued < total && ++copied_block == blocks) {
      copied_block = 0;
      begin_unit(++copied_unit, source, x_row);
    }
  }
  // acc[s] += the next block's products, of row set s.
  template <typename S, typename X>
  __device__ __forceinline__ void next(int i, v4f (&acc)[2], S&& source, X&& x_row) {
    const int newer = min(total - 1 - i, L::kBlocks - 1);  // blocks in flight after this one
    if (newer >= 3) few_copies_left<3 * L::kCopies>();
    else if (newer == 2) few_copies_left<2 * L::kCopies>();
    else if (newer == 1) few_copies_left<L::kCopies>();
    else few_copies_left<0>();
    const char* at = ring + read_slot * L::kSlot;
    read_slot = read_slot + 1 == L::kBlocks ? 0 : read_slot + 1;
    const int lr = lane & 15, q = lane >> 4, t = lr & (TX - 1);
    v4i codes[2][2], x[4];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        codes[s][h] = *reinterpret_cast<const v4i*>(at + s * 2048 + tile_byte(lr, 2 * q + h));
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const v4i*>(at + L::kX + t * 256 + ((4 * q + j) ^ t) * 16);
    const v2f_t scale = *reinterpret_cast<const v2f_t*>(at + L::kScales);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the block has been read
    if (issued < total) copy_next(source, x_row);
    v4f part[2] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        part[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(v8bf16_t, few_decode(codes[s][j / 2][2 * (j & 1)], codes[s][j / 2][2 * (j & 1) + 1])),
            __builtin_bit_cast(v8bf16_t, x[j]), part[s], 0, 0, 0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[s][r] = fmaf(scale[s] * 65536.f, part[s][r], acc[s][r]);
  }
};

// The waves' sums of a unit: [wave][token][32 rows], 16-byte piece c of token t at c ^ (t & 7).
template <int TX>
struct FewSums {
  float v[kFewWaves][TX][kFewRows];
  __device__ __forceinline__ void put(const v4f (&acc)[2]) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6, t = lane & 15, q = lane >> 4;
    if (t >= TX) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) *reinterpret_cast<v4f*>(&v[wave][t][((4 * s + q) ^ (t & 7)) * 4]) = acc[s];
  }
  __device__ __forceinline__ float get(int t, int row) const {
    const int at = ((row >> 2) ^ (t & 7)) * 4 + (row & 3);
    float sum = v[0][t][at];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) sum += v[w][t][at];
    return sum;
  }
};

// LDS of both kernels; the plan's scratch takes the ring's place before the first copy.
template <int TX>
struct FewLds {
  __attribute__((aligned(1024))) char ring[kFewWaves * FewRing<TX>::kWave];
  FewSums<TX> sums;
  FewPlan<FewRing<TX>::kMaxPairs> plan;
  static_assert(sizeof(FewPlanScratch<FewRing<TX>::kMaxPairs>) <= kFewWaves * FewRing<TX>::kWave, "scratch");
};

// Grid: any number of workgroups, which share the units (16 rows of G and of U each) in equal runs.
template <int TX>
__global__ void __launch_bounds__(kFewThreads) moe_few_up_kernel(const MoeFewArgs a) {
  __shared__ FewLds<TX> lds;
  using L = FewRing<TX>;
  auto& plan = lds.plan;
  few_plan<TX>(a, plan, *reinterpret_cast<FewPlanScratch<L::kMaxPairs>*>(lds.ring));
  const int sets = a.inter / 16, kg = a.hidden / kGroupK, tid = threadIdx.x;
  const int64_t units = int64_t(uniform(plan.tiles)) * sets;
  const int u0 = int(units * blockIdx.x / gridDim.x), u1 = int(units * (blockIdx.x + 1) / gridDim.x);
  if (u0 == u1) return;
  auto source = [&](int u) {
    const int e = uniform(plan.expert[u / sets]), row = u % sets * 16;
    FewSource s;
    s.codes[0] = a.up + (int64_t(e) * 2 * a.inter + row) * a.hidden;
    s.codes[1] = s.codes[0] + int64_t(a.inter) * a.hidden;
    s.scales[0] = a.up_scales + (int64_t(e) * 2 * (a.inter / kGroupK) + row / kGroupK) * kg;
    s.scales[1] = s.scales[0] + int64_t(a.inter / kGroupK) * kg;
    return s;
  };
  auto x_row = [&](int u, int t) {  // past the tile's pairs: the last one's again
    const int tile = u / sets;
    const int p = plan.pair[min(plan.start[tile] + t, plan.start[tile + 1] - 1)];
    return a.x + (p / a.topk) * a.x_ld;
  };
  FewStream<TX> stream;
  stream.start(lds.ring, a.hidden, u0, u1 - u0, source, x_row);
  int i = 0;
  for (int u = u0; u < u1; ++u) {
    v4f acc[2] = {};
    for (int b = 0; b < stream.blocks; ++b) stream.next(i++, acc, source, x_row);
    few_barrier();  // the sums of the unit before are read
    lds.sums.put(acc);
    few_barrier();
    const int tile = u / sets, row = tid & 15, t = tid >> 4, at = plan.start[tile] + t;
    if (t < TX && at < plan.start[tile + 1]) {
      const float v = activate(a.activation, lds.sums.get(t, row)) * lds.sums.get(t, 16 + row);
      a.mid[int64_t(plan.pair[at]) * a.inter + u % sets * 16 + row] = uint16_t(pack_bf16x2(v, 0.f));
    }
  }
}

// Grid: 32 rows of the output each, through all tiles.
template <int TX>
__global__ void __launch_bounds__(kFewThreads) moe_few_down_kernel(const MoeFewArgs a) {
  constexpr int kTokens = TX == 16 ? kFewTokens : 4;
  __shared__ FewLds<TX> lds;
  __shared__ float out[kTokens][kFewRows];
  __shared__ float weight[FewRing<TX>::kMaxPairs];
  using L = FewRing<TX>;
  auto& plan = lds.plan;
  const int tid = threadIdx.x, row0 = blockIdx.x * kFewRows, kg = a.inter / kGroupK;
  for (int p = tid; p < a.tokens * a.topk; p += kFewThreads) weight[p] = a.weights ? a.weights[p] : 1.f;
  for (int o = tid; o < a.tokens * kFewRows; o += kFewThreads) out[o / kFewRows][o % kFewRows] = 0.f;
  few_plan<TX>(a, plan, *reinterpret_cast<FewPlanScratch<L::kMaxPairs>*>(lds.ring));
  const int tiles = uniform(plan.tiles);
  auto source = [&](int u) {
    const int e = uniform(plan.expert[u]);
    FewSource s;
    s.codes[0] = a.down + (int64_t(e) * a.hidden + row0) * a.inter;
    s.codes[1] = s.codes[0] + int64_t(16) * a.inter;
    s.scales[0] = s.scales[1] = a.down_scales + (int64_t(e) * (a.hidden / kGroupK) + row0 / kGroupK) * kg;
    return s;
  };
  auto x_row = [&](int u, int t) {
    return a.mid + int64_t(plan.pair[min(plan.start[u] + t, plan.start[u + 1] - 1)]) * a.inter;
  };
  FewStream<TX> stream;
  stream.start(lds.ring, a.inter, 0, tiles, source, x_row);
  int i = 0;
  for (int u = 0; u < tiles; ++u) {
    v4f acc[2] = {};
    for (int b = 0; b < stream.blocks; ++b) stream.next(i++, acc, source, x_row);
    few_barrier();  // the sums of the unit before are read
    lds.sums.put(acc);
    few_barrier();
    const int first = plan.start[u], count = plan.start[u + 1] - first;
    for (int o = tid; o < count * kFewRows; o += kFewThreads) {
      const int row = o % kFewRows;
      int t = o / kFewRows;
      const int token = plan.pair[first + t] / a.topk;
      // pairs of one token (an expert picked twice) follow one another; the first one's thread adds them all
      if (t > 0 && plan.pair[first + t - 1] / a.topk == token) continue;
      float sum = out[token][row];
      for (; t < count && plan.pair[first + t] / a.topk == token; ++t)
        sum = fmaf(weight[plan.pair[first + t]], lds.sums.get(t, row), sum);
      out[token][row] = sum;
    }
  }
  __syncthreads();
  for (int o = tid; o < a.tokens * (kFewRows / 2); o += kFewThreads) {
    const int t = o / (kFewRows / 2), c = 2 * (o % (kFewRows / 2));
    *reinterpret_cast<uint32_t*>(a.out + int64_t(t) * a.hidden + row0 + c) = pack_bf16x2(out[t][c], out[t][c + 1]);
  }
}

}  // namespace fp8g
