// Launches of the 4-bit product kernels; compiled once for each FP8G_W4_KIND
// (0: INT4, 1: INT4 with zero points, 2: E2M1).
#include "w4_launch.hpp"

#include <algorithm>

#include "fp8gemm.h"
#include "w4_kernel.hpp"

namespace fp8g {
namespace host {
namespace {

// Figures below: both sides by calls issued back to back, in one run.
//
// k is split over the waves of a workgroup, 8 ways up to kSplit8 row sets, 4
// ways up to kSplit4, else 2 ways.  A workgroup of 8 waves fills a CU's LDS, one
// of 4 half of it, so kSplit8 workgroups run at once, or twice as many small
// ones, and a few more sets would cost a second round.  Measured with one token
// (16 for those marked *), 8, 4 and 2 ways: 256 sets (4096 x 7168) 6.5, 8.5 and
// 13 us; 320 (5120 x 5120) 7.6 and 7.0; 448 (7168 x 16384) 18.6 and 16.0.  4 and
// 2 ways: 640 sets (10240 x 4096) 8.6 and 9.7; 768* (24576 x 1536) 8.7 and 9.6;
// 896 (14336 x 4096) 10.7 and 10.1.
constexpr int kSplit8 = 256, kSplit4 = 768;
// Row sets from which on a wave takes whole rows.  Measured for one token,
// whole rows against k split: 1024 sets (16384 x 4096) 13.8 and 10.4 us, 1536
// (24576 x 1536) 7.7 and 8.1, (24576 x 7168) 23.9 and 21.6, 1792 (28672 x 2048)
// 9.3 and 10.8, 4096 (65536 x 1024) 9.9 and 10.7; six experts of 4096 x 2048
// (1536) 10.2 and 14.2, eight (2048) 11.6 and 13.5.
constexpr int kStreamSets = 1536;
constexpr int kStreamBytes = 64 * 1024;  // activations of a streaming workgroup, at most
// Workgroups that a long stream is dealt to: a wave then takes several sets one
// after another and the copies never pause between them (256 experts of 4096 x
// 1024: 139 us, 152 with a workgroup for every 8 sets; one token, 1048576 x
// 256: 38 and 49; no difference from k = 2048 on).
constexpr int kStreamWorkgroups = 2048;

int64_t cdiv64(int64_t x, int64_t y) { return (x + y - 1) / y; }

// Tiles of 16 that the routed form has as a rule: counted by the experts alone, 512 pairs with 8 experts of 1024 x 1024
// took 18.8 us, not 10.1 (k split in more parts than there was room for).
int64_t routed_tiles(const W4Args& a) { return std::max(a.experts, a.m / 16); }

template <int FMT, bool Z, int G, int TX, int R, int U, bool ROUTED>
int launch_kernel(W4Args a, hipStream_t s) {
  // Grid rows, and how many of them have a tile as a rule.
  const int64_t slots = !ROUTED ? cdiv64(a.m, TX) : w4_by_pair(TX) ? a.m : int64_t(a.experts) + 1 + (a.m - 1) / TX;
  const int64_t tiles = ROUTED && !w4_by_pair(TX) ? routed_tiles(a) : slots;
  if (slots > 65535) return FP8G_EUNSUPPORTED;
  const int64_t sets = cdiv64(a.n, 16 * R) * tiles, blocks = cdiv64(a.k, 128 * U);
  if constexpr (TX < 8 || R > 1) {  // the others are for few row sets
    // Rows for every place of the CUs, and a tile's activations fit LDS: whole rows per wave.
    const int64_t x_bytes = (blocks * (256 * U) + 1023) / 1024 * 1024 * TX;
    if (sets >= kStreamSets && x_bytes <= kStreamBytes) {
      using L = W4StreamRing<Z, G, R, U>;
      const int64_t row_sets = cdiv64(a.n, 16 * R);
      a.reps = int(std::max<int64_t>(1, sets / (kW4Waves * kStreamWorkgroups)));
      const int lds = kW4Waves * L::kWave + int(x_bytes);
      hipLaunchKernelGGL((w4_stream_kernel<FMT, Z, G, TX, R, U, ROUTED>),
                         dim3(unsigned(cdiv64(row_sets, kW4Waves * a.reps)), unsigned(slots)),
                         dim3(kW4Waves * kWave), lds, s, a);
      return hipGetLastError() == hipSuccess ? FP8G_OK : FP8G_ELAUNCH;
    }
  }
  int lks = sets <= kSplit8 ? 3 : sets <= kSplit4 ? 2 : sets < kStreamSets ? 1 : 0;
  while ((1 << lks) > std::max<int64_t>(1, blocks)) --lks;
  const int waves = lks == 3 ? 8 : 4;
  a.split_log2 = lks;
  const int lds = waves * W4Ring<Z, G, TX, R, U>::kWave;
  hipLaunchKernelGGL((w4_kernel<FMT, Z, G, TX, R, U, ROUTED>),
                     dim3(unsigned(cdiv64(a.n, (waves >> lks) * 16 * R)), unsigned(slots)),
                     dim3(waves * kWave), lds, s, a);
  return hipGetLastError() == hipSuccess ? FP8G_OK : FP8G_ELAUNCH;
}

template <int FMT, bool Z, int G, bool ROUTED>
int launch_tiles(const W4Args& a, hipStream_t s) {
  if (ROUTED && (a.experts > kW4MaxExperts || a.m > kW4MaxPairs)) return FP8G_EUNSUPPORTED;
  // 128-column steps of a block: two hide more of a wave's latency (one token, 4096 x 7168: 6.4 us, 6.7 with one; with
  // groups of 32 6.3 and 6.8; 8 experts of 4096 x 2048: 11.5 and 13.2).  For 16 tokens the rings would not fit LDS.
  constexpr int kSteps = 2;
  // Tokens a tile.  One, with more than one per expert unlikely (one token, 65536 x 1024: 9.1 us, 9.5 by tiles of 4;
  // 8 experts of 4096 x 2048: 11.5 and 12.0).  Up to 4: four (4 tokens, 4096 x 7168: 6.5 us, 8.6 by tiles of 16; 64
  // pairs with 64 experts of 4096 x 2048: 53.7 and 60.9).  Else 16 of 32 rows: a second tile decodes the matrix again
  // (16 tokens, 4096 x 7168: 7.9 us, 13.5 by tiles of 4; 128 experts with 4 tokens each on average 293, 451 by 4).
  if (ROUTED ? a.m <= a.experts / 8 : a.m == 1) return launch_kernel<FMT, Z, G, 1, 1, kSteps, ROUTED>(a, s);
  if (ROUTED ? a.m <= a.experts : a.m <= 4) return launch_kernel<FMT, Z, G, 4, 1, kSteps, ROUTED>(a, s);
  // But the smallest tiles and 16 rows as long as one workgroup for each takes them all; then a wave's chain is what
  // counts.  By 4, 8 and 16 tokens: 16 tokens, 1024 x 7168: 5.5, -, 6.5; 5 tokens, 2111 x 7168: 9.0, 5.8, 6.6; 8
  // tokens, 4096 x 7168: 9.0, 6.9, 7.2; beyond, 8 tokens, 4608 x 7168: -, 9.8, 8.9.  16 tokens by 16 and 32 rows:
  // 4096 x 7168 7.9 and 9.5; 4608 x 7168 11.1 and 9.6; 7168 x 16384 21.1 and 18.1.
  const int64_t row_sets = cdiv64(a.n, 16);
  if constexpr (!ROUTED) {
    if (row_sets * cdiv64(a.m, 4) <= kSplit8) return launch_kernel<FMT, Z, G, 4, 1, kSteps, false>(a, s);
    if (row_sets * cdiv64(a.m, 8) <= kSplit8) return launch_kernel<FMT, Z, G, 8, 1, kSteps, false>(a, s);
  }
  if (row_sets * (ROUTED ? routed_tiles(a) : cdiv64(a.m, 16)) <= kSplit8)
    return launch_kernel<FMT, Z, G, 16, 1, 1, ROUTED>(a, s);
  return launch_kernel<FMT, Z, G, 16, 2, 1, ROUTED>(a, s);
}

template <int FMT, bool Z>
int launch_group(const W4Args& a, int group, hipStream_t s) {
  if (a.expert_idx)
    return group == 32 ? launch_tiles<FMT, Z, 32, true>(a, s)
           : group == 64 ? launch_tiles<FMT, Z, 64, true>(a, s)
                         : launch_tiles<FMT, Z, 128, true>(a, s);
  return group == 32 ? launch_tiles<FMT, Z, 32, false>(a, s)
         : group == 64 ? launch_tiles<FMT, Z, 64, false>(a, s)
                       : launch_tiles<FMT, Z, 128, false>(a, s);
}

}  // namespace

template <>
int launch_w4<FP8G_W4_KIND>(const W4Args& a, int group, hipStream_t s) {
  return launch_group<FP8G_W4_KIND == 2 ? FP8G_E2M1 : FP8G_INT4, FP8G_W4_KIND == 1>(a, group, s);
}

}  // namespace host
}  // namespace fp8g
