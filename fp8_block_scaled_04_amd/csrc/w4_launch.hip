// Launches of the 4-bit product kernels; compiled once for each FP8G_W4_KIND
// (0: INT4, 1: INT4 with zero points, 2: E2M1).
#include "w4_launch.hpp"

#include <algorithm>

#include "fp8gemm.h"
#include "w4_kernel.hpp"

namespace fp8g {
namespace host {
namespace {

// 8 waves on each of 256 CUs.  k is split only as far as that needs: 8 ways,
// 4096 x 7168 (256 sets) takes 6.5 us, 4 ways 8.5, 2 ways 13, not split 22;
// the waves that split a row set also exchange its sums, so no wider split is
// made where the sets alone fill the CUs.
constexpr int kFullWaves = 2048;
// Row sets from which on a wave takes whole rows.  Measured for one token,
// whole rows against k split: 1024 sets (16384 x 4096) 13.8 and 10.4 us, 1536
// (24576 x 1536) 7.6 and 8.2, 2048 (32768 x 2048) 9.5 and 10.5, 4096 (65536 x
// 1024) 9.9 and 10.7; eight experts of 4096 x 2048 (2048) 11.6 and 13.5.
constexpr int kStreamSets = 2048;
constexpr int kStreamBytes = 64 * 1024;   // activations of a streaming workgroup, at most
constexpr int kStreamWorkgroups = 2048;   // workgroups a long stream is dealt to

int64_t cdiv64(int64_t x, int64_t y) { return (x + y - 1) / y; }

template <int FMT, bool Z, int G, int TX, int R, int U, bool ROUTED>
int launch_kernel(W4Args a, hipStream_t s) {
  a.by_pair = ROUTED && a.m <= a.experts;
  const int64_t slots = !ROUTED ? cdiv64(a.m, TX) : a.by_pair ? a.m : int64_t(a.experts) + 1;
  if (slots > 65535) return FP8G_EUNSUPPORTED;
  const int64_t sets = cdiv64(a.n, 16 * R) * slots, blocks = cdiv64(a.k, 128 * U);
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
  // k is split over the waves of a workgroup until there is a wave for each of the CUs' places
  int lks = 0;
  while (lks < 3 && (sets << lks) < kFullWaves && (2 << lks) <= blocks) ++lks;
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
  constexpr int kSteps = G == 32 ? 1 : 2;  // 128-column steps of a block: four groups or fewer
  // Tokens per expert: hardly ever above 1, 4 with 1/8, 1 on average (a second tile reads the matrix again: 128
  // experts with 4 tokens each on average took 451 us by tiles of 4, 293 by tiles of 16).
  if (ROUTED ? a.m <= a.experts / 8 : a.m == 1) return launch_kernel<FMT, Z, G, 1, 1, kSteps, ROUTED>(a, s);
  if (ROUTED ? a.m <= a.experts : a.m <= 4) return launch_kernel<FMT, Z, G, 4, 1, kSteps, ROUTED>(a, s);
  const int64_t sets = cdiv64(a.n, 32) * (ROUTED ? a.experts : cdiv64(a.m, 16));
  // 32 rows a wave where there are enough (16 tokens, 7168 x 16384: 21 us, 26 with 16 rows), else 16 (5 tokens,
  // 2111 x 7168: 6.8 us, 8.5 with 32)
  if (sets * kW4Waves < kFullWaves / 2) return launch_kernel<FMT, Z, G, 16, 1, 1, ROUTED>(a, s);
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
