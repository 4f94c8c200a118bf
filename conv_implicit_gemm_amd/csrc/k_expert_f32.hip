// k_expert_f32.hip -- fp32 products grouped by expert (expert_gemm.hpp).
#include "expert_gemm.hpp"

namespace ox {

namespace {

constexpr TileCost kTiles[] = {{32, 64, 4, 2.5, 0.42, 1.25},
                               {64, 64, 3, 2.5, 0.65, 1.55},
                               {128, 128, 2, 5.3, 1.90, 3.70},
                               {64, 64, 1, 3.0, 0.56, 0.56}};      // K in two groups

template <bool KN>
int launch(const ExpertArgs& a, hipStream_t s) {
  if (!a.vec) return launch_expert_tile<FMT_F32, 64, 64, 2, 2, 2, 1, false, KN>(a, s);
  if constexpr (!KN) {
    if (stream_pays(a, 4)) return launch_expert_stream<FMT_F32>(a, s);
  }
  switch (best_tile(a, 4, kTiles)) {
    case 0: return launch_expert_tile<FMT_F32, 32, 64, 1, 4, 3, 1, true, KN>(a, s);
    case 1: return launch_expert_tile<FMT_F32, 64, 64, 2, 4, 4, 1, true, KN>(a, s);
    case 3: return launch_expert_tile<FMT_F32, 64, 64, 2, 2, 3, 2, true, KN>(a, s);
    default: return launch_expert_tile<FMT_F32, 128, 128, 2, 4, 2, 1, true, KN>(a, s);
  }
}

}  // namespace

int launch_expert_f32(const ExpertArgs& a, void* stream) {
  return a.kn ? launch<true>(a, (hipStream_t)stream) : launch<false>(a, (hipStream_t)stream);
}

}  // namespace ox
