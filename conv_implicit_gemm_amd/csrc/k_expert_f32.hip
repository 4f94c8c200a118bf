// k_expert_f32.hip -- fp32 products grouped by expert (expert_gemm.hpp).
#include "expert_gemm.hpp"

namespace ox {

namespace {

// (xN: K divided over N groups of waves)
constexpr TileCost kTiles[] = {{"32x64", 32, 64, 4, 2.5, 0.42, 1.25},
                               {"64x64", 64, 64, 2, 2.5, 0.60, 1.10},
                               {"128x128", 128, 128, 2, 5.3, 1.90, 3.70},
                               {"64x64x2", 64, 64, 1, 3.0, 0.56, 0.56}};

template <bool KN>
int launch(ExpertArgs& a, hipStream_t s) {
  switch (pick_variant(a, 4, kTiles)) {
    case PICK_REGS: return launch_expert_tile<FMT_F32, 64, 64, 2, 2, 2, 1, false, KN>(a, s);
    case PICK_REGS_LARGE: return launch_expert_tile<FMT_F32, 128, 128, 2, 4, 2, 1, false, KN>(a, s);
    case PICK_STREAM: return launch_expert_stream<FMT_F32>(a, s);
    case 0: return launch_expert_tile<FMT_F32, 32, 64, 1, 4, 3, 1, true, KN>(a, s);
    case 1: return launch_expert_tile<FMT_F32, 64, 64, 2, 4, 4, 1, true, KN>(a, s);
    case 2: return launch_expert_tile<FMT_F32, 128, 128, 2, 4, 2, 1, true, KN>(a, s);
    case 3: return launch_expert_tile<FMT_F32, 64, 64, 2, 2, 3, 2, true, KN>(a, s);
    default: return kNoVariant;
  }
}

}  // namespace

int launch_expert_f32(ExpertArgs& a, void* stream) {
  return a.kn ? launch<true>(a, (hipStream_t)stream) : launch<false>(a, (hipStream_t)stream);
}

}  // namespace ox
