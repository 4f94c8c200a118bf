// k_expert_fp8.hip -- e4m3 products with block scales, of one matrix or
// grouped by expert (expert_gemm.hpp).
#include "expert_gemm.hpp"

namespace ox {

namespace {

// (xN: K divided over N groups of waves)
// codes straight to the matrix unit (bf16 results)
constexpr TileCost kCodes[] = {{"32x64", 32, 64, 4, 2.5, 0.30, 0.60},
                               {"64x64", 64, 64, 3, 2.5, 0.42, 0.57},
                               {"128x128", 128, 128, 2, 5.3, 0.69, 1.07},
                               {"256x256", 256, 256, 1, 11.3, 1.68, 1.68},
                               {"32x32x4", 32, 32, 2, 3.0, 0.19, 0.22},
                               {"64x64x2", 64, 64, 1, 3.0, 0.285, 0.285},
                               {"128x128x2", 128, 128, 1, 5.5, 0.60, 0.60}};
// codes widened to bf16 (fp32 results)
constexpr TileCost kWide[] = {{"32x64", 32, 64, 4, 2.5, 0.50, 0.90},
                              {"64x64", 64, 64, 3, 2.5, 0.63, 0.93},
                              {"128x128", 128, 128, 2, 5.3, 1.00, 2.20},
                              {"128x256", 128, 256, 1, 6.0, 1.90, 1.90},
                              {"32x32x4", 32, 32, 2, 3.0, 0.28, 0.35},
                              {"64x64x2", 64, 64, 1, 3.0, 0.54, 0.54},
                              {"128x128x2", 128, 128, 1, 5.5, 1.00, 1.00}};

template <int FMT>
int launch(ExpertArgs& a, hipStream_t s) {
  switch (FMT == FMT_FP8 ? pick_variant(a, 1, kCodes) : pick_variant(a, 1, kWide)) {
    case PICK_REGS: return launch_expert_tile<FMT, 64, 64, 2, 2, 2, 1, false, false>(a, s);
    case PICK_REGS_LARGE: return launch_expert_tile<FMT, 128, 128, 2, 4, 2, 1, false, false>(a, s);
    case PICK_STREAM: return launch_expert_stream<FMT>(a, s);
    case 0: return launch_expert_tile<FMT, 32, 64, 1, 4, 3, 1, true, false>(a, s);
    case 1: return launch_expert_tile<FMT, 64, 64, 2, 2, 3, 1, true, false>(a, s);
    case 2: return launch_expert_tile<FMT, 128, 128, 2, 4, 2, 1, true, false>(a, s);
    case 3:
      if constexpr (FMT == FMT_FP8) return launch_expert_tile<FMT, 256, 256, 2, 4, 2, 1, true, false>(a, s);
      else return launch_expert_tile<FMT, 128, 256, 2, 4, 2, 1, true, false>(a, s);
    case 4: return launch_expert_tile<FMT, 32, 32, 1, 2, 2, 4, true, false>(a, s);
    case 5: return launch_expert_tile<FMT, 64, 64, 2, 2, 3, 2, true, false>(a, s);
    case 6: return launch_expert_tile<FMT, 128, 128, 2, 4, 2, 2, true, false>(a, s);
    default: return kNoVariant;
  }
}

}  // namespace

int launch_expert_fp8(ExpertArgs& a, void* stream) {
  return a.out_dt == DT_F32 ? launch<FMT_FP8X>(a, (hipStream_t)stream) : launch<FMT_FP8>(a, (hipStream_t)stream);
}

}  // namespace ox
