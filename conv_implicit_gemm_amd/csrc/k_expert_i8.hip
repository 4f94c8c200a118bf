// k_expert_i8.hip -- int8 products with a scale for each row of both operands
// (expert_gemm.hpp).
#include "expert_gemm.hpp"

namespace ox {

namespace {

// (xN: K divided over N groups of waves)  The estimates are for the choice, which
// is within 4% of the fastest variant in 16 shapes from 1 x 4096 x 4096 to 8192^3.
// A call takes up to 40% more: operands that come from memory, sizes that end
// inside tiles and fp32 results are not in them (64x64x2: 1024 x 1024 x 2048 7.6
// us, 6.7 by the table; 1000 x 1000 x 2000 8.8 to bf16, 9.8 to fp32 with biases).
constexpr TileCost kTiles[] = {{"32x64", 32, 64, 4, 2.5, 0.31, 0.53},
                               {"64x64", 64, 64, 3, 2.5, 0.39, 0.59},
                               {"128x128", 128, 128, 2, 5.3, 0.71, 0.98},
                               {"256x256", 256, 256, 1, 11.3, 1.55, 1.55},
                               {"32x32x4", 32, 32, 2, 3.0, 0.19, 0.19},
                               {"64x64x2", 64, 64, 1, 3.0, 0.23, 0.23},
                               {"128x128x2", 128, 128, 1, 5.5, 0.57, 0.57}};

}  // namespace

int launch_expert_i8(ExpertArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  switch (pick_variant(a, 1, kTiles)) {
    case PICK_REGS: return launch_expert_tile<FMT_I8, 64, 64, 2, 2, 2, 1, false, false>(a, s);
    case PICK_REGS_LARGE: return launch_expert_tile<FMT_I8, 128, 128, 2, 4, 2, 1, false, false>(a, s);
    case PICK_STREAM: return launch_expert_stream<FMT_I8>(a, s);
    case 0: return launch_expert_tile<FMT_I8, 32, 64, 1, 4, 3, 1, true, false>(a, s);
    case 1: return launch_expert_tile<FMT_I8, 64, 64, 2, 2, 3, 1, true, false>(a, s);
    case 2: return launch_expert_tile<FMT_I8, 128, 128, 2, 4, 2, 1, true, false>(a, s);
    case 3: return launch_expert_tile<FMT_I8, 256, 256, 2, 4, 2, 1, true, false>(a, s);
    case 4: return launch_expert_tile<FMT_I8, 32, 32, 1, 2, 2, 4, true, false>(a, s);
    case 5: return launch_expert_tile<FMT_I8, 64, 64, 2, 2, 3, 2, true, false>(a, s);
    case 6: return launch_expert_tile<FMT_I8, 128, 128, 2, 4, 2, 2, true, false>(a, s);
    default: return kNoVariant;
  }
}

}  // namespace ox
