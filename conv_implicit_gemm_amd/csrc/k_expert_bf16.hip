// k_expert_bf16.hip -- bf16 products grouped by expert (expert_gemm.hpp).
#include "expert_gemm.hpp"

namespace ox {

namespace {

// (xN: K divided over N groups of waves)
constexpr TileCost kTiles[] = {{"32x64", 32, 64, 4, 2.5, 0.30, 0.60},
                               {"64x64", 64, 64, 3, 2.5, 0.42, 0.57},
                               {"128x128", 128, 128, 2, 5.3, 0.75, 1.16},
                               {"256x128", 256, 128, 1, 8.0, 0.91, 0.91},
                               {"256x256", 256, 256, 1, 11.3, 1.65, 1.65},
                               {"32x32x4", 32, 32, 2, 3.0, 0.19, 0.22},
                               {"64x64x2", 64, 64, 1, 3.0, 0.285, 0.285},
                               {"128x128x2", 128, 128, 1, 5.5, 0.70, 0.70}};

template <bool KN>
int launch(ExpertArgs& a, hipStream_t s) {
  const int p = pick_variant(a, 2, kTiles);
  // [K, N] weights that take longer to read than to multiply: blocks as wide
  // as 256 bytes of their rows (64 experts of 2048 x 1024, 4003 rows: 62 us, 71
  // on 64 x 64; 300 rows over 16 of 2048 x 2000: 24.1 us, 24.9 on 64 x 64; 1000
  // over 16 of 4096 x 4096: 125 us, 119 on 256 x 256; 64 over 4 of 4096 x 4096,
  // the worst found: 30.1 us, 25.7 on 32 x 64)
  if constexpr (KN)
    if (a.force ? !strcmp(a.force, "64x128") && a.vec : p >= 0 && tile_time(a, 2, kTiles[p]) < weights_time(a, 2)) {
      a.chosen = "64x128";
      return launch_expert_tile<FMT_BF16, 64, 128, 2, 4, 3, 1, true, KN>(a, s);
    }
  switch (p) {
    case PICK_REGS: return launch_expert_tile<FMT_BF16, 64, 64, 2, 2, 2, 1, false, KN>(a, s);
    case PICK_REGS_LARGE: return launch_expert_tile<FMT_BF16, 128, 128, 2, 4, 2, 1, false, KN>(a, s);
    case PICK_STREAM: return launch_expert_stream<FMT_BF16>(a, s);
    case 0: return launch_expert_tile<FMT_BF16, 32, 64, 1, 4, 3, 1, true, KN>(a, s);
    case 1: return launch_expert_tile<FMT_BF16, 64, 64, 2, 2, 3, 1, true, KN>(a, s);
    case 2: return launch_expert_tile<FMT_BF16, 128, 128, 2, 4, 2, 1, true, KN>(a, s);
    case 3: return launch_expert_tile<FMT_BF16, 256, 128, 4, 2, 3, 1, true, KN>(a, s);
    case 4: return launch_expert_tile<FMT_BF16, 256, 256, 2, 4, 2, 1, true, KN>(a, s);
    case 5: return launch_expert_tile<FMT_BF16, 32, 32, 1, 2, 2, 4, true, KN>(a, s);
    case 6: return launch_expert_tile<FMT_BF16, 64, 64, 2, 2, 3, 2, true, KN>(a, s);
    case 7: return launch_expert_tile<FMT_BF16, 128, 128, 2, 4, 2, 2, true, KN>(a, s);
    default: return kNoVariant;
  }
}

}  // namespace

int launch_expert_bf16(ExpertArgs& a, void* stream) {
  return a.kn ? launch<true>(a, (hipStream_t)stream) : launch<false>(a, (hipStream_t)stream);
}

}  // namespace ox
