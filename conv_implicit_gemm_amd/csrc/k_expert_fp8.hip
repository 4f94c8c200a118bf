// k_expert_fp8.hip -- e4m3 products with block scales, of one matrix or
// grouped by expert (expert_gemm.hpp).
#include "expert_gemm.hpp"

namespace ox {

int launch_expert_fp8(const ExpertArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (a.out_dt == DT_F32) return launch_expert_tile<FMT_FP8X, 64, 64, 2, 2, 2, false, false>(a, s);
  return launch_expert_tile<FMT_FP8, 64, 64, 2, 2, 2, false, false>(a, s);
}

}  // namespace ox
