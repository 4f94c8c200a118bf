// k_expert_bf16.hip -- bf16 products grouped by expert (expert_gemm.hpp).
#include "expert_gemm.hpp"

namespace ox {

int launch_expert_bf16(const ExpertArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (a.kn) return launch_expert_tile<FMT_BF16, 64, 64, 2, 2, 2, false, true>(a, s);
  return launch_expert_tile<FMT_BF16, 64, 64, 2, 2, 2, false, false>(a, s);
}

}  // namespace ox
