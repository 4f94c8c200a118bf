// k_expert_f32.hip -- fp32 products grouped by expert, on the tile engine:
// each 64 x 64 block finds its expert and row range from the device offsets
// and runs the engine's K loop over that expert's weights.
#include "expert_gemm.hpp"

namespace ox {

namespace {

template <bool KN>
__global__ __launch_bounds__(kThreads) void expert_f32_kernel(const ExpertArgs a) {
  constexpr int BM = 64, BN = 64, BKU = 2;
  __shared__ __attribute__((aligned(16))) char smem[2 * (BM + BN) * Lds<BKU>::ROWB];
  zero_outside(a);
  const int NT = (a.N + BN - 1) / BN;
  const int total = expert_tiles<BM>(a);
  if ((int64_t)blockIdx.x >= (int64_t)total * NT) return;
  int ti, nt;
  tile_order(xcd_tile(blockIdx.x, total * NT), total, NT, ti, nt);
  const ExpertTile t = expert_tile<BM>(a, ti);
  const int n0 = nt * BN;
  const float* B = (const float*)a.B + (int64_t)t.e * a.N * a.K;

  LoadRowK<DT_F32, BM, BKU> la;
  la.init((const float*)a.A, a.K, t.row0, t.row0 + t.rows, a.K, a.vec);
  f32x4_t acc[BM / 32][BN / 32];
#pragma unroll
  for (int i = 0; i < BM / 32; ++i)
#pragma unroll
    for (int j = 0; j < BN / 32; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if constexpr (KN) {
    LoadColK<DT_F32, BN, BKU> lb;
    const int n = n0 + threadIdx.x % BN;
    lb.init_col(B + n, n < a.N, a.N, a.K);
    engine_mainloop<DT_F32, BM, BN, BKU>(la, lb, a.K, smem, acc);
  } else {
    LoadRowK<DT_F32, BN, BKU> lb;
    lb.init(B, a.K, n0, a.N, a.K, a.vec);
    engine_mainloop<DT_F32, BM, BN, BKU>(la, lb, a.K, smem, acc);
  }
  float* Y = (float*)a.Y;
  const float* bias = a.bias ? (const float*)a.bias + (int64_t)t.e * a.N : nullptr;
  float bc[BN / 32];
#pragma unroll
  for (int fn = 0; fn < BN / 32; ++fn) bc[fn] = bias ? bias[min(n0 + lane_col<BN>(fn), a.N - 1)] : 0.0f;
  wait_vmem();
  with_act(a.act, [&](auto act) {
    for_each_result_fn<BM, BN>(acc, [&](int fn, int r, int c, float v) {
      if (r < t.rows && n0 + c < a.N)
        Y[(int64_t)(t.row0 + r) * a.N + n0 + c] = act_c<decltype(act)::value>(v + bc[fn]);
    });
  });
}

}  // namespace

int launch_expert_f32(const ExpertArgs& a, void* stream) {
  const int64_t blocks = expert_tile_bound(a, 64) * ((a.N + 63) / 64);
  if (blocks >= ((int64_t)1 << 31)) return (int)hipErrorInvalidValue;
  const dim3 g((uint32_t)blocks), b(kThreads);
  if (a.kn) hipLaunchKernelGGL((expert_f32_kernel<true>), g, b, 0, (hipStream_t)stream, a);
  else hipLaunchKernelGGL((expert_f32_kernel<false>), g, b, 0, (hipStream_t)stream, a);
  return (int)hipGetLastError();
}

}  // namespace ox
