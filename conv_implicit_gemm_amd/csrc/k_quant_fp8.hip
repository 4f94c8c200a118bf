// k_quant_fp8.hip -- quantisation to e4m3 with one fp32 scale per block of
// 128 along K: of one row (activations, rows optionally gathered in the order
// of an index) or of 128 rows (weights).
//
//   m = max(|finite x|, 2^-100), scale = m / 448, q = e4m3(x * (448 / m))
//
// One correctly rounded division per block; the elements are multiplied by
// the rounded 448 / m.  Sixteen lanes share a row's block, eight elements
// each; the maximum crosses them with four DPP steps.
#include "engine.hpp"

namespace ox {

namespace {

constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100: below it 448 / m would leave fp32
constexpr float kMax = 448.0f;

// Eight elements of a row from column k (zeros from column K on).
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const QuantF8Args& a, int row, int k, float (&x)[8]) {
  const int64_t at = (int64_t)row * a.K + k;
  if constexpr (VEC) {
    if (k >= a.K) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    } else if constexpr (F32) {
      const f32x4_t u = *(const f32x4_t*)((const float*)a.X + at), v = *(const f32x4_t*)((const float*)a.X + at + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = u[i];
        x[i + 4] = v[i];
      }
    } else {
      const u32x4_t u = *(const u32x4_t*)((const uint16_t*)a.X + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = 0.0f;
      if (k + i < a.K) x[i] = F32 ? ((const float*)a.X)[at + i] : bf16_to_f32(((const uint16_t*)a.X)[at + i]);
    }
  }
}

// Largest magnitude; fmaxf passes over a NaN.  FINITE: infinities are passed over too.
template <bool FINITE>
__device__ __forceinline__ float amax8(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = fabsf(x[i]);
    m = fmaxf(m, FINITE && v == __builtin_inff() ? 0.0f : v);
  }
  return m;
}

// the maximum over the sixteen lanes of a row's block
__device__ __forceinline__ float max16(float m) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
  return m;
}

// Eight codes.  An infinite product is an infinite x: +-448.
__device__ __forceinline__ u32x2_t codes8(const float (&x)[8], float r) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = x[i] * r;
    if (__builtin_isinf(v[i])) v[i] = __builtin_copysignf(kMax, v[i]);
  }
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  return u32x2_t{(uint32_t)lo, (uint32_t)hi};
}

template <bool VEC>
__device__ __forceinline__ void store8(const QuantF8Args& a, int r, int k, u32x2_t q) {
  uint8_t* y = a.Q + (int64_t)r * a.K + k;
  if constexpr (VEC) {
    if (k < a.K) *(u32x2_t*)y = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < a.K) y[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
  }
}

// A scale per row and block: each wave takes one row's four blocks (512
// columns).
template <bool F32, bool VEC>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(const QuantF8Args a) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int per = (a.K + 511) / 512;
  const int r = (int)(unit / per), k = (int)(unit - (int64_t)r * per) * 512 + lane * 8;
  if (r >= a.R) return;
  const int src = a.index ? a.index[r] : r;
  float x[8];
  if (src >= 0 && src < a.rows) {
    load8<F32, VEC>(a, src, k, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
  }
  float m = max16(amax8<false>(x));
  if (m == __builtin_inff()) m = max16(amax8<true>(x));   // (all sixteen lanes agree)
  m = fmaxf(m, kTiny);
  if (k < a.K) {
    if ((lane & 15) == 0) a.scales[(int64_t)(k >> 7) * a.R + r] = m / kMax;
    store8<VEC>(a, r, k, codes8(x, kMax / m));
  }
}

// A scale per 128 x 128: one block of threads each, its values in registers.
template <bool F32, bool VEC>
__global__ __launch_bounds__(kThreads) void quant_tiles_kernel(const QuantF8Args a) {
  __shared__ float part[2][kThreads / 64];
  const int kb = (a.K + 127) / 128;
  const int rb = blockIdx.x / kb, b = blockIdx.x - rb * kb;
  const int k = b * 128 + (threadIdx.x & 15) * 8, r0 = rb * 128 + (threadIdx.x >> 4);
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + 16 * i < a.R) {
      load8<F32, VEC>(a, r0 + 16 * i, k, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = 0.0f;
    }
  }
  float m = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, pass ? amax8<true>(x[i]) : amax8<false>(x[i]));
    m = max16(m);
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    if ((threadIdx.x & 63) == 0) part[pass][threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(part[pass][0], part[pass][1]), fmaxf(part[pass][2], part[pass][3]));
    if (m != __builtin_inff()) break;
  }
  m = fmaxf(m, kTiny);
  if (threadIdx.x == 0) a.scales[(int64_t)rb * kb + b] = m / kMax;
  const float r = kMax / m;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < a.R) store8<VEC>(a, r0 + 16 * i, k, codes8(x[i], r));
}

template <bool F32, bool VEC>
int launch(const QuantF8Args& a, hipStream_t s) {
  const int64_t units = (int64_t)a.R * ((a.K + 511) / 512);
  if (a.block_rows == 1) {
    const int64_t blocks = (units + kThreads / 64 - 1) / (kThreads / 64);
    hipLaunchKernelGGL((quant_rows_kernel<F32, VEC>), dim3((uint32_t)blocks), dim3(kThreads), 0, s, a);
  } else {
    const int64_t blocks = (int64_t)((a.R + 127) / 128) * ((a.K + 127) / 128);
    hipLaunchKernelGGL((quant_tiles_kernel<F32, VEC>), dim3((uint32_t)blocks), dim3(kThreads), 0, s, a);
  }
  return (int)hipGetLastError();
}

}  // namespace

int launch_quantize_fp8(const QuantF8Args& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (a.dt == DT_F32) return a.vec ? launch<true, true>(a, s) : launch<true, false>(a, s);
  return a.vec ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace ox
