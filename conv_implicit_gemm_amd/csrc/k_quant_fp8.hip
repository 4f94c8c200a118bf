// k_quant_fp8.hip -- quantisation to e4m3 with one fp32 scale per block of
// 128 along K: of one row (activations, rows optionally gathered in the order
// of an index) or of 128 rows (weights).
//
//   m = max(|finite x|, 2^-100), scale = m / 448, q = e4m3(448 * x / m)
//
// bf16 values fall on the halfway points of e4m3 often, and a product with a
// rounded 448 / m would send them either way: the quotient is corrected by its
// remainder (three more operations an element).  An fp32 quotient goes to the
// side of a halfway point that the exact one lies on, or to even where that is
// the point itself; the few elements near enough to need it are found by a
// second product (8192 rows of 4096 fp32, 168 MB: 34 us, as without; 24 rows 2.6
// us, 2.5 without).  Sixteen lanes share a row's block, eight elements
// each; the maximum crosses them with four DPP steps.  What bounds it is the
// bytes: each element is read once and its code written once (16384 gathered
// rows of 4096 bf16, 201 MB: 37 us, 5.4 TB/s; 24 rows: 2.5 us, one trip to HBM).
#include "quant_codes.hpp"

namespace ox {

namespace {

// Columns and rows of a last block run past K and R, which end below 2^31: they
// are counted in 32 bits without a sign.

// Eight elements of a row from column k (zeros from column K on).
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const QuantF8Args& a, int64_t row, uint32_t k, float (&x)[8]) {
  const int64_t at = row * a.K + k;
  const uint32_t K = (uint32_t)a.K;
  if constexpr (VEC) {
    if (k >= K) {
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
      if (k + i < K) x[i] = F32 ? ((const float*)a.X)[at + i] : bf16_to_f32(((const uint16_t*)a.X)[at + i]);
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(const QuantF8Args& a, int64_t r, uint32_t k, u32x2_t q) {
  uint8_t* y = a.Q + r * a.K + k;
  const uint32_t K = (uint32_t)a.K;
  if constexpr (VEC) {
    if (k < K) *(u32x2_t*)y = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) y[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
  }
}

// A scale per row and block.  A wave takes RW rows' four blocks (512 columns):
// all RW loads go out before the first maximum, and a block's scales of RW
// consecutive rows, which lie side by side, leave as one store.
template <bool F32, bool VEC, int RW>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(const QuantF8Args a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t K = (uint32_t)a.K, per = (K + 511) / 512;
  const uint32_t unit = blockIdx.x * (kThreads / 64) + wave, row = unit / per;
  const uint32_t k = unit % per * 512 + lane * 8;
  if ((int64_t)row * RW >= a.R) return;
  const int r0 = (int)row * RW, rows = min(RW, a.R - r0);
  int src[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int r = r0 + min(i, rows - 1);
    src[i] = __builtin_amdgcn_readfirstlane(a.index ? a.index[r] : r);
  }
  float x[RW][8];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    // (an index outside X reads row 0 and is then zeroed; X may have no row)
    const bool in = src[i] >= 0 && src[i] < a.rows;
    if (a.rows > 0) load8<F32, VEC>(a, in ? src[i] : 0, k, x[i]);
    if (!in) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = 0.0f;
    }
  }
  float sc[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const uint32_t bits = max16(amax8<false>(x[i]));
    float m;
    u32x2_t q;
    if (bits >= kInfBits) {                                    // (all sixteen lanes agree)
      m = block_max(max16(amax8<true>(x[i])));
      q = codes8<F32, true>(x[i], m);
    } else {
      m = block_max(bits);
      q = codes8<F32, false>(x[i], m);
    }
    sc[i] = m / kMax;
    if (k < K && i < rows) store8<VEC>(a, r0 + i, k, q);
  }
  if (k < K && (lane & 15) == 0) {
    float* s = a.scales + (int64_t)(k >> 7) * a.R + r0;
    if (RW == 4 && a.R % 4 == 0 && (uintptr_t)a.scales % 16 == 0) {
      *(f32x4_t*)s = f32x4_t{sc[0], sc[1 % RW], sc[2 % RW], sc[3 % RW]};
    } else {
#pragma unroll
      for (int i = 0; i < RW; ++i)
        if (i < rows) s[i] = sc[i];
    }
  }
}

// A scale per 128 x 128: one block of threads each, its values in registers.
template <bool F32, bool VEC>
__global__ __launch_bounds__(kThreads) void quant_tiles_kernel(const QuantF8Args a) {
  __shared__ uint32_t part[2][kThreads / 64];
  const uint32_t R = (uint32_t)a.R, kb = ((uint32_t)a.K + 127) / 128;
  const uint32_t rb = blockIdx.x / kb, b = blockIdx.x - rb * kb;
  const uint32_t k = b * 128 + (threadIdx.x & 15) * 8, r0 = rb * 128 + (threadIdx.x >> 4);
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + 16 * i < R) {
      load8<F32, VEC>(a, r0 + 16 * i, k, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = 0.0f;
    }
  }
  uint32_t bits = 0;
  int pass = 0;
  for (; pass < 2; ++pass) {
    bits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) bits = max(bits, pass ? amax8<true>(x[i]) : amax8<false>(x[i]));
    bits = max16(bits);
    bits = max(bits, (uint32_t)__shfl_xor((int)bits, 16));
    bits = max(bits, (uint32_t)__shfl_xor((int)bits, 32));
    if ((threadIdx.x & 63) == 0) part[pass][threadIdx.x >> 6] = bits;
    __syncthreads();
    bits = max(max(part[pass][0], part[pass][1]), max(part[pass][2], part[pass][3]));
    if (bits < kInfBits) break;
  }
  const float m = block_max(bits);
  if (threadIdx.x == 0) a.scales[(int64_t)rb * kb + b] = m / kMax;
  const bool infinite = !F32 || pass > 0;      // (bf16 takes one form for all: infinities cost it two operations)
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + 16 * i < R)
      store8<VEC>(a, r0 + 16 * i, k, infinite ? codes8<F32, true>(x[i], m) : codes8<F32, false>(x[i], m));
}

template <bool F32, bool VEC>
int launch(const QuantF8Args& a, hipStream_t s) {
  if (a.block_rows == 1) {
    // four rows a wave once that still gives every CU 16 waves
    const int64_t R = a.R, per = ((int64_t)a.K + 511) / 512;
    const int rw = R * per >= 4 * 256 * 16 ? 4 : 1;
    const int64_t blocks = ((R + rw - 1) / rw * per + kThreads / 64 - 1) / (kThreads / 64);
    if (!fits_one_launch(blocks, kThreads)) return kNoGrid;
    if (rw == 4) hipLaunchKernelGGL((quant_rows_kernel<F32, VEC, 4>), dim3((uint32_t)blocks), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((quant_rows_kernel<F32, VEC, 1>), dim3((uint32_t)blocks), dim3(kThreads), 0, s, a);
  } else {
    const int64_t blocks = ((int64_t)a.R + 127) / 128 * (((int64_t)a.K + 127) / 128);
    if (!fits_one_launch(blocks, kThreads)) return kNoGrid;
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
