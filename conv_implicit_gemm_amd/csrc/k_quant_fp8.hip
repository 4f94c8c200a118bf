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
#include "engine.hpp"

namespace ox {

namespace {

constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100: below it 448 / m would leave fp32
constexpr float kMax = 448.0f;

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

// Largest magnitude, as the bits of a float: magnitudes order as their bits
// do, with infinities and NaN above every number.  FINITE: those are passed
// over.
constexpr uint32_t kInfBits = 0x7f800000u;
template <bool FINITE>
__device__ __forceinline__ uint32_t amax8(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = __float_as_uint(x[i]) & 0x7fffffffu;
    m = max(m, FINITE && v >= kInfBits ? 0u : v);
  }
  return m;
}

// the maximum over the sixteen lanes of a row's block
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  // lane ^ 1, ^ 2 within quads, then the mirrored half row and row (every
  // lane of a quad, of a half row, already agrees)
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xf, 0xf, true));    // quad_perm 1,0,3,2
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xf, 0xf, true));    // quad_perm 2,3,0,1
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xf, 0xf, true));   // row_half_mirror
  return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xf, 0xf, true));   // row_mirror
}

// m of a block from the bits of its largest finite magnitude
__device__ __forceinline__ float block_max(uint32_t bits) { return fmaxf(__uint_as_float(bits), kTiny); }

__device__ __forceinline__ uint32_t convert4(float a, float b, float c, float d) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}

// The codes of N elements, of the exact quotients 448 x / m.  v = x * r is off by the
// rounding of r = 448 / m; the remainder 448 x - v m, taken 2^-9 times (m / 512
// is exact and stays in range), over m / 512 is what it lacks, and the corrected
// v is the quotient rounded to fp32.  For bf16 0.875 x is exact too, and a
// quotient that is no halfway point h is too far from one to be rounded to it
// (448 x and h m, of 16 bits, differ by a unit at least).  For fp32 (7/8 of 24
// bits) the error of 0.875 x, exact in turn, is carried along, and a quotient
// can be nearer to h than fp32 tells: where v may be a halfway point (5 bits, 19
// zeros behind them) and its remainder is not zero, v moves one step the
// remainder's way.  INF: an infinite x gives +-448 (asked for only where the
// block holds one; finite quotients cannot leave the format, |448 x / m| <= 448
// but for roundings that the conversion takes back).
template <bool F32, bool INF, int N>
__device__ __forceinline__ void exact_codes(const float* x, float m, float r, uint32_t* q) {
  const float m9 = m * 0.001953125f, r9 = r * 1.142857143f;
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float v0 = x[i] * r, p = x[i] * 0.875f;
    if constexpr (F32) {
      const float e = __builtin_fmaf(x[i], 0.875f, -p);
      v[i] = __builtin_fmaf(__builtin_fmaf(-v0, m9, p) + e, r9, v0);
      const uint32_t u = __float_as_uint(v[i]);
      const float d = __builtin_fmaf(-v[i], m9, p) + e;
      const uint32_t to = ((__float_as_uint(d) ^ u) >> 31) ? u - 1 : u + 1;
      if ((u & 0x7ffffu) == 0 && d != 0.0f && (u << 1) != 0) v[i] = __uint_as_float(to);
    } else {
      v[i] = __builtin_fmaf(__builtin_fmaf(-v0, m9, p), r9, v0);
    }
    if (INF && __builtin_isinf(x[i])) v[i] = __builtin_copysignf(kMax, x[i]);
  }
#pragma unroll
  for (int i = 0; i < N; i += 4) q[i / 4] = convert4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

// Eight codes.  fp32: x * r is within 2^-22 of the quotient, and numbers that far below and
// above it have the same code but for one in 2^17 or so: only it and its
// neighbours take the exact form.
template <bool F32, bool INF>
__device__ __forceinline__ u32x2_t codes8(const float (&x)[8], float m) {
  const float r = kMax / m;
  uint32_t q[2];
  if constexpr (F32 && !INF) {
    const float below = r * (1.0f - 0x1p-22f), above = r * (1.0f + 0x1p-22f);
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = x[i] * below;
      hi[i] = x[i] * above;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      q[h] = convert4(lo[4 * h], lo[4 * h + 1], lo[4 * h + 2], lo[4 * h + 3]);
      if (q[h] != convert4(hi[4 * h], hi[4 * h + 1], hi[4 * h + 2], hi[4 * h + 3]))
        exact_codes<F32, INF, 4>(x + 4 * h, m, r, q + h);
    }
  } else {
    exact_codes<F32, INF, 8>(x, m, r, q);
  }
  return u32x2_t{q[0], q[1]};
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
