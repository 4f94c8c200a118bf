// quant_codes.hpp -- the arithmetic of 8-bit codes with scales, shared by the
// quantisation and the norm kernels: largest magnitudes, and the codes of exact
// quotients (e4m3: 448 x / m, int8: 127 x / m, m the largest magnitude of a
// block or a row), round half to even.
#pragma once

#include "engine.hpp"

namespace ox {

constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100: below it 448 / m would leave fp32
constexpr float kMax = 448.0f;

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

// Eight codes of 448 x / m for |x| <= m that are themselves results of fp32
// arithmetic: the quotient to one rounding (r + low is 448 / m to 48 bits), which
// the exact one of a rounded x need not go beyond, without a branch.
__device__ __forceinline__ u32x2_t codes8_of_result(const float (&x)[8], float m) {
  const float r = kMax / m, low = __builtin_fmaf(-r, m, kMax) * (r * 0.002232142857f);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(x[i], r, x[i] * low);
  return u32x2_t{convert4(v[0], v[1], v[2], v[3]), convert4(v[4], v[5], v[6], v[7])};
}

// --- int8

// The integer nearest to the exact quotient 127 x / m (half to even; finite
// |x| <= m, so at most 127 in magnitude), from a first answer n that is off by
// one at most: the remainder of x * 127/128 over m / 128 (both stay in range),
// against m / 256.  x * 127/128 is p + e exactly.  p - n m / 128 is exact (a
// multiple of ulp(m) / 128 below m / 255, or with n = 1 a difference of
// neighbours; a quotient below 1/2 that came as 1 goes down in any case); so is
// its distance to m / 256 where the two are within a factor of two of each
// other, and adding e then keeps the sign.
__device__ __forceinline__ float exact_int8(float x, float m, float n) {
  const float p = x * 0.9921875f, e = __builtin_fmaf(x, 0.9921875f, -p);
  const float m7 = m * 0.0078125f, d = __builtin_fmaf(-n, m7, p);
  const float up = (d - 0.5f * m7) + e, down = (-d - 0.5f * m7) - e;      // past n + 1/2, past n - 1/2
  const bool odd = ((int)n & 1) != 0;
  if (up > 0.0f || (up == 0.0f && odd)) return n + 1.0f;
  if (down > 0.0f || (down == 0.0f && odd)) return n - 1.0f;
  return n;
}

// Eight codes of |x| <= m.  r + low is 127 / m to 48 bits.  Adding 1.5 * 2^23 to x
// r leaves a nearest integer n in the low bits of a float; x r - n, exact, plus
// x low is what the quotient has beside n, and adding it rounds n to the nearest
// integer of the quotient, half to even.  For bf16 x and m no quotient is within
// 2^-18 of a halfway point without being it, and those come out as it: exact
// codes without a branch (a test for values near a halfway point and a longer
// form for those, as for fp32, is taken by 44% of the waves on bf16 data: 8192
// rows of 8192 55 us).  EXACT (fp32): what the sum cannot tell from a halfway
// point takes the longer form.  INF: an infinite x gives +-127 and a NaN 0.
template <bool EXACT, bool INF>
__device__ __forceinline__ u32x2_t codes8_i8(const float (&x)[8], float m) {
  constexpr float kMagic = 12582912.0f;
  const float r = 127.0f / m, low = __builtin_fmaf(-r, m, 127.0f) * (r * 0.007874016f);
  float t[8], off = 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = __builtin_fmaf(x[i], r, kMagic);
    const float f = __builtin_fmaf(x[i], low, __builtin_fmaf(x[i], r, kMagic - n));
    t[i] = n + f;
    if constexpr (EXACT && !INF) off = fminf(off, fabsf(fabsf(f) - 0.5f));
  }
  // (r * 2^-24 leaves the normal numbers for a large m)
  if (INF || m > 0x1p64f || (EXACT && off < 0x1p-22f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float n = rintf(x[i] * r);
      if (INF && __builtin_isinf(x[i])) n = __builtin_copysignf(127.0f, x[i]);
      else if (INF && __builtin_isnan(x[i])) n = 0.0f;
      else n = exact_int8(x[i], m, n);
      t[i] = n + kMagic;
    }
  }
  u32x2_t q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // the low bytes of four floats
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 1]), __float_as_uint(t[4 * h]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 3]), __float_as_uint(t[4 * h + 2]), 0x04000c0cu);
    q[h] = lo | hi;
  }
  return q;
}

}  // namespace ox
