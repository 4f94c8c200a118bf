// k_norm.hip -- kernels whose threads hold a row between them: the RMS norm with
// the residual's addition and results of 8 bits with scales, and the
// quantisation to int8 with a scale per row.
//
//   s = x + r,  z = s * gamma,  y = z / sqrt(mean(s^2) + eps)
//   same type:  y, rounded once
//   e4m3:       per block of 128, m = max|y|: scale m / 448, code 448 y / m
//   int8:       per row, m = max|y|: scale m / 127, code rint(127 y / m)
//
// A code does not need the norm: 448 y / m = 448 z / max|z|.  So the sum of
// squares and the largest |z| are found in one pass and cross the row's threads
// together, behind one barrier, and the codes are those of exact quotients of z.
// Where that shortcut does not hold (infinities or NaN in the row, magnitudes
// next to the ends of fp32) the codes are taken of y itself.
//
// A row's TPR threads hold eight neighbouring elements C times over; short rows
// have a wave each, longer ones a block of threads.  What bounds it is the bytes,
// each read or written once: 8192 rows of 4096 bf16, residual, norm and e4m3
// codes (236 MB) 45 us, 5.2 TB/s; int8 codes of 8192 rows of 8192 bf16 (201 MB)
// 38.9 us, 5.2 TB/s, what a large copy reaches.  24 rows are one trip to HBM, a
// barrier and a store: 3.4 and 2.8 us.  Blocks that stay and load the next row
// ahead were no faster (47.7 us).
//
// Rows of up to 16384 elements lie in registers, and so do norms of bf16 rows, and
// of fp32 rows to fp32, up to 32768.  Past that 1024 threads, of 128 registers
// each, keep a part of their row in scratch memory: bf16 rows to int8 with the
// norm, 1024 of 32768 56 us (4.2 TB/s), 512 of 65536 178 us (1.3 TB/s); quantised
// alone 26 and 52 us (3.8 and 2.0 TB/s).  Rows below 512 elements leave lanes of
// their wave idle: 8192 x 4096 as 262144 rows of 128, bf16 with the norm, takes
// 101 us to bf16, 162 to e4m3 and 141 to int8, 44 to 48 as rows of 4096.
#include "quant_codes.hpp"

namespace ox {

namespace {

enum Out : int { OUT_SAME = 0, OUT_F8 = 1, OUT_I8 = 2 };

struct __attribute__((packed, aligned(1))) Bytes16 { u32x4_t v; };
struct __attribute__((packed, aligned(1))) Bytes8 { u32x2_t v; };

// Eight elements of a row as they lie in memory, and as floats.
template <bool F32>
struct Raw {
  u32x4_t v[F32 ? 2 : 1];

  // The piece at column k, or the row's last eight elements where it ends
  // before k + 8 (K >= 8): no branch, so that a row's loads go out together
  // (8192 rows of 4096: 50.6 us, 56.6 with a branch around each piece).
  __device__ __forceinline__ void load(const void* row, int k, int K) {
    const int64_t at = min(k, K - 8);
    const char* p = (const char*)row + at * (F32 ? 4 : 2);
    v[0] = ((const Bytes16*)p)->v;
    if constexpr (F32) v[1] = ((const Bytes16*)(p + 16))->v;
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        x[i] = __uint_as_float(v[0][i]);
        x[i + 4] = __uint_as_float(v[F32][i]);
      } else {
        x[2 * i] = __uint_as_float(v[0][i] << 16);
        x[2 * i + 1] = __uint_as_float(v[0][i] & 0xffff0000u);
      }
    }
  }
};
// A piece that the row ends inside of, from n of its elements (zeros behind them).
template <bool F32>
__device__ __forceinline__ void load_part(const void* row, int k, int n, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = 0.0f;
    if (i < n) x[i] = F32 ? ((const float*)row)[k + i] : bf16_to_f32(((const uint16_t*)row)[k + i]);
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, int n, const float (&x)[8]) {
  if (n >= 8) {
    if constexpr (F32) {
      float* p = (float*)base + at;
      ((Bytes16*)p)->v = u32x4_t{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
      ((Bytes16*)(p + 4))->v = u32x4_t{__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])};
    } else {
      ((Bytes16*)((uint16_t*)base + at))->v =
          u32x4_t{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (F32) ((float*)base)[at + i] = x[i];
        else ((uint16_t*)base)[at + i] = (uint16_t)pack_bf16x2(x[i], 0.0f);
      }
  }
}

__device__ __forceinline__ void store_codes(uint8_t* y, int n, u32x2_t q) {
  if (n >= 8) {
    ((Bytes8*)y)->v = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) y[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
  }
}

// over the 64 lanes of a wave, in every lane: within rows of sixteen lanes by
// DPP, then the rows' values by scalar reads
__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
  m = max16(m);
  const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)m, 0), (uint32_t)__builtin_amdgcn_readlane((int)m, 16));
  const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)m, 32), (uint32_t)__builtin_amdgcn_readlane((int)m, 48));
  return max(a, b);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xB1>(v);    // quad_perm 1,0,3,2
  v += dpp<0x4E>(v);    // quad_perm 2,3,0,1
  v += dpp<0x141>(v);   // row_half_mirror
  v += dpp<0x140>(v);   // row_mirror
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// The largest `m` and the sum of `v` over a row's threads (the waves' parts are
// added in their order).
template <int TPR>
__device__ __forceinline__ void row_reduce(float& v, uint32_t& m, float* sums, uint32_t* tops) {
  v = wave_sum(v);
  m = wave_max(m);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((threadIdx.x & 63) == 0) {
      sums[threadIdx.x >> 6] = v;
      tops[threadIdx.x >> 6] = m;
    }
    __syncthreads();
    v = 0.0f;
    m = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v += sums[i];
      m = max(m, tops[i]);
    }
  }
}

constexpr int row_threads(int TPR) { return TPR > 64 ? TPR : kThreads; }      // threads of a block

template <bool F32, int OUT, bool NORM, int TPR, int C>
__global__ __launch_bounds__(row_threads(TPR)) void row_kernel(const NormArgs a) {
  constexpr int RPB = row_threads(TPR) / TPR;      // rows of a block
  __shared__ float sums[2][TPR / 64];
  __shared__ uint32_t tops[2][TPR / 64];
  const int t = threadIdx.x % TPR;
  static_assert(TPR == 64 || RPB == 1, "a barrier is for one row");
  // (rows in the order of the blocks: a range of rows for each XCD, powers of two
  // apart, measured 5 to 15% slower)
  const uint32_t row = blockIdx.x * RPB + threadIdx.x / TPR;
  if (row >= (uint32_t)a.rows) return;             // (whole waves; rows of a block share no barrier)
  const int64_t at = (int64_t)row * a.K;
  const int64_t size = F32 ? 4 : 2;
  const char* xr = (const char*)a.X + at * size;
  const char* rr = (const char*)a.residual + at * size;
  const bool whole = a.K >= 8;                     // (else the row is part of one piece)
  float z[C][8];
  int n[C];                                        // elements of the row from this piece's first on
  Raw<F32> x[C], r[NORM ? C : 1], g[NORM ? C : 1];
#pragma unroll
  for (int c = 0; c < C; ++c) n[c] = a.K - (c * TPR + t) * 8;
  if (whole) {
#pragma unroll
    for (int c = 0; c < C; ++c) x[c].load(xr, (c * TPR + t) * 8, a.K);
    if constexpr (NORM) {
      if (a.residual) {
#pragma unroll
        for (int c = 0; c < C; ++c) r[c].load(rr, (c * TPR + t) * 8, a.K);
      }
      if (a.gamma) {
#pragma unroll
        for (int c = 0; c < C; ++c) g[c].load(a.gamma, (c * TPR + t) * 8, a.K);
      }
    }
  }
  // a piece's eight floats: zeros past the row's end
  auto floats = [&](const Raw<F32>& raw, const void* from, int c, float (&v)[8]) {
    if (n[c] >= 8) raw.widen(v);
    else load_part<F32>(from, (c * TPR + t) * 8, n[c], v);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) floats(x[c], xr, c, z[c]);
  float ss = 0.0f;
  if constexpr (NORM) {
    float v[8];
    if (a.residual) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        floats(r[c], rr, c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[c][i] += v[i];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(z[c][i], z[c][i], ss);
    if (a.sum_out) {
#pragma unroll
      for (int c = 0; c < C; ++c) store8<F32>(a.sum_out, at + (c * TPR + t) * 8, n[c], z[c]);
    }
    if (a.gamma) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        floats(g[c], a.gamma, c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[c][i] *= v[i];
      }
    }
  }
  uint32_t top = 0, block_top[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    block_top[c] = OUT == OUT_SAME ? 0u : amax8<false>(z[c]);
    top = max(top, block_top[c]);
  }
  if constexpr (NORM || OUT == OUT_I8) row_reduce<TPR>(ss, top, sums[0], tops[0]);
  const float rs = NORM ? 1.0f / sqrtf(ss / (float)a.K + a.eps) : 1.0f;

  if constexpr (OUT == OUT_SAME) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[c][i] *= rs;
      store8<F32>(a.Y, at + (c * TPR + t) * 8, n[c], z[c]);
    }
  } else if constexpr (OUT == OUT_I8) {
    const float zm = __uint_as_float(top);
    const bool plain = top < kInfBits && ss < __uint_as_float(kInfBits) && zm >= kTiny && zm * rs >= kTiny &&
                       zm * rs < __uint_as_float(kInfBits);      // (the same in all the row's threads)
    float m = zm;
    uint32_t any = 0;
    if (!plain) {
      uint32_t fin = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[c][i] *= rs;
        any = max(any, amax8<false>(z[c]));
        fin = max(fin, amax8<true>(z[c]));
      }
      float none = 0.0f;
      row_reduce<TPR>(none, fin, sums[1], tops[1]);
      // a NaN in the row: its scale is NaN too, as no int8 code can say it
      if constexpr (TPR > 64) any = (uint32_t)__syncthreads_or(any > kInfBits);
      else any = __any(any > kInfBits) ? 1u : 0u;
      m = block_max(fin);
    }
    if (t == 0) a.scales[row] = any ? __uint_as_float(0x7fc00000u) : (plain ? m * rs : m) / 127.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const u32x2_t q = plain ? codes8_i8<!NORM && F32, false>(z[c], m) : codes8_i8<true, true>(z[c], m);
      store_codes((uint8_t*)a.Y + at + (c * TPR + t) * 8, n[c], q);
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t bits = max16(block_top[c]);
      const float zm = __uint_as_float(bits);
      const bool plain = bits < kInfBits && ss < __uint_as_float(kInfBits) && zm >= kTiny && zm * rs >= kTiny &&
                         zm * rs < __uint_as_float(kInfBits);    // (the same in a block's sixteen lanes)
      float m = zm, scale = zm * rs / kMax;
      u32x2_t q;
      if (plain) {
        q = codes8_of_result(z[c], m);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[c][i] *= rs;
        m = block_max(max16(amax8<true>(z[c])));
        scale = m / kMax;
        q = codes8<true, true>(z[c], m);
      }
      const int k = (c * TPR + t) * 8;
      store_codes((uint8_t*)a.Y + at + k, n[c], q);
      if (n[c] > 0 && (t & 15) == 0) a.scales[(int64_t)(k >> 7) * a.rows + row] = scale;
    }
  }
}

template <bool F32, int OUT, bool NORM, int TPR, int C>
int launch(const NormArgs& a, hipStream_t s) {
  constexpr int TH = row_threads(TPR), RPB = TH / TPR;
  const int64_t blocks = ((int64_t)a.rows + RPB - 1) / RPB;
  if (!fits_one_launch(blocks, TH)) return kNoGrid;
  hipLaunchKernelGGL((row_kernel<F32, OUT, NORM, TPR, C>), dim3((uint32_t)blocks), dim3(TH), 0, s, a);
  return (int)hipGetLastError();
}

template <bool F32, int OUT, bool NORM>
int pick(const NormArgs& a, hipStream_t s) {
  // One or two pieces a thread: one barrier for few loads, and still enough in
  // flight.  e4m3 codes, whose scales are found sixteen lanes at a time, take one
  // (24 rows of 4096: 3.2 us, 3.5 with two; 8192 rows 45.0 and 45.4), a scale per
  // row and results of X's type two (int8 norm of 8192 rows of 4096: 43.4 us, 49
  // with one, 53 with a wave's eight; quantisation of 8192 rows of 8192: 38.9, 54
  // with one).
  constexpr bool ONE = OUT == OUT_F8;
  if (a.K <= 512) return launch<F32, OUT, NORM, 64, 1>(a, s);
  if (a.K <= 1024) return launch<F32, OUT, NORM, ONE ? 128 : 64, ONE ? 1 : 2>(a, s);
  if (a.K <= 2048) return launch<F32, OUT, NORM, ONE ? 256 : 128, ONE ? 1 : 2>(a, s);
  if (a.K <= 4096) return launch<F32, OUT, NORM, ONE ? 512 : 256, ONE ? 1 : 2>(a, s);
  if (a.K <= 8192) return launch<F32, OUT, NORM, 512, 2>(a, s);
  if (a.K <= 16384) return launch<F32, OUT, NORM, 1024, 2>(a, s);
  if (a.K <= 32768) return launch<F32, OUT, NORM, 1024, 4>(a, s);
  return launch<F32, OUT, NORM, 1024, 8>(a, s);
}

}  // namespace

int launch_rmsnorm(const NormArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  const bool f32 = a.dt == DT_F32;
  if (a.out_dt == DT_F8) return f32 ? pick<true, OUT_F8, true>(a, s) : pick<false, OUT_F8, true>(a, s);
  if (a.out_dt == DT_I8) return f32 ? pick<true, OUT_I8, true>(a, s) : pick<false, OUT_I8, true>(a, s);
  return f32 ? pick<true, OUT_SAME, true>(a, s) : pick<false, OUT_SAME, true>(a, s);
}

int launch_quantize_i8(const NormArgs& a, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  return a.dt == DT_F32 ? pick<true, OUT_I8, false>(a, s) : pick<false, OUT_I8, false>(a, s);
}

}  // namespace ox
