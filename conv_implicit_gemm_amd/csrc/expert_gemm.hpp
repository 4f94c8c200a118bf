// expert_gemm.hpp -- products whose rows are grouped by expert, and products
// of 8-bit floating-point operands with block scales.
//
//   Y[m, n] = act( sum_k A[m, k] * B[e(m)][n, k] + bias[e(m)][n] )
//
// The rows of A are sorted by expert: rows offsets[e] .. offsets[e+1]-1 belong
// to expert e, and the offsets live on the device, so the host never learns
// how many rows an expert has.  The grid is the largest number of tiles that
// any offsets can give (T / BM full tiles plus one partial tile per expert);
// each block scans the offsets, finds its own tile and leaves if there is
// none.  A product without experts is the same with one group of all rows.
//
// e4m3 operands carry one fp32 scale per 1 x 128 block of A and per 128 x 128
// block of B.  One v_mfma_f32_16x16x128 covers exactly one block of K, so its
// sum of 128 products (a zero accumulator goes in) is multiplied by
// a_scale * b_scale and added to the running sum in fp32: four fused
// multiply-adds per lane beside an MFMA of 32 cycles.
//
// The weights are the MFMA's row operand and the tokens its column operand,
// so a lane's four results are four consecutive columns of one row of Y.
// Both operands are staged in LDS as rows of 128 bytes of K (128 e4m3 or 64
// bf16): a fragment is the 16-byte pieces g and g + 4 of a row for lane group
// g = lane / 16 (the order of k inside a block is free as long as both
// operands agree on it).  Piece c of row r lies at piece c ^ f(r), with f
// chosen so that the 16 rows a read touches fall on all 64 banks.
#pragma once

#include "lds_dma.hpp"

namespace ox {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// Operand formats of the tile kernel.  For e4m3 there are two ways to the
// matrix unit.  FMT_FP8 feeds the codes to the K = 128 instruction, at full
// rate; inside it the products of a lane's neighbouring k are added with
// about 15 bits below the largest of them (448*448 + 4*1 gives 448*448; the
// accumulator itself is fp32), an error below 2^-15 of sum |a||b| and 1.5e-5
// of the norm of a random result.  bf16 results, rounded at 2^-9, take it.
// FMT_FP8X widens the codes to bf16 (exact) for the bf16 instruction, whose
// sums are fp32 throughout, at half the rate: fp32 results take it.
enum Fmt : int { FMT_BF16 = 0, FMT_FP8 = 1, FMT_FP8X = 2 };

// One piece of 16 bytes at any address.
struct __attribute__((packed, aligned(1))) Bytes16 { u32x4_t v; };

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// Rows [lo, hi) of expert e, kept inside [0, T] whatever the offsets hold.
__device__ __forceinline__ void expert_rows(const ExpertArgs& a, int e, int& lo, int& hi) {
  if (!a.offsets) {
    lo = 0;
    hi = a.T;
    return;
  }
  lo = clampi(a.offsets[e], 0, a.T);
  hi = clampi(a.offsets[e + 1], lo, a.T);
}

// inclusive prefix sum over the wave
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

struct ExpertTile {
  int e, row0, rows;   // expert, first row of the tile, rows in it (<= BM)
};

// Number of row tiles of all experts (every lane of the wave takes part).
template <int BM>
__device__ __forceinline__ int expert_tiles(const ExpertArgs& a) {
  if (!a.offsets) return (a.T + BM - 1) / BM;
  int total = 0;
  for (int base = 0; base < a.E; base += 64) {
    const int e = base + (threadIdx.x & 63);
    int n = 0;
    if (e < a.E) {
      int lo, hi;
      expert_rows(a, e, lo, hi);
      n = (hi - lo + BM - 1) / BM;
    }
    total += __builtin_amdgcn_readlane(wave_scan(n), 63);
  }
  return total;
}

// Row tile t of those, 0 <= t < expert_tiles().
template <int BM>
__device__ __forceinline__ ExpertTile expert_tile(const ExpertArgs& a, int t) {
  ExpertTile r = {0, 0, 0};
  if (!a.offsets) {
    r.row0 = t * BM;
    r.rows = min(BM, a.T - r.row0);
    return r;
  }
  int before = 0;
  for (int base = 0; base < a.E; base += 64) {
    const int e = base + (threadIdx.x & 63);
    int lo = 0, hi = 0;
    if (e < a.E) expert_rows(a, e, lo, hi);
    const int n = (hi - lo + BM - 1) / BM;
    const int s = before + wave_scan(n);          // tiles up to and including e's
    const uint64_t past = __ballot(s > t);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = __builtin_amdgcn_readlane(s - n, l);
      r.e = base + l;
      r.row0 = __builtin_amdgcn_readlane(lo, l) + (t - first) * BM;
      r.rows = min(BM, __builtin_amdgcn_readlane(hi, l) - r.row0);
      return r;
    }
    before = __builtin_amdgcn_readlane(s, 63);
  }
  return r;
}

// Zeros in the rows before the first expert's and past the last one's, spread
// over the grid's blocks.
__device__ __forceinline__ void zero_outside(const ExpertArgs& a) {
  if (!a.offsets) return;
  const int first = clampi(a.offsets[0], 0, a.T);
  const int last = clampi(a.offsets[a.E], 0, a.T);
  if (first == 0 && last == a.T) return;
  const int64_t head = (int64_t)first * a.N, tail = (int64_t)max(first, last) * a.N, all = (int64_t)a.T * a.N;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (int64_t)gridDim.x * blockDim.x) {
    if (i >= head && i < tail) continue;
    if (a.out_dt == DT_F32) ((float*)a.Y)[i] = 0.0f;
    else ((uint16_t*)a.Y)[i] = 0;
  }
}

// The block's tile among total row tiles x NT column tiles: each XCD runs one
// contiguous range of an order that takes bands of four row tiles and walks
// the columns inside a band, so the blocks that run together on an XCD share
// both operands' tiles through its L2.
__device__ __forceinline__ void tile_order(int u, int total, int NT, int& t, int& nt) {
  const int band = u / (4 * NT), in = u - band * 4 * NT;
  const int h = min(4, total - band * 4);
  nt = in / h;
  t = band * 4 + in - nt * h;
}

// The tile kernel: BM rows x BN columns per block, WM x WN waves, S stages of
// 128 bytes of K.  DMA: both operands arrive by buffer-to-LDS loads (16-byte
// aligned rows); otherwise through registers, from any address.  KN (bf16):
// B is [K, N] per expert; its stage holds 64 rows of BN columns, read back
// with transposing LDS reads.
template <int FMT, int BM, int BN, int WM, int WN, int S, bool DMA, bool KN>
struct ExpertTileKernel {
  static constexpr int NW = WM * WN, TH = NW * 64;
  static constexpr int TM = BM / WM, TN = BN / WN, MF = TM / 16, NF = TN / 16;
  static constexpr bool F8 = FMT != FMT_BF16;
  static constexpr int ESZ = F8 ? 1 : 2;
  static constexpr int KE = 128 / ESZ;                       // elements of K per stage
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int SA_BYTES = F8 ? (BM < 64 ? 64 : BM) * 4 : 0;
  static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES;
  static constexpr int LDS_BYTES = S * STAGE;
  static constexpr int DA = BM / 8 / NW, DB = BN / 8 / NW;   // DMA instructions per wave and stage
  static constexpr int D = DA + DB + (F8 ? 1 : 0);
  static_assert(!DMA || (DA * NW * 8 == BM && DB * NW * 8 == BN), "whole DMA instructions per wave");
  static_assert(!KN || FMT == FMT_BF16, "[K, N] weights are bf16");
  static_assert(!F8 || TN <= 128, "a wave's columns share a scale block");

  static __device__ __forceinline__ int sw_a(int r) { return (r >> 1) & 7; }
  // a lane of row group i/4 reads row (i/4)*4*NF + 4*j + i%4 for fragment j
  static __device__ __forceinline__ int sw_b(int r) { return ((r >> 1) & 1) | (((r / (4 * NF)) & 3) << 1); }
  // [K, N]: a transposing read touches rows {0..3, 8..11} (+ 16, + 4) x 32 bytes
  static __device__ __forceinline__ int sw_kn(int k) { return (((k & 3) | ((k >> 1) & 4)) << 1) & (BN / 8 - 1); }

  const ExpertArgs& a;
  char* smem;
  const char* Ab;        // the tile's first row of A
  const char* Bb;        // [N, K]: the tile's first row of B; [K, N]: its first column
  const float* sa;       // a_scales of the tile's first row (k-block 0)
  const float* sb;       // b_scales of this wave's block row
  int rows, cols;        // valid rows and columns of the tile
  int64_t lda, ldb;      // row strides in bytes
  int nk;
  uint32_t va[DA ? DA : 1], vb[DB ? DB : 1], vs;

  __device__ __forceinline__ ExpertTileKernel(const ExpertArgs& a_, char* s) : a(a_), smem(s) {}

  __device__ __forceinline__ uint32_t stage_base(int k) const { return lds_addr(smem) + (uint32_t)(k % S) * STAGE; }

  // --- DMA staging
  __device__ __forceinline__ void init_dma() {
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < DA; ++i) {
      const int r = (w * DA + i) * 8 + (lane >> 3);
      va[i] = r < rows ? (uint32_t)(r * (int)lda + (((lane & 7) ^ sw_a(r)) << 4)) : 0xFFFFFF00u;
    }
#pragma unroll
    for (int i = 0; i < DB; ++i) {
      if constexpr (KN) {
        const int p = (w * DB + i) * 64 + lane, k = p / (BN / 8), c = p % (BN / 8);
        vb[i] = (uint32_t)(k * (int)ldb + ((c ^ sw_kn(k)) << 4));
      } else {
        const int r = (w * DB + i) * 8 + (lane >> 3);
        vb[i] = r < cols ? (uint32_t)(r * (int)ldb + (((lane & 7) ^ sw_b(r)) << 4)) : 0xFFFFFF00u;
      }
    }
    if constexpr (F8) {
      const int r = (w * 64) % (BM < 64 ? 64 : BM) + lane;
      vs = r < rows ? (uint32_t)r * 4u : 0xFFFFFF00u;
    }
  }
  __device__ __forceinline__ void issue(int k) {
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t base = __builtin_amdgcn_readfirstlane(stage_base(k));
    const int left = a.K * ESZ - k * 128;       // bytes of K from this stage on
    const bool tail = left < 128;
    const u32x4_t ra = buffer_words(Ab + (int64_t)k * 128, (uint32_t)((int64_t)(rows - 1) * lda + left));
#pragma unroll
    for (int i = 0; i < DA; ++i) {
      const int r = (w * DA + i) * 8 + (lane >> 3);
      const bool past = tail && (((lane & 7) ^ sw_a(r)) << 4) >= left;
      dma16(base + (w * DA + i) * 1024, past ? 0xFFFFFF00u : va[i], ra);
    }
    if constexpr (KN) {
      const int64_t kl = min(64, a.K - k * 64);   // rows of K in this stage
      const u32x4_t rb = buffer_words(Bb + (int64_t)k * 64 * ldb, (uint32_t)((kl - 1) * ldb + (int64_t)cols * ESZ));
#pragma unroll
      for (int i = 0; i < DB; ++i) dma16(base + A_BYTES + (w * DB + i) * 1024, vb[i], rb);
    } else {
      const u32x4_t rb = buffer_words(Bb + (int64_t)k * 128, (uint32_t)((int64_t)(cols - 1) * ldb + left));
#pragma unroll
      for (int i = 0; i < DB; ++i) {
        const int r = (w * DB + i) * 8 + (lane >> 3);
        const bool past = tail && (((lane & 7) ^ sw_b(r)) << 4) >= left;
        dma16(base + A_BYTES + (w * DB + i) * 1024, past ? 0xFFFFFF00u : vb[i], rb);
      }
    }
    if constexpr (F8) {
      const u32x4_t rs = buffer_words(sa + (int64_t)k * a.T, (uint32_t)rows * 4u);
      dma4(base + A_BYTES + B_BYTES + (w * 256) % SA_BYTES, vs, rs);
    }
  }

  // --- staging through registers
  static constexpr int CA = BM * 8 / TH, CB = BN * 8 / TH;
  static_assert(DMA || (CA * TH == BM * 8 && CB * TH == BN * 8), "whole pieces per thread");
  struct Regs {
    u32x4_t ra[DMA ? 1 : CA], rb[DMA ? 1 : CB];
    float s;
  };
  // bytes [0, n) of 16 at p (n <= 0: none)
  static __device__ __forceinline__ u32x4_t piece(const char* p, int64_t n) {
    if (n >= 16) return ((const Bytes16*)p)->v;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) w[i / 4] |= (uint32_t)(uint8_t)p[i] << (8 * (i % 4));
    return u32x4_t{w[0], w[1], w[2], w[3]};
  }
  __device__ __forceinline__ void load_regs(int k, Regs& g) {
    const int64_t left = (int64_t)a.K * ESZ - (int64_t)k * 128;
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      const int q = threadIdx.x + i * TH, r = q >> 3, c = (q & 7) ^ sw_a(r);
      g.ra[i] = piece(Ab + r * lda + (int64_t)k * 128 + c * 16, r < rows ? left - c * 16 : 0);
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int q = threadIdx.x + i * TH;
      if constexpr (KN) {
        const int kr = q / (BN / 8), c = (q % (BN / 8)) ^ sw_kn(kr);
        g.rb[i] = piece(Bb + ((int64_t)k * 64 + kr) * ldb + c * 16,
                        k * 64 + kr < a.K ? (int64_t)cols * ESZ - c * 16 : 0);
      } else {
        const int r = q >> 3, c = (q & 7) ^ sw_b(r);
        g.rb[i] = piece(Bb + r * ldb + (int64_t)k * 128 + c * 16, r < cols ? left - c * 16 : 0);
      }
    }
    if constexpr (F8) g.s = (int)threadIdx.x < rows ? sa[(int64_t)k * a.T + threadIdx.x] : 0.0f;
  }
  __device__ __forceinline__ void store_regs(int k, const Regs& g) {
    char* st = smem + (k % S) * STAGE;
#pragma unroll
    for (int i = 0; i < CA; ++i) *(u32x4_t*)(st + (threadIdx.x + i * TH) * 16) = g.ra[i];
#pragma unroll
    for (int i = 0; i < CB; ++i) *(u32x4_t*)(st + A_BYTES + (threadIdx.x + i * TH) * 16) = g.rb[i];
    if constexpr (F8)
      if ((int)threadIdx.x < BM) *(float*)(st + A_BYTES + B_BYTES + threadIdx.x * 4) = g.s;
  }

  // --- one stage's products
  // column of Y (within the tile) of fragment j, element r of this lane
  static __device__ __forceinline__ int col_of(int wn, int j, int r) {
    const int g = (threadIdx.x & 63) >> 4;
    return wn * TN + (KN ? j * 16 + g * 4 + r : g * 4 * NF + j * 4 + r);
  }
  __device__ __forceinline__ void frag_a(uint32_t st, int wm, int f, u32x4_t& x, u32x4_t& y) const {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int r = wm * TM + f * 16 + (lane & 15);
    const uint32_t p = st + r * 128;
    x = lds_read_b128(p + ((g ^ sw_a(r)) << 4));
    y = lds_read_b128(p + (((g + 4) ^ sw_a(r)) << 4));
  }
  __device__ __forceinline__ void frag_b(uint32_t st, int wn, int f, u32x4_t& x, u32x4_t& y) const {
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
    if constexpr (KN) {
      const int c = wn * TN + f * 16 + 4 * (i & 3);            // first of this lane's four columns
      auto rd = [&](int k) {
        return lds_read_tr16(st + A_BYTES + k * (BN * 2) + (((c >> 3) ^ sw_kn(k)) << 4) + (c & 4) * 2);
      };
      const int k = g * 8 + (i >> 2);
      const u32x2_t x0 = rd(k), x1 = rd(k + 4), y0 = rd(k + 32), y1 = rd(k + 36);
      x = u32x4_t{x0[0], x0[1], x1[0], x1[1]};
      y = u32x4_t{y0[0], y0[1], y1[0], y1[1]};
    } else {
      const int r = wn * TN + (i >> 2) * 4 * NF + f * 4 + (i & 3);
      const uint32_t p = st + A_BYTES + r * 128;
      x = lds_read_b128(p + ((g ^ sw_b(r)) << 4));
      y = lds_read_b128(p + (((g + 4) ^ sw_b(r)) << 4));
    }
  }
  static __device__ __forceinline__ i32x8_t cat(u32x4_t x, u32x4_t y) {
    return i32x8_t{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  }
  // a fragment's operands as the matrix instructions take them
  struct Frag { u32x4_t v[FMT == FMT_FP8X ? 4 : 2]; };
  static __device__ __forceinline__ Frag widen(u32x4_t x, u32x4_t y) {
    Frag f;
    if constexpr (FMT == FMT_FP8X) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t c = i < 4 ? x[i] : y[i - 4];
        f.v[i / 2][2 * (i % 2)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
        f.v[i / 2][2 * (i % 2) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
      }
    } else {
      f.v[0] = x;
      f.v[1] = y;
    }
    return f;
  }
  static __device__ __forceinline__ f32x4_t mma_bf16(u32x4_t b, u32x4_t a, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b), __builtin_bit_cast(bf16x8_t, a), c, 0,
                                                   0, 0);
  }
  // the 16 x 16 sums of one block of 128 k of e4m3
  static __device__ __forceinline__ f32x4_t mma_block(const Frag& b, const Frag& a) {
    f32x4_t p = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FMT == FMT_FP8) {
      p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(cat(b.v[0], b.v[1]), cat(a.v[0], a.v[1]), p, 0, 0, 0, 0, 0, 0);
    } else if constexpr (FMT == FMT_FP8X) {
#pragma unroll
      for (int h = 0; h < 4; ++h) p = mma_bf16(b.v[h], a.v[h], p);
    }
    return p;
  }
  __device__ __forceinline__ void compute(int k, int wm, int wn, float sbk, f32x4_t (&acc)[MF][NF]) {
    const uint32_t st = stage_base(k);
    Frag b[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      u32x4_t x, y;
      frag_b(st, wn, j, x, y);
      b[j] = widen(x, y);
    }
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      u32x4_t x, y;
      frag_a(st, wm, f, x, y);
      const Frag a = widen(x, y);
      if constexpr (F8) {
        const float s = sbk * *(const OX_LDS float*)(uintptr_t)(st + A_BYTES + B_BYTES +
                                                               (wm * TM + f * 16 + (threadIdx.x & 15)) * 4);
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const f32x4_t p = mma_block(b[j], a);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[f][j][r] = __builtin_fmaf(s, p[r], acc[f][j][r]);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NF; ++j) acc[f][j] = mma_bf16(b[j].v[h], a.v[h], acc[f][j]);
      }
    }
  }

  // --- results: bias, activation, one rounding
  template <int ACT>
  __device__ __forceinline__ void store(const ExpertTile& t, int n0, int wm, int wn, f32x4_t (&acc)[MF][NF]) {
    const int lane = threadIdx.x & 63;
    float bv[NF][4];
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = col_of(wn, j, r);
        bv[j][r] = 0.0f;
        if (a.bias && n < cols) {
          const int64_t at = (int64_t)t.e * a.N + n0 + n;
          bv[j][r] = a.out_dt == DT_F32 ? ((const float*)a.bias)[at] : bf16_to_f32(((const uint16_t*)a.bias)[at]);
        }
      }
    wait_vmem();
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const int m = wm * TM + f * 16 + (lane & 15);
      if (m >= t.rows) continue;
      float v[NF][4];
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[j][r] = act_c<ACT>(acc[f][j][r] + bv[j][r]);
      const int64_t at = (int64_t)(t.row0 + m) * a.N + n0;
      if (a.out_dt == DT_F32) {
        float* y = (float*)a.Y + at;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const int n = col_of(wn, j, 0);
          if (a.y_vec) {
            if (n < cols) *(f32x4_t*)(y + n) = f32x4_t{v[j][0], v[j][1], v[j][2], v[j][3]};
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < cols) y[n + r] = v[j][r];
          }
        }
      } else {
        uint16_t* y = (uint16_t*)a.Y + at;
        if (a.y_vec && !KN && NF % 2 == 0) {
#pragma unroll
          for (int j = 0; j < NF; j += 2) {
            const int n = col_of(wn, j, 0);
            const u32x4_t o = {pack_bf16x2(v[j][0], v[j][1]), pack_bf16x2(v[j][2], v[j][3]),
                               pack_bf16x2(v[(j + 1) % NF][0], v[(j + 1) % NF][1]),
                               pack_bf16x2(v[(j + 1) % NF][2], v[(j + 1) % NF][3])};
            if (n < cols) *(u32x4_t*)(y + n) = o;
          }
        } else {
#pragma unroll
          for (int j = 0; j < NF; ++j) {
            const int n = col_of(wn, j, 0);
            const u32x2_t o = {pack_bf16x2(v[j][0], v[j][1]), pack_bf16x2(v[j][2], v[j][3])};
            if (a.y_vec) {
              if (n < cols) *(u32x2_t*)(y + n) = o;
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (n + r < cols) y[n + r] = (uint16_t)(o[r / 2] >> (16 * (r % 2)));
            }
          }
        }
      }
    }
  }

  __device__ __forceinline__ void run() {
    zero_outside(a);
    const int NT = (a.N + BN - 1) / BN;
    const int total = expert_tiles<BM>(a);
    if ((int64_t)blockIdx.x >= (int64_t)total * NT) return;
    int ti, nt;
    tile_order(xcd_tile(blockIdx.x, total * NT), total, NT, ti, nt);
    ExpertTile t = expert_tile<BM>(a, ti);
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    const int n0 = nt * BN;
    rows = t.rows;
    cols = min(BN, a.N - n0);
    lda = (int64_t)a.K * ESZ;
    ldb = KN ? (int64_t)a.N * ESZ : lda;
    Ab = (const char*)a.A + (int64_t)t.row0 * lda;
    Bb = (const char*)a.B + (int64_t)t.e * a.N * a.K * ESZ + (KN ? (int64_t)n0 * ESZ : (int64_t)n0 * ldb);
    nk = (a.K + KE - 1) / KE;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int kb = (a.K + 127) / 128;
    if constexpr (F8) {
      sa = a.sa + t.row0;
      const int nb = (a.N + 127) / 128;
      sb = a.sb + ((int64_t)t.e * nb + min((n0 + wn * TN) / 128, nb - 1)) * kb;
    }
    f32x4_t acc[MF][NF];
#pragma unroll
    for (int f = 0; f < MF; ++f)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[f][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    float sbl = 0.0f;      // lane l: the wave's b_scale of k-block (k & ~63) + l
    auto scale_of = [&](int k) -> float {
      if constexpr (F8)
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sbl), k & 63));
      return 1.0f;
    };
    auto refill = [&](int k) {
      if constexpr (F8)
        if ((k & 63) == 0) sbl = sb[min(k + (int)(threadIdx.x & 63), kb - 1)];
    };
    if constexpr (DMA) {
      init_dma();
#pragma unroll
      for (int k = 0; k < S - 1; ++k)
        if (k < nk) issue(k);
      for (int k = 0; k < nk; ++k) {
        // stages k+1 .. min(nk, k+S-1)-1 may still be in flight
        wait_dma_barrier_rt<D, S - 2>(min(nk - 1 - k, S - 2));
        refill(k);
        if (k + S - 1 < nk) issue(k + S - 1);
        compute(k, wm, wn, scale_of(k), acc);
      }
    } else {
      Regs g;
      if (nk > 0) load_regs(0, g);
      for (int k = 0; k < nk; ++k) {
        refill(k);
        store_regs(k, g);
        lds_barrier();
        if (k + 1 < nk) load_regs(k + 1, g);
        compute(k, wm, wn, scale_of(k), acc);
      }
    }
    with_act(a.act, [&](auto act) { store<decltype(act)::value>(t, n0, wm, wn, acc); });
  }
};

template <int FMT, int BM, int BN, int WM, int WN, int S, bool DMA, bool KN>
__global__ __launch_bounds__(WM* WN * 64) void expert_gemm_kernel(const ExpertArgs a) {
  typedef ExpertTileKernel<FMT, BM, BN, WM, WN, S, DMA, KN> TK;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  TK k(a, smem);
  k.run();
}

// The most row tiles that any offsets can give.
inline int64_t expert_tile_bound(const ExpertArgs& a, int BM) {
  if (!a.offsets) return ((int64_t)a.T + BM - 1) / BM;
  return (int64_t)a.T / BM + (a.E < a.T ? a.E : a.T);
}

template <int FMT, int BM, int BN, int WM, int WN, int S, bool DMA, bool KN>
int launch_expert_tile(const ExpertArgs& a, hipStream_t s) {
  typedef ExpertTileKernel<FMT, BM, BN, WM, WN, S, DMA, KN> TK;
  int64_t blocks = expert_tile_bound(a, BM) * ((a.N + BN - 1) / BN);
  if (blocks >= ((int64_t)1 << 31)) return (int)hipErrorInvalidValue;
  hipLaunchKernelGGL((expert_gemm_kernel<FMT, BM, BN, WM, WN, S, DMA, KN>), dim3((uint32_t)blocks), dim3(TK::TH),
                     TK::LDS_BYTES, s, a);
  return (int)hipGetLastError();
}

}  // namespace ox
