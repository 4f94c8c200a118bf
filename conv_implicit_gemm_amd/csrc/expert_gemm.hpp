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

#include <string.h>

#include "expert_tiles.hpp"
#include "lds_dma.hpp"

namespace ox {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// Operand formats of the tile kernel.  For e4m3 there are two ways to the
// matrix unit.  FMT_FP8 feeds the codes to the K = 128 instruction, at full
// rate; inside it the products of eight neighbouring k are cut off (towards
// zero) at 2^-13 of 2^(ea + eb), the power of two below the largest of them, and
// then added (448*448 + 4*1 gives 448*448; all sums after that are fp32): at
// worst 7 * 2^-13 of each eight's largest product, 1.5e-5 of the norm of a
// random result.  bf16 results, rounded at 2^-8, take it: the whole error of
// 2048 random k is 1.6617e-3 of the norm, that of the exact sums rounded once
// 1.6616e-3 (2.0129e-3 each where all products are positive).
// FMT_FP8X widens the codes to bf16 (exact) for the bf16 instruction, whose
// sums are fp32 throughout, at half the rate: fp32 results take it.
// fp32 operands take the K = 4 fp32 instruction, four to a 16-byte piece; every
// eight blocks (256 k) the chain of sums is added to a second set and starts
// from zero again (one chain over K = 2800 is 9e-7 of the norm off, this 3e-7
// for any K; adding every block costs 10% of the time, as the fp32 instruction
// leaves the vector unit no room beside it).
// int8 operands take the K = 64 int8 instruction; their sums are int32, exact,
// kept in the same registers as the others' (only the bits travel as floats),
// and meet the scales (one per row of A, one per row of B) with the bias.
enum Fmt : int { FMT_BF16 = 0, FMT_FP8 = 1, FMT_FP8X = 2, FMT_F32 = 3, FMT_I8 = 4 };

template <int FMT>
struct FmtOps {
  static constexpr bool F8 = FMT == FMT_FP8 || FMT == FMT_FP8X;
  static constexpr bool INT = FMT == FMT_I8;
  static constexpr int ESZ = F8 || INT ? 1 : FMT == FMT_F32 ? 4 : 2;
  // c + o: sums of products, or what the integers behind them add up to
  static __device__ __forceinline__ f32x4_t add(f32x4_t c, f32x4_t o) {
    if constexpr (INT) {
      return __builtin_bit_cast(f32x4_t, __builtin_bit_cast(i32x4_t, c) + __builtin_bit_cast(i32x4_t, o));
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) c[r] += o[r];
      return c;
    }
  }
  // the sum that v holds, under its scales (int8)
  static __device__ __forceinline__ float value(float v, float sa, float sb) {
    if constexpr (INT) return (float)__float_as_int(v) * sa * sb;
    return v;
  }
  // a fragment's 128 bytes of K as the matrix instructions take them
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
  static __device__ __forceinline__ i32x8_t cat(u32x4_t x, u32x4_t y) {
    return i32x8_t{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  }
  // c += the products of piece h of both fragments
  template <int H>
  static __device__ __forceinline__ f32x4_t half(const Frag& b, const Frag& a, f32x4_t c) {
    if constexpr (FMT == FMT_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b.v[H][i]), __uint_as_float(a.v[H][i]), c, 0, 0, 0);
      return c;
    } else if constexpr (INT) {
      return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_mfma_i32_16x16x64_i8(
          __builtin_bit_cast(i32x4_t, b.v[H]), __builtin_bit_cast(i32x4_t, a.v[H]), __builtin_bit_cast(i32x4_t, c), 0, 0, 0));
    } else {
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b.v[H]),
                                                     __builtin_bit_cast(bf16x8_t, a.v[H]), c, 0, 0, 0);
    }
  }
  // the 16 x 16 sums of one block of 128 k of e4m3
  static __device__ __forceinline__ f32x4_t block(const Frag& b, const Frag& a) {
    f32x4_t p = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FMT == FMT_FP8) {
      p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(cat(b.v[0], b.v[1]), cat(a.v[0], a.v[1]), p, 0, 0, 0, 0, 0, 0);
    } else if constexpr (FMT == FMT_FP8X) {
      p = half<0>(b, a, p);
      p = half<1>(b, a, p);
      p = half<2>(b, a, p);
      p = half<3>(b, a, p);
    }
    return p;
  }
};

// LDS by pointer and constant, so that the constant goes into the instruction
__device__ __forceinline__ const OX_LDS char* lds_ptr(uint32_t a) { return (const OX_LDS char*)(uintptr_t)a; }
__device__ __forceinline__ u32x4_t lds_read_at(const OX_LDS char* p, int o) { return *(const OX_LDS u32x4_t*)(p + o); }

// One piece of 16 bytes at any address.
struct __attribute__((packed, aligned(1))) Bytes16 { u32x4_t v; };
struct __attribute__((packed, aligned(1))) Bytes8 { u32x2_t v; };

// Bytes [n, 16) of v moved to its front, and zeros behind them (n <= 0: v).
__device__ __forceinline__ u32x4_t moved_down(u32x4_t v, int n) {
  n = max(n, 0);
  const uint64_t a = (uint64_t)v[1] << 32 | v[0], b = (uint64_t)v[3] << 32 | v[2];
  const uint64_t lo = n < 8 ? a : n < 16 ? b : 0, hi = n < 8 ? b : 0;
  const int bits = (n & 7) * 8;
  const uint64_t l = lo >> bits | (hi << 1) << (63 - bits), h = hi >> bits;
  return u32x4_t{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
}

// The descriptor in scalar registers, where the DMA wants it.  A vector
// instruction that writes a scalar register (v_readfirstlane) needs five wait
// states before a vector-memory instruction reads it; the compiler does not
// see the reader inside the DMA's assembly, so they are spent here.
__device__ __forceinline__ u32x4_t uniform_words(const char* p, int64_t bytes) {
  u32x4_t w = buffer_words(p, (uint32_t)bytes);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_readfirstlane(w[i]);
  asm volatile("s_nop 4" : "+s"(w));
  return w;
}

// the same address in scalar registers
template <typename T>
__device__ __forceinline__ T* uniform_ptr(T* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (T*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}

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

// inclusive prefix sum over the wave: shifts within rows of 16 lanes, then
// each row's last lane broadcast to the rows behind it
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
  return v;
}

// Zeros in rows [0, first) and [last, T), spread over the grid's blocks.
__device__ __forceinline__ void zero_outside(const ExpertArgs& a, int first, int last) {
  const int64_t head = (int64_t)first * a.N, tail = (int64_t)max(first, last) * a.N, all = (int64_t)a.T * a.N;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (int64_t)gridDim.x * blockDim.x) {
    if (i >= head && i < tail) continue;
    if (a.out_dt == DT_F32) ((float*)a.Y)[i] = 0.0f;
    else ((uint16_t*)a.Y)[i] = 0;
  }
}

// This block's tile, from the offsets; false when the offsets have fewer (and
// for all blocks when decreasing offsets make more than the grid was sized
// for).  Each XCD runs one contiguous range of tile_order(), so the blocks that
// run together on an XCD share both operands' tiles through its L2.
// Also writes its share of the zeros outside the experts' rows.  Up to 64
// experts are one load and one scan across the wave (a second round for each
// 64 more); every wave does it for itself, without a barrier.
template <int BM>
__device__ __forceinline__ bool find_tile(const ExpertArgs& a, int NT, ExpertTile& r, int& nt) {
  const int b = blockIdx.x;
  int t;
  if (!a.offsets) {
    const int total = ceil_div(a.T, BM);
    tile_order(xcd_tile(b, total * NT), total, NT, t, nt);
    r.e = 0;
    r.row0 = t * BM;
    r.rows = min(BM, a.T - r.row0);
    return true;
  }
  const int lane = threadIdx.x & 63;
  int lo, n, s, first = 0, last = 0;
  int64_t total = 0;
  for (int base = 0; base < a.E; base += 64) {
    int hi = 0;
    lo = 0;
    if (base + lane < a.E) expert_rows(a, base + lane, lo, hi);
    if (base == 0) first = __builtin_amdgcn_readlane(lo, 0);
    last = max(last, __builtin_amdgcn_readlane(hi, min(63, a.E - 1 - base)));
    n = ceil_div(hi - lo, BM);
    s = wave_scan(n);
    total += __builtin_amdgcn_readlane(s, 63);
    r.rows = hi;
  }
  if (first != 0 || last != a.T) zero_outside(a, first, last);
  if (!block_has_tile(b, total, NT, expert_tile_bound(a.T, a.E, BM))) return false;
  tile_order(xcd_tile(b, (int)total * NT), (int)total, NT, t, nt);
  int hi = r.rows;
  int64_t before = 0;
  for (int base = 0; base < a.E; base += 64) {
    if (a.E > 64) {
      lo = hi = 0;
      if (base + lane < a.E) expert_rows(a, base + lane, lo, hi);
      n = ceil_div(hi - lo, BM);
      s = wave_scan(n);
    }
    const uint64_t past = __ballot(before + s > t);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int64_t skip = t - before - __builtin_amdgcn_readlane(s - n, l);   // tiles of this expert before this one
      r.e = base + l;
      return expert_tile_rows(__builtin_amdgcn_readlane(lo, l), __builtin_amdgcn_readlane(hi, l), skip, BM, r);
    }
    before += __builtin_amdgcn_readlane(s, 63);
  }
  return false;
}

// The tile kernel: BM rows x BN columns per block, WM x WN waves, S stages of
// KS blocks of 128 bytes of K: KS groups of WM x WN waves take one block of
// each stage and their sums are added at the end, in order (with few tiles a
// stage costs its latency, not its products: KS = 2 halves the stages).  DMA: both operands arrive by buffer-to-LDS loads (16-byte
// aligned rows); otherwise through registers, from any address.  KN (bf16):
// B is [K, N] per expert; its stage holds 64 (fp32: 32) rows of BN columns, read
// back with transposing LDS reads.
//
// What bounds it: at 8192^3 e4m3 (256 x 256, two waves a SIMD, 128 accumulator
// registers each) 468 to 492 us on different cards, 2.2 to 2.35 PFLOP/s: the matrix units are busy 54% of the
// cycles, LDS reads take 75% of what it delivers in a step (24 KB a wave and
// block of K, the reason for the tall wave tiles), and each tile adds 11 us,
// 6 of them the stores of all CUs at once.  bf16 at 8192^3: 1.3 PFLOP/s.
// Weights for few rows stream at 4.7-4.9 TB/s ([N, K], 32 x 64 tiles).
template <int FMT, int BM, int BN, int WM, int WN, int S, int KS, bool DMA, bool KN>
struct ExpertTileKernel {
  static constexpr int NW = WM * WN, TH = NW * KS * 64;     // waves of a group, threads of a block
  static constexpr int TM = BM / WM, TN = BN / WN, MF = TM / 16, NF = TN / 16;
  typedef FmtOps<FMT> Mm;
  typedef typename Mm::Frag Frag;
  static constexpr bool F8 = Mm::F8;
  static constexpr int ESZ = Mm::ESZ;
  static constexpr int KE = 128 / ESZ;                       // elements of K per stage
  static constexpr int MPP = FMT == FMT_F32 ? 4 : 1;         // matrix instructions per piece
  static constexpr int KNR = FMT == FMT_F32 ? 8 : 4;         // [K, N]: LDS reads per fragment
  static constexpr int PE = 16 / ESZ;                        // elements per piece
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  static constexpr int SA_BYTES = F8 ? (BM < 64 ? 64 : BM) * 4 : 0;
  static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES;
  static constexpr int LDS_BYTES = S * KS * STAGE;
  static_assert(KS == 1 || LDS_BYTES >= (KS - 1) * BM * BN * 4, "the groups' sums go through the stages' memory");
  static constexpr int DA = BM / 8 / NW, DB = BN / 8 / NW;   // DMA instructions per wave and stage
  static constexpr int D = DA + DB + (F8 ? 1 : 0);
  static_assert(!DMA || (DA * NW * 8 == BM && DB * NW * 8 == BN), "whole DMA instructions per wave");
  static_assert(DMA || KS == 1, "one block per stage through registers");
  static_assert(MF % 2 == 0, "row fragments alternate between two sets of block sums");
  static_assert(!KN || (NF & (NF - 1)) == 0, "fragments are bits of the column");
  static_assert(!KN || ESZ > 1, "8-bit weights are [N, K]");
  static_assert(!KN || FMT != FMT_F32 || BN % 64 == 0, "the swizzle of fp32 rows spans 64 columns");
  static_assert(!F8 || TN <= 128, "a wave's columns share a scale block");

  static __device__ __forceinline__ int sw_a(int r) { return (r >> 1) & 7; }
  // a lane of row group i/4 reads row (i/4)*4*NF + 4*j + i%4 for fragment j
  static __device__ __forceinline__ int sw_b(int r) { return ((r >> 1) & 1) | (((r / (4 * NF)) & 3) << 1); }
  // [K, N], bf16: a transposing read touches rows {0..3, 8..11} (+ 16, + 4) x
  // 32 bytes; fp32: a read touches rows {0, 4, 8, 12} (+ 0..3, + 16) x 64 bytes
  static __device__ __forceinline__ int sw_kn(int k) {
    if constexpr (FMT == FMT_F32) return ((k >> 2) & 3) << 2;
    return (((k & 3) | ((k >> 1) & 4)) << 1) & (BN / 8 - 1);
  }

  const ExpertArgs& a;
  char* smem;
  const char* Ab;        // the tile's first row of A
  const char* Bb;        // [N, K]: the tile's first row of B; [K, N]: its first column
  const float* sa;       // a_scales of the tile's first row (k-block 0)
  const float* sb;       // b_scales of this wave's block row
  int rows, cols;        // valid rows and columns of the tile
  int64_t lda, ldb;      // row strides in bytes
  int nk, gwave;         // blocks of K; this wave in its group, which loads the blocks that it multiplies
  uint32_t va[DA ? DA : 1], vb[DB ? DB : 1], vs;

  __device__ __forceinline__ ExpertTileKernel(const ExpertArgs& a_, char* s) : a(a_), smem(s) {}

  __device__ __forceinline__ uint32_t stage_base(int k) const { return lds_addr(smem) + (uint32_t)(k % (S * KS)) * STAGE; }

  // --- DMA staging
  __device__ __forceinline__ void init_dma() {
    const int lane = threadIdx.x & 63, w = gwave;
#pragma unroll
    for (int i = 0; i < DA; ++i) {
      const int r = (w * DA + i) * 8 + (lane >> 3);
      va[i] = r < rows ? (uint32_t)(r * (int)lda + (((lane & 7) ^ sw_a(r)) << 4)) : 0xFFFFFF00u;
    }
#pragma unroll
    for (int i = 0; i < DB; ++i) {
      if constexpr (KN) {
        const int p = (w * DB + i) * 64 + lane, k = p / (BN / PE), c = p % (BN / PE);
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
  // Blocks of K in the order of the stages: a block that K ends inside comes
  // first, so that every later stage is whole and the loop has no branch (a
  // branch inside it would let the compiler move additions past it).
  int part;              // 1 when K ends inside a block
  __device__ __forceinline__ int block_of(int k) const { return DMA && part ? (k == 0 ? nk - 1 : k - 1) : k; }

  // Stage k into its slot.  PART: the pieces of the block from K on are zeros.
  // A stage past the last one is loaded from an empty range (zeros, no
  // traffic), which keeps the number of loads in flight the same for all.
  template <bool PART>
  __device__ __forceinline__ void issue(int k) {
    const int lane = threadIdx.x & 63, w = gwave;
    const uint32_t base = __builtin_amdgcn_readfirstlane(stage_base(k));
    const bool any = k < nk;
    const int kb = any ? block_of(k) : 0;
    const int left = PART ? a.K * ESZ - kb * 128 : 128;       // bytes of K from this block on
    const u32x4_t ra = uniform_words(Ab + (int64_t)kb * 128, any ? (int64_t)(rows - 1) * lda + left : 0);
#pragma unroll
    for (int i = 0; i < DA; ++i) {
      const bool past = PART && (((lane & 7) ^ sw_a((w * DA + i) * 8 + (lane >> 3))) << 4) >= left;
      dma16(base + (w * DA + i) * 1024, past ? 0xFFFFFF00u : va[i], ra);
    }
    if constexpr (KN) {
      const int64_t kl = PART ? min(KE, a.K - kb * KE) : KE;   // rows of K in this block
      const u32x4_t rb = uniform_words(Bb + (int64_t)kb * KE * ldb, any ? (kl - 1) * ldb + (int64_t)cols * ESZ : 0);
#pragma unroll
      for (int i = 0; i < DB; ++i) dma16(base + A_BYTES + (w * DB + i) * 1024, vb[i], rb);
    } else {
      const u32x4_t rb = uniform_words(Bb + (int64_t)kb * 128, any ? (int64_t)(cols - 1) * ldb + left : 0);
#pragma unroll
      for (int i = 0; i < DB; ++i) {
        const bool past = PART && (((lane & 7) ^ sw_b((w * DB + i) * 8 + (lane >> 3))) << 4) >= left;
        dma16(base + A_BYTES + (w * DB + i) * 1024, past ? 0xFFFFFF00u : vb[i], rb);
      }
    }
    if constexpr (F8) {
      const u32x4_t rs = uniform_words((const char*)(sa + (int64_t)kb * a.T), any ? (int64_t)rows * 4 : 0);
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
  // K ends inside block k, of rows that hold a piece.  Byte by byte such a block
  // takes several trips to memory (2048 rows of 4096 x 1001 int8 25.6 us, 22.5 with
  // the row's last piece moved; bf16 49.5 and 46.1; fp32, four elements a piece,
  // gains nothing and loses up to 12%).
  __device__ __forceinline__ bool cut_here(int k) const {
    return !KN && FMT != FMT_F32 && (int64_t)a.K * ESZ - (int64_t)k * 128 < 128 && a.K >= 16 / ESZ;
  }
  // A block that lies inside K (and for [K, N] a tile inside N) takes its pieces
  // without a question; rows past the tile are read again from its last one,
  // their results are never stored.
  __device__ __forceinline__ void load_regs(int k, Regs& g) {
    const int64_t left = (int64_t)a.K * ESZ - (int64_t)k * 128;
    if constexpr (F8) g.s = (int)threadIdx.x < rows ? sa[(int64_t)k * a.T + threadIdx.x] : 0.0f;
    if (KN ? left >= 128 && k < a.K / KE && cols == BN : left >= 128) {
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        const int q = threadIdx.x + i * TH, r = q >> 3, c = (q & 7) ^ sw_a(r);
        g.ra[i] = ((const Bytes16*)(Ab + min(r, rows - 1) * lda + (int64_t)k * 128 + c * 16))->v;
      }
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int q = threadIdx.x + i * TH;
        if constexpr (KN) {
          const int kr = q / (BN / PE), c = (q % (BN / PE)) ^ sw_kn(kr);
          g.rb[i] = ((const Bytes16*)(Bb + ((int64_t)k * KE + kr) * ldb + c * 16))->v;
        } else {
          const int r = q >> 3, c = (q & 7) ^ sw_b(r);
          g.rb[i] = ((const Bytes16*)(Bb + min(r, cols - 1) * ldb + (int64_t)k * 128 + c * 16))->v;
        }
      }
      return;
    }
    if (cut_here(k)) {
      // the pieces that K ends in front of or inside: the row's last 16 bytes,
      // which store_regs moves into place
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        const int q = threadIdx.x + i * TH, r = q >> 3, c = (q & 7) ^ sw_a(r);
        g.ra[i] = ((const Bytes16*)(Ab + min(r, rows - 1) * lda + (int64_t)k * 128 + min(c * 16, (int)left - 16)))->v;
      }
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int q = threadIdx.x + i * TH, r = q >> 3, c = (q & 7) ^ sw_b(r);
        g.rb[i] = ((const Bytes16*)(Bb + min(r, cols - 1) * ldb + (int64_t)k * 128 + min(c * 16, (int)left - 16)))->v;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      const int q = threadIdx.x + i * TH, r = q >> 3, c = (q & 7) ^ sw_a(r);
      g.ra[i] = piece(Ab + r * lda + (int64_t)k * 128 + c * 16, r < rows ? left - c * 16 : 0);
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int q = threadIdx.x + i * TH;
      if constexpr (KN) {
        const int kr = q / (BN / PE), c = (q % (BN / PE)) ^ sw_kn(kr);
        g.rb[i] = piece(Bb + ((int64_t)k * KE + kr) * ldb + c * 16,
                        k * KE + kr < a.K ? (int64_t)cols * ESZ - c * 16 : 0);
      } else {
        const int r = q >> 3, c = (q & 7) ^ sw_b(r);
        g.rb[i] = piece(Bb + r * ldb + (int64_t)k * 128 + c * 16, r < cols ? left - c * 16 : 0);
      }
    }
  }
  __device__ __forceinline__ void store_regs(int k, Regs& g) {
    char* st = smem + (k % (S * KS)) * STAGE;
    if (cut_here(k)) {
      const int past = 16 - (int)((int64_t)a.K * ESZ - (int64_t)k * 128);
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        const int q = threadIdx.x + i * TH;
        g.ra[i] = moved_down(g.ra[i], (((q & 7) ^ sw_a(q >> 3)) * 16) + past);
      }
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int q = threadIdx.x + i * TH;
        g.rb[i] = moved_down(g.rb[i], (((q & 7) ^ sw_b(q >> 3)) * 16) + past);
      }
    }
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
  // This lane's fragment addresses inside a stage.  f(r) is the same for every
  // fragment of a lane, so fragment f lies f * 2048 (A), f * 512 ([N, K]) past
  // the first, and the second piece of a row is the first's address ^ 64.
  uint32_t oa, ob[KN ? 4 : 1];
  __device__ __forceinline__ void init_frags(int wm, int wn) {
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
    const int r = wm * TM + i;
    oa = r * 128 + ((g ^ sw_a(r)) << 4);
    if constexpr (KN && FMT == FMT_F32) {
      // column i of the fragment, row g * 4 (+ e, + 16)
      ob[0] = A_BYTES + g * 4 * (BN * 4) + (i & 3) * 4 + (((wn * TN / 4 + (i >> 2)) ^ sw_kn(g * 4)) << 4);
    } else if constexpr (KN) {
      // (column 4*(i & 3) of the fragment; the rows g*8 + i/4, + 4, + 32, + 36)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int k = g * 8 + (i >> 2) + (h & 1) * 4 + (h >> 1) * 32;
        ob[h] = A_BYTES + k * (BN * 2) + (i & 1) * 8 + (((wn * TN / 8 + ((i >> 1) & 1)) ^ sw_kn(k)) << 4);
      }
    } else {
      const int q = wn * TN + (i >> 2) * 4 * NF + (i & 3);
      ob[0] = A_BYTES + q * 128 + ((g ^ sw_b(q)) << 4);
    }
  }
  __device__ __forceinline__ void frag_a(uint32_t st, int f, u32x4_t& x, u32x4_t& y) const {
    x = lds_read_at(lds_ptr(st + oa), f * 2048);
    y = lds_read_at(lds_ptr(st + (oa ^ 64)), f * 2048);
  }
  __device__ __forceinline__ void frag_b(uint32_t st, int f, u32x4_t& x, u32x4_t& y) const {
    if constexpr (KN && FMT == FMT_F32) {
      const OX_LDS char* p = lds_ptr(st + (ob[0] ^ (uint32_t)(f * 64)));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = *(const OX_LDS uint32_t*)(p + e * (BN * 4));
        y[e] = *(const OX_LDS uint32_t*)(p + (16 + e) * (BN * 4));
      }
    } else if constexpr (KN) {
      // f * 32 bytes further in the row, through the swizzle (a power of two per bit of f)
      u32x2_t v[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) v[h] = lds_read_tr16(st + (ob[h] ^ (uint32_t)(f * 32)));
      x = u32x4_t{v[0][0], v[0][1], v[1][0], v[1][1]};
      y = u32x4_t{v[2][0], v[2][1], v[3][0], v[3][1]};
    } else {
      x = lds_read_at(lds_ptr(st + ob[0]), f * 512);
      y = lds_read_at(lds_ptr(st + (ob[0] ^ 64)), f * 512);
    }
  }
  // What a step hands to the next: the weights' fragments and the first row
  // fragment of its stage, and the last block sums, not yet added.
  struct Flow {
    Frag b[NF];
    u32x4_t x, y;      // row fragment 0
    float s;           // its row's scale
    f32x4_t p[2][NF];  // block sums of the last two row fragments
    float sp;          // the scale of the last ones
  };
  __device__ __forceinline__ float row_scale(uint32_t st, int wm, int f) const {
    if constexpr (F8)
      return *(const OX_LDS float*)(lds_ptr(st + A_BYTES + B_BYTES + (wm * TM + (threadIdx.x & 15)) * 4) + f * 64);
    return 0.0f;
  }
  __device__ __forceinline__ void read_b(uint32_t st, int j, Flow& w) const {
    u32x4_t x, y;
    frag_b(st, j, x, y);
    w.b[j] = Mm::widen(x, y);
  }
  __device__ __forceinline__ void reload(int k, int wm, Flow& w) const {
    const uint32_t st = stage_base(k);
    frag_a(st, 0, w.x, w.y);
    w.s = row_scale(st, wm, 0);
#pragma unroll
    for (int j = 0; j < NF; ++j) read_b(st, j, w);
  }
  __device__ __forceinline__ void begin(int k, int wm, Flow& w) const {
    reload(k, wm, w);
#pragma unroll
    for (int j = 0; j < NF; ++j) w.p[1][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    w.sp = 0.0f;
  }
  static __device__ __forceinline__ void add_block(f32x4_t (&c)[NF], const f32x4_t (&p)[NF], float s) {
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) c[j][r] = __builtin_fmaf(s, p[j][r], c[j][r]);
  }
  // One stage.  Row fragment f + 1 is read while f is multiplied, and the
  // block sums of f are scaled and added under the products of f + 1 (those
  // of the last f under the next stage's first).  Before the last fragment's
  // products every read of this stage has returned: turn() waits for the next
  // stage and passes the barrier, the next stage's first fragments are read
  // under these products, and refill() loads this slot again behind them.  The
  // scheduler would sink the reads to their uses, so the order is pinned.
  template <bool NEXT, class Turn, class Refill>
  __device__ __forceinline__ void compute(int k, int wm, float sbk, f32x4_t (&acc)[MF][NF], Flow& w, Turn&& turn,
                                          Refill&& refill) {
    const uint32_t st = stage_base(k), st1 = stage_base(k + KS);
    static_for<MF>([&](auto F) {
      constexpr int f = F.value;
      constexpr bool last = f + 1 == MF, load = !last || NEXT;
      const Frag a = Mm::widen(w.x, w.y);
      const float s1 = w.s;
      if constexpr (last && NEXT) {
        turn();
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (load) {
        frag_a(last ? st1 : st, last ? 0 : f + 1, w.x, w.y);
        w.s = row_scale(last ? st1 : st, wm, last ? 0 : f + 1);
      }
      if constexpr (F8) {
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          w.p[f & 1][j] = Mm::block(w.b[j], a);
          if constexpr (last && NEXT) read_b(st1, j, w);
        }
        add_block(acc[(f + MF - 1) % MF], w.p[(f & 1) ^ 1], w.sp);
        w.sp = sbk * s1;
        __builtin_amdgcn_sched_group_barrier(0x100, load ? 3 : 0, 0);
        static_for<NF>([&](auto) {
          __builtin_amdgcn_sched_group_barrier(0x008, FMT == FMT_FP8X ? 4 : 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, last && NEXT ? 2 : 0, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        });
      } else {
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[f][j] = Mm::template half<0>(w.b[j], a, acc[f][j]);
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          acc[f][j] = Mm::template half<1>(w.b[j], a, acc[f][j]);
          if constexpr (last && NEXT) read_b(st1, j, w);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, load ? 2 : 0, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, NF * MPP, 0);
        static_for<NF>([&](auto) {
          __builtin_amdgcn_sched_group_barrier(0x008, MPP, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, last && NEXT ? (KN ? KNR : 2) : 0, 0);
        });
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (last && NEXT) refill();
    });
  }

  // --- results: bias, activation, one rounding.  A lane's neighbouring columns
  // leave as one store from any address, the last columns of a row one by one
  // (6261 x 2494 x 656 int8 to fp32, rows that start 8 bytes off a piece: 36.6 us,
  // 90.8 with single elements throughout; to bf16 31.1 and 63.6 with 2495)
  struct Where { int e, row0, rows, n0, cols; };
  __device__ __forceinline__ void load_bias(const Where& t, int wn, float (&bv)[NF][4]) const {
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = col_of(wn, j, r);
        bv[j][r] = 0.0f;
        if (a.bias && n < t.cols) {
          const int64_t at = (int64_t)t.e * a.N + t.n0 + n;
          bv[j][r] = a.out_dt == DT_F32 ? ((const float*)a.bias)[at] : bf16_to_f32(((const uint16_t*)a.bias)[at]);
        }
      }
  }
  // int8: the columns' scales, as the biases; rows without columns (K = 0) have
  // none to read
  __device__ __forceinline__ void load_scales(const Where& t, int wn, float (&sv)[NF][4]) const {
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = col_of(wn, j, r);
        sv[j][r] = Mm::INT && nk > 0 && n < t.cols ? a.sb[(int64_t)t.e * a.N + t.n0 + n] : 0.0f;
      }
  }
  template <int ACT>
  __device__ __forceinline__ void store(const Where& t, int wm, int wn, const f32x4_t (&acc)[MF][NF],
                                        const float (&bv)[NF][4], const float (&sv)[NF][4], const float (&sm)[MF]) const {
    const int lane = threadIdx.x & 63, cols = t.cols;
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const int m = wm * TM + f * 16 + (lane & 15);
      if (m >= t.rows) continue;
      float v[NF][4];
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[j][r] = act_c<ACT>(Mm::value(acc[f][j][r], sm[f], sv[j][r]) + bv[j][r]);
      const int64_t at = (int64_t)(t.row0 + m) * a.N + t.n0;
      if (a.out_dt == DT_F32) {
        float* y = (float*)a.Y + at;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const int n = col_of(wn, j, 0);
          if (n + 3 < cols) {
            ((Bytes16*)(y + n))->v = u32x4_t{__float_as_uint(v[j][0]), __float_as_uint(v[j][1]), __float_as_uint(v[j][2]),
                                             __float_as_uint(v[j][3])};
          } else {
#pragma unroll
            for (int r = 0; r < 3; ++r)
              if (n + r < cols) y[n + r] = v[j][r];
          }
        }
      } else {
        uint16_t* y = (uint16_t*)a.Y + at;
        if (!KN && NF % 2 == 0) {
#pragma unroll
          for (int j = 0; j < NF; j += 2) {
            const int n = col_of(wn, j, 0);
            const u32x4_t o = {pack_bf16x2(v[j][0], v[j][1]), pack_bf16x2(v[j][2], v[j][3]),
                               pack_bf16x2(v[(j + 1) % NF][0], v[(j + 1) % NF][1]),
                               pack_bf16x2(v[(j + 1) % NF][2], v[(j + 1) % NF][3])};
            if (n + 7 < cols) {
              ((Bytes16*)(y + n))->v = o;
            } else {
#pragma unroll
              for (int r = 0; r < 7; ++r)
                if (n + r < cols) y[n + r] = (uint16_t)(o[r / 2] >> (16 * (r % 2)));
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < NF; ++j) {
            const int n = col_of(wn, j, 0);
            const u32x2_t o = {pack_bf16x2(v[j][0], v[j][1]), pack_bf16x2(v[j][2], v[j][3])};
            if (n + 3 < cols) {
              ((Bytes8*)(y + n))->v = o;
            } else {
#pragma unroll
              for (int r = 0; r < 3; ++r)
                if (n + r < cols) y[n + r] = (uint16_t)(o[r / 2] >> (16 * (r % 2)));
            }
          }
        }
      }
    }
  }

  // Where the tile lies, and its operands' addresses.
  __device__ __forceinline__ void setup(const ExpertTile& x, int nt, int wn, Where& t) {
    t.e = __builtin_amdgcn_readfirstlane(x.e);
    t.row0 = __builtin_amdgcn_readfirstlane(x.row0);
    t.rows = rows = __builtin_amdgcn_readfirstlane(x.rows);
    t.n0 = __builtin_amdgcn_readfirstlane(nt) * BN;
    t.cols = cols = min(BN, a.N - t.n0);
    Ab = uniform_ptr((const char*)a.A + (int64_t)t.row0 * lda);
    Bb = uniform_ptr((const char*)a.B + (int64_t)t.e * a.N * a.K * ESZ + (KN ? (int64_t)t.n0 * ESZ : (int64_t)t.n0 * ldb));
    if constexpr (F8) {
      sa = uniform_ptr(a.sa + t.row0);
      const int nb = ceil_div(a.N, 128);
      sb = uniform_ptr(a.sb + ((int64_t)t.e * nb + min((int)(((uint32_t)t.n0 + wn * TN) / 128), nb - 1)) * nk);
    }
  }
  // The b_scale of stage block k, by a scalar load (a vector load would have to
  // be waited for with the DMA behind it).  A group's block past the last one
  // has none: its products are zeros, and an infinite scale would make NaN of them.
  __device__ __forceinline__ float scale_of(int k) const {
    typedef const __attribute__((address_space(4))) float* Scalar;
    if constexpr (F8) {
      const float v = *(Scalar)(uintptr_t)(sb + min(block_of(k), nk - 1));
      return KS == 1 || k < nk ? v : 0.0f;
    }
    return 1.0f;
  }
  __device__ __forceinline__ void start_loads(int grp) {
    init_dma();
    if (part && grp == 0) issue<true>(0);
    else issue<false>(grp);
#pragma unroll
    for (int x = 1; x < S; ++x) issue<false>(x * KS + grp);
  }

  __device__ __forceinline__ void run(const ExpertTile& x, int nt) {
    lda = (int64_t)a.K * ESZ;
    ldb = KN ? (int64_t)a.N * ESZ : lda;
    nk = ceil_div(a.K, KE);
    part = (a.K * (int64_t)ESZ) % 128 != 0;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), grp = wave / NW;
    gwave = wave % NW;
    const int wm = gwave / WN, wn = gwave % WN;
    Where t;
    setup(x, nt, wn, t);
    init_frags(wm, wn);
    auto nothing = [] {};
    f32x4_t acc[MF][NF];
#pragma unroll
    for (int f = 0; f < MF; ++f)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[f][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr bool F32 = FMT == FMT_F32;
    f32x4_t sum[F32 ? MF : 1][F32 ? NF : 1];
    auto flush = [&](int stage) {
      if constexpr (F32) {
        if ((stage & 7) != 7) return;
#pragma unroll
        for (int f = 0; f < MF; ++f)
#pragma unroll
          for (int j = 0; j < NF; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              sum[f][j][r] += acc[f][j][r];
              acc[f][j][r] = 0.0f;
            }
      }
    };
    if constexpr (F32) {
#pragma unroll
      for (int f = 0; f < MF; ++f)
#pragma unroll
        for (int j = 0; j < NF; ++j) sum[f][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    Flow w;
    if constexpr (DMA) {
      if (nk > 0) {
        start_loads(grp);
        wait_dma_barrier<D*(S - 1)>();
        begin(grp, wm, w);
        int k = 0;
        float sk = scale_of(grp);
#pragma unroll 1
        for (; k + KS < nk; k += KS) {
          const float next = scale_of(k + KS + grp);
          compute<true>(k + grp, wm, sk, acc, w, [&] {
            wait_dma_barrier<D*(S - 2)>();      // the next stage is there, the S - 2 after it may be in flight
          }, [&] { issue<false>(k + S * KS + grp); });
          sk = next;
          flush(k / KS);
        }
        // (a block past the last one holds zeros)
        compute<false>(k + grp, wm, sk, acc, w, nothing, nothing);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
    } else {
      // PF blocks in flight, each in registers of its own (the large tile has
      // more than one block on a CU only without them: 2048 rows over 8 experts
      // of 4096 x 1001 bf16 31 us, 42 us with four; 2018 over 8 of 96 x 1998
      // fp32 on the small one 52 us with four, 118 us with one)
      constexpr int PF = BM >= 128 ? 1 : 4;
      Regs g[PF];
      static_for<PF>([&](auto V) {
        if (V.value < nk) load_regs(V.value, g[V.value]);
      });
#pragma unroll 1
      for (int k0 = 0; k0 < nk; k0 += PF)
        static_for<PF>([&](auto V) {
          const int k = k0 + V.value;
          if (k >= nk) return;
          const float sk = scale_of(k);
          store_regs(k, g[V.value]);
          lds_barrier();
          if (k + PF < nk) load_regs(k + PF, g[V.value]);
          if (k == 0) begin(0, wm, w);
          else reload(k, wm, w);
          compute<false>(k, wm, sk, acc, w, nothing, nothing);
          flush(k);
        });
    }
    if constexpr (F8)
      if (nk > 0) add_block(acc[MF - 1], w.p[1], w.sp);
    flush(7);
    if constexpr (F32) {
#pragma unroll
      for (int f = 0; f < MF; ++f)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[f][j] = sum[f][j];
    }
    if constexpr (KS > 1) {
      // the groups' sums, through the stages' memory: this lane's results side
      // by side, 16 bytes apart from the next lane's
      lds_barrier();
      f32x4_t* part = (f32x4_t*)smem + (gwave * MF * NF) * 64 + (threadIdx.x & 63);
      if (grp > 0) {
#pragma unroll
        for (int f = 0; f < MF; ++f)
#pragma unroll
          for (int j = 0; j < NF; ++j) part[((grp - 1) * NW * MF * NF + f * NF + j) * 64] = acc[f][j];
      }
      __syncthreads();
      if (grp > 0) return;
#pragma unroll
      for (int q = 0; q < KS - 1; ++q)
#pragma unroll
        for (int f = 0; f < MF; ++f)
#pragma unroll
          for (int j = 0; j < NF; ++j) {
            const f32x4_t o = part[(q * NW * MF * NF + f * NF + j) * 64];
            acc[f][j] = Mm::add(acc[f][j], o);
          }
    }
    float bv[NF][4], sv[NF][4], sm[MF];
    load_bias(t, wn, bv);
    load_scales(t, wn, sv);
#pragma unroll
    for (int f = 0; f < MF; ++f)
      sm[f] = Mm::INT && nk > 0 ? a.sa[t.row0 + min(wm * TM + f * 16 + (int)(threadIdx.x & 15), t.rows - 1)] : 0.0f;
    wait_vmem();
    with_act(a.act, [&](auto act) { store<decltype(act)::value>(t, wm, wn, acc, bv, sv, sm); });
  }
};

template <int FMT, int BM, int BN, int WM, int WN, int S, int KS, bool DMA, bool KN>
__global__ __launch_bounds__(WM* WN* KS * 64) void expert_gemm_kernel(const ExpertArgs a) {
  typedef ExpertTileKernel<FMT, BM, BN, WM, WN, S, KS, DMA, KN> TK;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  ExpertTile x;
  int nt;
  if (!find_tile<BM>(a, ceil_div(a.N, BN), x, nt)) return;
  TK k(a, smem);
  k.run(x, nt);
}

// --- few rows: the weights are streamed once, straight into registers.
//
// A wave takes 16 columns of one expert and a slice of its K, 16 rows of
// tokens at a time (an expert with more rows runs the loop again).  A weight
// fragment's pieces come from global memory as the matrix instruction takes
// them (a wave reads whole 128-byte lines of 16 rows), kStreamDepth blocks in
// flight; with SPL slices the waves' partial sums are added in LDS in slice
// order.  What bounds it is the weights' bytes and one trip to HBM: no LDS
// staging, no barrier before the sums, and enough waves that their loads cover
// the latency.  One row of 4096 x 4096 e4m3: 5.8 us (2.9 TB/s); of 8192 x 8192:
// 13 us (5.1 TB/s).
constexpr int kStreamWaves = 8, kStreamDepth = 4;

template <int FMT>
__global__ __launch_bounds__(kStreamWaves * 64) void expert_stream_kernel(const ExpertArgs a, int SPL) {
  typedef FmtOps<FMT> Mm;
  typedef typename Mm::Frag Frag;
  constexpr bool F8 = Mm::F8;
  constexpr int ESZ = Mm::ESZ, KE = 128 / ESZ, U = kStreamDepth;
  __shared__ float part[kStreamWaves][4][64];
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int CT = kStreamWaves / SPL, NT = ceil_div(a.N, 16 * CT);
  const int e = blockIdx.x / NT, nt = blockIdx.x - e * NT;
  int lo, hi;
  expert_rows(a, e, lo, hi);
  if (a.offsets) {
    const int first = clampi(a.offsets[0], 0, a.T), last = max(first, clampi(a.offsets[a.E], 0, a.T));
    if (first != 0 || last != a.T) zero_outside(a, first, last);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  if (lo >= hi) return;                     // the whole block
  const int ct = wave / SPL, sl = wave - ct * SPL;
  const int n0 = (nt * CT + ct) * 16;
  const bool live = n0 < a.N;               // whole waves; the barrier below is passed by all
  const int64_t ld = (int64_t)a.K * ESZ;
  const int nk = ceil_div(a.K, KE), per = ceil_div(nk, SPL);
  const int k0 = sl * per, k1 = min(nk, k0 + per);
  const char* W = (const char*)a.B + ((int64_t)e * a.N + min(n0 + i, a.N - 1)) * ld;
  const float* sb = F8 ? a.sb + ((int64_t)e * ceil_div(a.N, 128) + min(n0, a.N - 1) / 128) * nk : nullptr;
  const int last_piece = (int)ld - 16;

  for (int row0 = lo; row0 < hi; row0 += 16) {
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    const int m = row0 + i, mr = min(m, hi - 1);
    const char* A = (const char*)a.A + (int64_t)mr * ld;
    if (live) {
#pragma unroll 1
      for (int k = k0; k < k1; k += U) {
        u32x4_t wx[U], wy[U], ax[U], ay[U];
        float sa[U], sw[U];
        // a block past the slice is read again from its last one, a piece past K
        // from the row's last one
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int kk = min(k + u, k1 - 1), o = kk * 128 + g * 16;
          const int px = min(o, last_piece), py = min(o + 64, last_piece);
          wx[u] = *(const u32x4_t*)(W + px);
          wy[u] = *(const u32x4_t*)(W + py);
          ax[u] = *(const u32x4_t*)(A + px);
          ay[u] = *(const u32x4_t*)(A + py);
          if constexpr (F8) {
            sw[u] = sb[kk];
            sa[u] = a.sa[(int64_t)kk * a.T + mr];
          }
        }
        __builtin_amdgcn_sched_barrier(0);      // every load goes out before the first product
        const u32x4_t zero = {0u, 0u, 0u, 0u};
        f32x4_t chain = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int o = (k + u) * 128 + g * 16;
          const bool in = k + u < k1;
          // what was read again counts as zeros on both sides: an infinity on
          // either would make 0 * inf (8-bit codes have none, and a NaN among
          // the weights has made its column's sum NaN already)
          const bool px = in && o <= last_piece, py = in && o + 64 <= last_piece;
          const Frag b = Mm::widen(ESZ == 1 || px ? wx[u] : zero, ESZ == 1 || py ? wy[u] : zero);
          const Frag x = Mm::widen(px ? ax[u] : zero, py ? ay[u] : zero);
          if constexpr (F8) {
            const f32x4_t p = Mm::block(b, x);
            const float s = in ? sa[u] * sw[u] : 0.0f;      // (0 * inf again)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(s, p[r], acc[r]);
          } else {
            chain = Mm::template half<0>(b, x, chain);
            chain = Mm::template half<1>(b, x, chain);
          }
        }
        if constexpr (!F8) acc = Mm::add(acc, chain);
      }
    }
    if (SPL > 1) {
      if (row0 > lo) __syncthreads();
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][r][lane] = acc[r];
      __syncthreads();
      if (sl != 0) continue;
      for (int q = 1; q < SPL; ++q)
        acc = Mm::add(acc, f32x4_t{part[wave + q][0][lane], part[wave + q][1][lane], part[wave + q][2][lane],
                                   part[wave + q][3][lane]});
    }
    const int n = n0 + g * 4;
    if (!live || m >= hi || n >= a.N) continue;
    float v[4];
    const float sm = Mm::INT && nk > 0 ? a.sa[m] : 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float bv = 0.0f;
      const float sv = Mm::INT && nk > 0 && n + r < a.N ? a.sb[(int64_t)e * a.N + n + r] : 0.0f;
      if (a.bias && n + r < a.N) {
        const int64_t at = (int64_t)e * a.N + n + r;
        bv = a.out_dt == DT_F32 ? ((const float*)a.bias)[at] : bf16_to_f32(((const uint16_t*)a.bias)[at]);
      }
      v[r] = apply_act(a.act, Mm::value(acc[r], sm, sv) + bv);
    }
    const int64_t at = (int64_t)m * a.N + n;
    if (a.out_dt == DT_F32) {
      float* y = (float*)a.Y + at;
      if (n + 3 < a.N) {
        ((Bytes16*)y)->v = u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < a.N) y[r] = v[r];
      }
    } else {
      uint16_t* y = (uint16_t*)a.Y + at;
      const u32x2_t o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      if (n + 3 < a.N) {
        ((Bytes8*)y)->v = o;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < a.N) y[r] = (uint16_t)(o[r / 2] >> (16 * (r % 2)));
      }
    }
  }
}

template <int FMT>
int launch_expert_stream(const ExpertArgs& a, hipStream_t s) {
  // slices of at least kStreamDepth blocks of K, so that a wave has as many in flight
  const int nk = ceil_div(a.K, 128 / FmtOps<FMT>::ESZ);
  int spl = 1;
  while (spl < kStreamWaves && nk > spl * kStreamDepth) spl *= 2;
  const int ct = kStreamWaves / spl;
  const int64_t blocks = (int64_t)a.E * ceil_div(a.N, 16 * ct);
  if (!fits_one_launch(blocks, kStreamWaves * 64)) return kNoGrid;
  hipLaunchKernelGGL((expert_stream_kernel<FMT>), dim3((uint32_t)blocks), dim3(kStreamWaves * 64), 0, s, a, spl);
  return (int)hipGetLastError();
}

// --- which tile
//
// A tile's time on this card, measured over uniform problems (microseconds):
// a round of blocks, one on each of the 256 CUs, takes o + c1 * nk for nk
// blocks of 128 bytes of K; with `per` blocks on every CU, o + c * nk.
struct TileCost {
  const char* name;
  int bm, bn, per;
  double o, c1, c;
};
constexpr int kCus = 256;

// The estimate for this call.  The host knows only the rows per expert on
// average: an expert's last tile is taken to be half full.
inline double tile_time(const ExpertArgs& a, int esz, const TileCost& t) {
  const double experts = a.offsets ? (a.E < a.T ? a.E : a.T) : 1, rows = a.T / experts;
  double tall = ceil_div(a.T, t.bm);
  if (experts > 1) tall = experts * (rows / t.bm + 0.5 > 1 ? rows / t.bm + 0.5 : 1);
  const double tiles = tall * ceil_div(a.N, t.bn), nk = ((int64_t)a.K * esz + 127) / 128;
  const double slots = (double)kCus * t.per;
  const double full = (double)(int64_t)(tiles / slots), rest = tiles - full * slots;
  double time = full * (t.o + t.c * nk);
  if (rest > 0) {
    // (as slow as the CUs that hold the most blocks)
    const int most = (int)((rest + kCus - 1) / kCus);
    time += t.o + nk * (t.c1 + (t.per > 1 ? (t.c - t.c1) * (most - 1) / (t.per - 1) : 0));
  }
  return time;
}
template <int N>
inline int best_tile(const ExpertArgs& a, int esz, const TileCost (&t)[N]) {
  int best = 0;
  for (int i = 1; i < N; ++i)
    if (tile_time(a, esz, t[i]) < tile_time(a, esz, t[best])) best = i;
  return best;
}
// Whether an expert has one fragment of rows or less and the tiles are too few
// to fill the chip (one token through 4096 x 4096 e4m3: 6.0 us streamed, 12.4
// us on 32 x 64 tiles; 16 rows over 8 experts of 4096 x 1024 bf16, 512 tiles:
// 14.4 us streamed, 12.0 on tiles).
inline bool stream_pays(const ExpertArgs& a, int esz) {
  const int64_t experts = a.offsets ? (a.E < a.T ? a.E : a.T) : 1;
  return a.T <= 16 * experts && experts * ceil_div(a.N, 64) < kCus && (int64_t)a.K * esz >= 1024;
}

// The named variant's place in the table, or -1.
template <int N>
inline int named_tile(const char* name, const TileCost (&t)[N]) {
  for (int i = 0; i < N; ++i)
    if (strcmp(name, t[i].name) == 0) return i;
  return -1;
}
// Which kernel a call takes: an index of its table, or one of these.
enum Pick : int { PICK_REGS = -2, PICK_REGS_LARGE = -3, PICK_STREAM = -4, PICK_NONE = -1 };
// Rows from any address go through registers: 128 x 128 tiles once those
// number two for every CU, else 64 x 64.
inline int pick_regs(const ExpertArgs& a) {
  const int64_t experts = a.offsets ? (a.E < a.T ? a.E : a.T) : 1;
  const int64_t tall = a.T / 128 > experts ? a.T / 128 : experts;
  return tall * ceil_div(a.N, 128) >= 2 * kCus && a.T >= 128 * experts ? PICK_REGS_LARGE : PICK_REGS;
}
template <int N>
inline int pick_variant(ExpertArgs& a, int esz, const TileCost (&t)[N]) {
  int p;
  if (a.force) {
    p = !strcmp(a.force, "regs") ? PICK_REGS : !strcmp(a.force, "regs128") ? PICK_REGS_LARGE
        : !strcmp(a.force, "stream") && !a.kn && a.vec ? PICK_STREAM : a.vec ? named_tile(a.force, t) : PICK_NONE;
  } else if (!a.vec) {
    p = pick_regs(a);
  } else if (!a.kn && stream_pays(a, esz)) {
    p = PICK_STREAM;
  } else {
    p = best_tile(a, esz, t);
  }
  a.chosen = p >= 0 ? t[p].name : p == PICK_REGS ? "regs" : p == PICK_REGS_LARGE ? "regs128" : "stream";
  return p;
}

// Reading the weights of every expert that can have rows, at 5 TB/s.
inline double weights_time(const ExpertArgs& a, int esz) {
  const double experts = a.offsets ? (a.E < a.T ? a.E : a.T) : 1;
  return experts * a.N * a.K * esz / 5e6;
}

template <int FMT, int BM, int BN, int WM, int WN, int S, int KS, bool DMA, bool KN>
int launch_expert_tile(const ExpertArgs& a, hipStream_t s) {
  typedef ExpertTileKernel<FMT, BM, BN, WM, WN, S, KS, DMA, KN> TK;
  const int64_t tall = a.offsets ? expert_tile_bound(a.T, a.E, BM) : ceil_div(a.T, BM);
  const int64_t blocks = tall * ceil_div(a.N, BN);
  if (!fits_one_launch(blocks, TK::TH)) return kNoGrid;
  hipLaunchKernelGGL((expert_gemm_kernel<FMT, BM, BN, WM, WN, S, KS, DMA, KN>), dim3((uint32_t)blocks), dim3(TK::TH),
                     TK::LDS_BYTES, s, a);
  return (int)hipGetLastError();
}

}  // namespace ox
