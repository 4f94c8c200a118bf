// k_moe.hip -- a routed feed-forward layer for up to 64 tokens, in two kernels.
//
//   up:    router scores -> each token's best experts and their weights;
//          h = act(W1[e] x + b1[e]), or act(gate) * up where W1 holds both
//   down:  Y = sum over a token's experts of weight * (W2[e] h + b2[e])
//
// With so few tokens the chosen experts' weights are what there is to move: they
// are read once, straight into registers, as the matrix instructions take them
// (16 rows of weights x 16 tokens).  A wave takes two or four fragments of 16 rows
// and a range of K, so that a fragment of the tokens serves them all, and the
// waves' sums are added in their order: every sum's order depends on the sizes and
// on the routing alone.
//
// Every block of the first kernel routes all tokens for itself (a launch and a
// trip to memory less than a kernel of its own); its last block does nothing else
// and leaves the result for the second kernel.
// The second kernel's K is the experts' hidden rows one after the other; it is
// cut into equal ranges whatever the routing.  Blocks that share columns leave
// fp32 sums, and the last of them to arrive adds them in order.
//
// Precision.  bf16 weights (and e4m3 ones, widened: exact) meet bf16 tokens in
// the bf16 instruction, whose sums are fp32; h is kept as two bf16 numbers (16
// bits of significand, off by 2^-17 at most), each of which meets W2, so that the
// only rounding that counts is Y's.  Every batch of K starts a chain of sums from zero.
#include "expert_gemm.hpp"

namespace ox {

namespace {

constexpr int kMoeThreads = 512, kMoeWaves = kMoeThreads / 64;
constexpr int kPairs = kMoeTokens * kMoeTop;

__device__ __forceinline__ f32x4_t add4(f32x4_t a, f32x4_t b) {
#pragma unroll
  for (int r = 0; r < 4; ++r) a[r] += b[r];
  return a;
}

__device__ __forceinline__ float moe_act(int act, float v) {
  return act == ACT_SILU ? v / (1.0f + expf(-v)) : apply_act(act, v);
}

// ------------------------------------------------------------- routing --

// What every block finds for itself: the tokens of each expert, as bits.
struct Route {
  uint64_t mask[kMoeExperts];
};

// What the first kernel's last block leaves for the second, in the workspace:
// the slots (token, expert) in the order of the experts.
struct RouteOut {
  int nact, slots;
  int act[kMoeExperts], off[kMoeExperts + 1];      // the experts that have tokens, and their first slots
  int tok[kPairs];
  float weight[kPairs];
};

// Scores as whole numbers in their order; 0 for what is never chosen (NaN, -inf)
__device__ __forceinline__ uint32_t score_key(float s) {
  if (!(s > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(s == 0.0f ? 0.0f : fminf(s, 3.4028234663852886e38f));      // (-0 and 0 are a tie)
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}

// over the sixteen lanes of a row, in every lane (quad_perm 1,0,3,2 and 2,3,0,1,
// then the mirrored half row and row)
template <typename F>
__device__ __forceinline__ uint32_t row16(uint32_t v, F&& f) {
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));
  return f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  return row16(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint32_t row16_min(uint32_t v) {
  return row16(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
__device__ __forceinline__ float row16_sum(float v) {
  return __uint_as_float(row16(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// Sixteen lanes take a token, with PL scores each: its best expert is found
// `top` times, and lane j of the sixteen keeps the j-th.  A wave does four tokens
// at once (one token a wave, over all lanes, took 12 us for 64 tokens and 8 of 64
// experts).  WEIGHTS: the block that writes what comes of it.
template <int PL, bool WEIGHTS>
__device__ __forceinline__ void route_tokens(const MoeArgs& a, Route& rt, int16_t* choice, float* weight) {
  const int r = threadIdx.x & 15;
  for (int t0 = 0; t0 < a.T; t0 += kMoeThreads / 16) {
    const int t = t0 + threadIdx.x / 16;
    const bool in = t < a.T;
    uint32_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = i * 16 + r;
      key[i] = 0u;
      if (in && e < a.E) {
        const int64_t at = (int64_t)t * a.E + e;
        key[i] = score_key(a.scores_dt == DT_F32 ? ((const float*)a.scores)[at] : bf16_to_f32(((const uint16_t*)a.scores)[at]));
      }
    }
    if (t0 == 0) {      // (under the first loads)
      for (int e = threadIdx.x; e < a.E; e += kMoeThreads) rt.mask[e] = 0;
      __syncthreads();
    }
    uint32_t mine = 0u, best = 0u;
    int expert = -1;
    float all = 0.0f;
#pragma unroll 1
    for (int j = 0; j < a.top; ++j) {
      uint32_t m = key[0];
#pragma unroll
      for (int i = 1; i < PL; ++i) m = max(m, key[i]);
      m = row16_max(m);
      // the lowest of the experts that have it
      uint32_t e = 0xffffu;
#pragma unroll
      for (int i = PL - 1; i >= 0; --i) e = key[i] == m ? i * 16 + r : e;
      e = row16_min(e);
      if (j == 0) {
        best = m;
        if (WEIGHTS && !a.renormalise) {
#pragma unroll 1
          for (int i = 0; i < PL; ++i) all += key[i] ? expf(key_score(key[i]) - key_score(best)) : 0.0f;
          all = row16_sum(all);
        }
      }
      if (r == j && m) {
        mine = m;
        expert = (int)e;
      }
#pragma unroll
      for (int i = 0; i < PL; ++i) key[i] = (uint32_t)(i * 16 + r) == e ? 0u : key[i];
    }
    if (in && expert >= 0) atomicOr((unsigned long long*)&rt.mask[expert], 1ull << t);
    if constexpr (WEIGHTS) {
      const float p = mine ? expf(key_score(mine) - key_score(best)) : 0.0f;
      if (a.renormalise) all = row16_sum(p);
      if (in && r < a.top) {
        choice[t * kMoeTop + r] = (int16_t)expert;
        weight[t * kMoeTop + r] = mine ? p / all : 0.0f;
      }
    }
  }
  __syncthreads();
}
template <bool WEIGHTS>
__device__ __forceinline__ void route(const MoeArgs& a, Route& rt, int16_t* choice = nullptr, float* weight = nullptr) {
  if (a.E <= 16) route_tokens<1, WEIGHTS>(a, rt, choice, weight);
  else if (a.E <= 64) route_tokens<4, WEIGHTS>(a, rt, choice, weight);
  else if (a.E <= 128) route_tokens<8, WEIGHTS>(a, rt, choice, weight);
  else route_tokens<32, WEIGHTS>(a, rt, choice, weight);
}

// Experts that have tokens.
__device__ __forceinline__ int active_experts(const MoeArgs& a, const Route& rt) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int base = 0; base < a.E; base += 64) n += __popcll(__ballot(base + lane < a.E && rt.mask[min(base + lane, a.E - 1)]));
  return n;
}
// The ai-th of them: its index, first slot, and tokens (a wave's work).
struct Active {
  int e, first;
  uint64_t mask;
};
__device__ __forceinline__ Active find_active(const MoeArgs& a, const Route& rt, int ai) {
  const int lane = threadIdx.x & 63;
  Active r = {0, 0, 0};
  for (int base = 0; base < a.E; base += 64) {
    const uint64_t m = base + lane < a.E ? rt.mask[base + lane] : 0;
    const uint64_t has = __ballot(m != 0);
    const int n = __popcll(m), s = wave_scan(n);
    if (ai < __popcll(has)) {
      // the lane whose bit is the ai-th
      const uint64_t at = __ballot(m != 0 && (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(has >> 32),
                                                                           __builtin_amdgcn_mbcnt_lo((uint32_t)has, 0)) == ai);
      const int l = __ffsll((unsigned long long)at) - 1;
      r.e = base + l;
      r.first += __builtin_amdgcn_readlane(s - n, l);
      r.mask = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)m, l) |
               (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(m >> 32), l) << 32;
      return r;
    }
    ai -= __popcll(has);
    r.first += __builtin_amdgcn_readlane(s, 63);
  }
  return r;
}
// Lane i gets the i-th token of the mask.
__device__ __forceinline__ int tokens_of(uint64_t mask) {
  const int lane = threadIdx.x & 63;
  const int before = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
  const bool has = (mask >> lane) & 1;
  return __builtin_amdgcn_ds_permute(4 * (has ? before : __popcll(mask) + lane - before), lane);
}

// The first kernel's last block: what the second kernel and the caller read.
__device__ __forceinline__ void write_route(const MoeArgs& a, Route& rt, char* smem) {
  float* weight = (float*)smem;                                        // [kMoeTokens][kMoeTop]
  int16_t* choice = (int16_t*)(smem + kPairs * 4);
  uint16_t* first = (uint16_t*)(smem + kPairs * 6);                    // [kMoeExperts]: an expert's first slot
  route<true>(a, rt, choice, weight);
  RouteOut* ro = (RouteOut*)a.route;
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int acts = 0, slots = 0;
    for (int base = 0; base < a.E; base += 64) {
      const int e = base + lane, n = e < a.E ? __popcll(rt.mask[e]) : 0;
      const int s = wave_scan(n), k = wave_scan(n ? 1 : 0);
      if (e < a.E) first[e] = (uint16_t)(slots + s - n);
      if (n) {
        ro->act[acts + k - 1] = e;
        ro->off[acts + k - 1] = slots + s - n;
      }
      slots += __builtin_amdgcn_readlane(s, 63);
      acts += __builtin_amdgcn_readlane(k, 63);
    }
    if (lane == 0) {
      ro->off[acts] = slots;
      ro->nact = acts;
      ro->slots = slots;
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < a.T * a.top; p += kMoeThreads) {
    const int t = p / a.top, j = p - t * a.top, e = choice[t * kMoeTop + j];
    const float w = weight[t * kMoeTop + j];
    if (e >= 0) {
      const int slot = first[e] + __popcll(rt.mask[e] & ((1ull << t) - 1));
      ro->tok[slot] = t;
      ro->weight[slot] = w;
    }
    if (a.experts) a.experts[p] = e;
    if (a.weights) a.weights[p] = w;
  }
  for (int i = threadIdx.x; i < a.tiles; i += kMoeThreads) a.counters[i] = 0;
}

// ------------------------------------------------------------ products --

// A pointer in scalar registers, known to be global memory: loads take it as
// their base beside a 32-bit offset.
#define OX_GLOBAL __attribute__((address_space(1)))
typedef const OX_GLOBAL char* Global;
__device__ __forceinline__ Global uniform_global(const void* p) {
  return (Global)(uintptr_t)uniform_ptr((const char*)p);
}

// The same number, of which the compiler knows nothing: it would add a lane's
// offsets to the bases once for all, 64 bits for every load, and spill.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// bytes [0, n) of 16 at p, whole elements of ESZ bytes; zeros behind them (n <= 0:
// none)
template <int ESZ>
__device__ __forceinline__ u32x4_t part_of_piece(Global p, int n) {
  if (n >= 16) return ((const OX_GLOBAL Bytes16*)p)->v;
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; i += ESZ)
    if (i < n) {
      if constexpr (ESZ == 4) w[i / 4] = *(const OX_GLOBAL uint32_t*)(p + i);
      else if constexpr (ESZ == 2) w[i / 4] |= (uint32_t)*(const OX_GLOBAL uint16_t*)(p + i) << (8 * (i % 4));
      else w[i / 4] |= (uint32_t)(uint8_t)p[i] << (8 * (i % 4));
    }
  return u32x4_t{w[0], w[1], w[2], w[3]};
}

// NF fragments of 16 rows of weights times MF fragments of 16 tokens, over steps
// [k0, k1) of K (128 bytes of a weight row each).
// ONE: a fragment's sixteen rows of weights share a scale (e4m3).
template <int FMT, int NF, int MF, bool ONE, int BUDGET>
struct MoeProduct {
  typedef FmtOps<FMT> Mm;
  typedef typename Mm::Frag Frag;
  static constexpr bool F8 = FMT == FMT_FP8X;
  static constexpr int KE = 128 / Mm::ESZ;         // K of a step
  static constexpr int XP = F8 ? 4 : 2;            // pieces of a token's step
  static constexpr int XB = F8 ? 256 : 128;        // its bytes
  // Steps in flight, as many as BUDGET registers hold.
  static constexpr int REGS = NF * 8 + MF * XP * 4;
  static constexpr int U = BUDGET / REGS;
  static_assert(U >= 1, "a step fits");

  // Bases for all lanes, and this lane's offsets from them (its row, its first
  // piece): a load is a scalar base, a 32-bit offset and a constant.
  Global w[NF];                // the fragments' first rows of weights
  uint32_t wo[NF];
  Global x;                    // the first token
  uint32_t xo[MF];
  bool on[MF];                 // this lane's column of the fragment holds a token
  int frags;                   // token fragments that hold tokens
  const float* sw[NF];         // e4m3: the scales of the fragment's first row (step 0)
  int sw_next[NF], sw_rows[NF];      // ... those of its last row, from there; the rows in front of them
  int K;

  // piece i of a token's step, behind the lane's first
  static __device__ __forceinline__ constexpr int x_at(int i) { return F8 ? (i & 1) * 16 + (i >> 1) * 128 : i * 64; }

  struct Step {
    u32x4_t w[NF][2], x[MF][XP];
    float s[NF][ONE ? 1 : 2];
  };
  // PART: K may end inside the step
  template <bool PART>
  __device__ __forceinline__ void load(int k, Step& st) const {
    const int g = (threadIdx.x & 63) >> 4;
    const int left = (int)min((int64_t)XB, ((int64_t)K - (int64_t)k * KE) * Mm::ESZ);      // bytes of a weight row
    const int64_t wk = (int64_t)k * 128, xk = (int64_t)k * XB;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const Global p = w[f] + wk;
      const uint32_t o = opaque(wo[f]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if constexpr (PART) {
          st.w[f][i] = part_of_piece<Mm::ESZ>(p + o + i * 64, left - g * 16 - i * 64);
          __builtin_amdgcn_sched_barrier(0);      // (one at a time: registers)
        } else {
          st.w[f][i] = ((const OX_GLOBAL Bytes16*)(p + o + i * 64))->v;
        }
    }
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      if (m > 0 && m >= frags) break;
      if (!on[m]) continue;      // (its column's sums are never looked at)
      const Global p = x + xk;
      const uint32_t o = opaque(xo[m]);
#pragma unroll
      for (int i = 0; i < XP; ++i)
        if constexpr (PART) {
          st.x[m][i] = part_of_piece<F8 ? 2 : Mm::ESZ>(p + o + x_at(i), (left - g * 16) * (XB / 128) - x_at(i));
          __builtin_amdgcn_sched_barrier(0);
        } else {
          st.x[m][i] = ((const OX_GLOBAL Bytes16*)(p + o + x_at(i)))->v;
        }
    }
    if constexpr (F8) {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        typedef const __attribute__((address_space(4))) float* Scalar;
        st.s[f][0] = *(Scalar)(uintptr_t)(sw[f] + k);      // (by scalar loads)
        if constexpr (!ONE) st.s[f][1] = *(Scalar)(uintptr_t)(sw[f] + sw_next[f] + k);
      }
    }
  }
  static __device__ __forceinline__ Frag token_frag(const u32x4_t (&p)[XP]) {
    Frag f;
#pragma unroll
    for (int i = 0; i < XP; ++i) f.v[i] = p[i];
    return f;
  }
  __device__ __forceinline__ void multiply(const Step& st, f32x4_t (&acc)[NF][MF]) const {
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const Frag b = Mm::widen(st.w[f][0], st.w[f][1]);
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        if (m > 0 && m >= frags) break;
        f32x4_t chain = {0.f, 0.f, 0.f, 0.f};
        const Frag t = token_frag(st.x[m]);
        chain = Mm::template half<0>(b, t, chain);
        chain = Mm::template half<1>(b, t, chain);
        if constexpr (F8) {
          chain = Mm::template half<2>(b, t, chain);
          chain = Mm::template half<3>(b, t, chain);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool front = ONE || ((threadIdx.x & 63) >> 4) * 4 + r < sw_rows[f];
          acc[f][m][r] = F8 ? __builtin_fmaf(front ? st.s[f][0] : st.s[f][ONE ? 0 : 1], chain[r], acc[f][m][r])
                            : acc[f][m][r] + chain[r];
        }
        // The addition stays here: moved behind the next branch, where it is taken,
        // it came without the wait that the matrix instruction's result needs.
        asm volatile("" : "+v"(acc[f][m]));
      }
    }
  }
  // All steps [first, end).  They are taken in turn from an eighth of the way that
  // `phase` gives: waves that all begin with a row's first bytes, and rows that
  // are a power of two apart, would keep asking the same few memory channels.
  __device__ __forceinline__ void run(int first, int end, int phase, f32x4_t (&acc)[NF][MF]) const {
    const int k0 = __builtin_amdgcn_readfirstlane(first), k1 = __builtin_amdgcn_readfirstlane(end);
    if (K == 0) return;
    const int whole = min(k1, K / KE);      // steps that K does not end inside
    const int turned = __builtin_amdgcn_readfirstlane(max(0, whole - k0) * phase / 8);
    auto at = [&](int j) { return j + turned < whole ? j + turned : j + turned - (whole - k0); };
    int k = k0;
    if (k + U <= whole) {
      // U steps in flight: each is loaded again, U further on, as soon as it is
      // multiplied (the order is pinned: loads would sink to their uses)
      Step st[U];
#pragma unroll
      for (int u = 0; u < U; ++u) load<false>(at(k + u), st[u]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll 1
      for (; k + 2 * U <= whole; k += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          multiply(st[u], acc);
          load<false>(at(k + U + u), st[u]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      // what is left: fewer than U steps behind those in flight
#pragma unroll
      for (int u = 0; u < U; ++u) {
        multiply(st[u], acc);
        if (u + 1 < U && k + U + u < whole) load<false>(at(k + U + u), st[u]);
        __builtin_amdgcn_sched_barrier(0);
      }
      k += U;
#pragma unroll
      for (int u = 0; u + 1 < U; ++u)
        if (k + u < whole) multiply(st[u], acc);
      k = max(k, whole);
    }
    if (k < whole) {      // fewer than U in all: their loads together
      Step st[U];
#pragma unroll
      for (int u = 0; u + 1 < U; ++u)
        if (k + u < whole) load<false>(at(k + u), st[u]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u + 1 < U; ++u)
        if (k + u < whole) multiply(st[u], acc);
      k = whole;
    }
    if (k < k1) {
      Step st;
      load<true>(k, st);
      multiply(st, acc);
    }
  }
  // token fragment m: this lane's row, `ld` bytes to a row, if it holds one
  __device__ __forceinline__ void token(int m, bool holds, uint32_t row, uint32_t ld) {
    on[m] = holds;
    xo[m] = row * ld + ((threadIdx.x & 63) >> 4) * (XB / 8);
  }
  // fragment f: rows n .. n + 15 of expert e's `rows` rows, of which those below
  // `end` count
  __device__ __forceinline__ void weights(int f, const void* W, const float* scales, int e, int rows, int n, int end) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    w[f] = uniform_global((const char*)W + ((int64_t)e * rows + n) * K * Mm::ESZ);
    wo[f] = (uint32_t)min(i, end - 1 - n) * (uint32_t)K * Mm::ESZ + g * 16;
    if constexpr (F8) {
      const int nb = ceil_div(rows, 128), kb = ceil_div(K, 128), b = min(n, end - 1) / 128;
      sw[f] = uniform_ptr(scales + ((int64_t)e * nb + b) * kb);
      sw_next[f] = min(n + 15, end - 1) / 128 > b ? kb : 0;
      sw_rows[f] = (b + 1) * 128 - n;
    }
  }
};

// Four sums that a block of another XCD reads: past the L2s, which are not
// coherent, by accesses of agent scope (an agent fence instead, which writes the
// whole L2 back, cost 80 us in a kernel of 512 blocks).
__device__ __forceinline__ void store_shared(f32x4_t* p, f32x4_t v) {
  uint64_t w[2];
  __builtin_memcpy(w, &v, 16);
  __hip_atomic_store((uint64_t*)p, w[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store((uint64_t*)p + 1, w[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4_t load_shared(const f32x4_t* p) {
  uint64_t w[2] = {__hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT),
                   __hip_atomic_load((const uint64_t*)p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)};
  f32x4_t v;
  __builtin_memcpy(&v, w, 16);
  return v;
}

// A hidden value of a slot, as the second kernel reads it.
template <int FMT>
__device__ __forceinline__ void store_hidden(const MoeArgs& a, int slot, int n, float h) {
  if constexpr (FMT == FMT_F32) {
    ((float*)a.hidden)[(int64_t)slot * a.ldh + n] = h;
  } else {
    const uint16_t hi = (uint16_t)pack_bf16x2(h, 0.0f);
    const float v = bf16_to_f32(hi), lo = __builtin_isfinite(v) ? h - v : 0.0f;
    uint16_t* p = (uint16_t*)a.hidden + (int64_t)slot * 2 * a.ldh + n;      // the two parts in turn
    p[0] = hi;
    p[a.ldh] = (uint16_t)pack_bf16x2(lo, 0.0f);
  }
}
template <int FMT>
__device__ __forceinline__ float value_at(const void* p, int64_t at) {
  return FMT == FMT_F32 ? ((const float*)p)[at] : bf16_to_f32(((const uint16_t*)p)[at]);
}

// Units of one expert x a group of column tiles, in turn over the grid's blocks
// (the last of them routes for the second kernel instead).  A column tile is 16
// gate rows and the 16 up rows beside them, or 32 rows.
template <int FMT, int MF, bool ONE>
__global__ __launch_bounds__(kMoeThreads, 4) void moe_up_kernel(const MoeArgs a) {
  typedef MoeProduct<FMT, 2, MF, ONE, 80> MP;
  constexpr int LANE = 4, SET = 64 * LANE + 48;      // floats: a lane's results, a fragment's (16 apart every 16 lanes: all banks)
  __shared__ Route rt;
  __shared__ __attribute__((aligned(16))) float part[2][kMoeWaves][2 * MF * SET];
  if (blockIdx.x == gridDim.x - 1) {
    write_route(a, rt, (char*)part);
    return;
  }
  route<false>(a, rt);
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wide = a.gated ? 2 * a.H : a.H, per = a.gated ? 16 : 32, tiles = ceil_div(a.H, per);
  const int nk = ceil_div(a.D, MP::KE);
  // Slices of K: as few as still give every block two units (64 experts of 1024 x
  // 2048, 4096 tiles: 188 us with two slices, 195 with eight, 208 with one)
  const int experts = active_experts(a, rt), blocks = gridDim.x - 1;
  int SPL = 1;
  while (SPL < a.slices && experts * ceil_div(tiles, kMoeWaves / SPL) < 2 * blocks) SPL *= 2;
  const int CT = kMoeWaves / SPL, groups = ceil_div(tiles, CT), units = experts * groups;
  const int ct = __builtin_amdgcn_readfirstlane(wave / SPL), sl = wave - ct * SPL;
  const int k0 = (int)((int64_t)nk * sl / SPL), k1 = (int)((int64_t)nk * (sl + 1) / SPL);
  int turn = 0;
  for (int unit = blockIdx.x; unit < units; unit += blocks) {
    const int ai = __builtin_amdgcn_readfirstlane(unit / groups), tile0 = (unit - ai * groups) * CT;
    const Active ac = find_active(a, rt, ai);
    const int e = ac.e, count = __popcll(ac.mask), tile = tile0 + ct, n0 = tile * per;
    const int tok = tokens_of(ac.mask);
    const bool live = tile < tiles;      // whole waves; the barriers below are passed by all
    MP mp;
    mp.K = a.D;
    mp.x = uniform_global(a.X);
    if (live) {
      mp.weights(0, a.W1, a.s1, e, wide, n0, a.H);
      if (a.gated) mp.weights(1, a.W1, a.s1, e, wide, a.H + n0, wide);
      else mp.weights(1, a.W1, a.s1, e, wide, min(n0 + 16, a.H - 1), a.H);
    }
    for (int s0 = 0; s0 < count; s0 += 16 * MF, turn ^= 1) {
      f32x4_t acc[2][MF];
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int m = 0; m < MF; ++m) acc[f][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      mp.frags = ceil_div(count - s0, 16);
#pragma unroll
      for (int m = 0; m < MF; ++m)
        mp.token(m, s0 + m * 16 + i < count, __builtin_amdgcn_ds_bpermute(4 * min(s0 + m * 16 + i, count - 1), tok), a.D * (FMT == FMT_F32 ? 4 : 2));
      if (live) mp.run(k0, k1, (blockIdx.x + ct) & 7, acc);
      float* to = part[turn][wave] + lane * LANE + g * 16;
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int m = 0; m < MF; ++m) *(f32x4_t*)(to + (f * MF + m) * SET) = acc[f][m];
      __syncthreads();
      // Every wave: four tokens x 16 columns of a tile, from the slices' sums in
      // their order.  A wave may be a pass ahead of one that still reads, no more:
      // two sets in turn.
      const int quads = (min(count - s0, 16 * MF) + 3) / 4;
#pragma unroll 1
      for (int w = wave; w < CT * quads; w += kMoeWaves) {
        const int c = w / quads, q = w - c * quads, t = q * 4 + g, col = i;
        const int at = ((col >> 2) * 16 + (t & 15)) * LANE + (col >> 2) * 16 + (col & 3) + (t >> 4) * SET;
        float v[2] = {0.0f, 0.0f};
        for (int x = 0; x < SPL; ++x) {
          v[0] += part[turn][c * SPL + x][at];
          v[1] += part[turn][c * SPL + x][at + MF * SET];
        }
        const int slot = s0 + t, n = (tile0 + c) * per + col;
        if (slot >= count || n >= a.H) continue;
        if (a.gated) {
          if (a.b1) {
            v[0] += value_at<FMT>(a.b1, (int64_t)e * wide + n);
            v[1] += value_at<FMT>(a.b1, (int64_t)e * wide + a.H + n);
          }
          store_hidden<FMT>(a, ac.first + slot, n, moe_act(a.act, v[0]) * v[1]);
        } else {
#pragma unroll 1
          for (int f = 0; f < 2; ++f) {
            if (n + f * 16 >= a.H) break;
            const float b = a.b1 ? value_at<FMT>(a.b1, (int64_t)e * wide + n + f * 16) : 0.0f;
            store_hidden<FMT>(a, ac.first + slot, n + f * 16, moe_act(a.act, (f ? v[1] : v[0]) + b));
          }
        }
      }
    }
  }
}

// Block (tile, s): 16 NF columns of Y, range s of all the chosen
// experts' hidden rows.  A hidden row's two parts lie in neighbouring columns of
// a token fragment, which holds eight slots then, and their sums are added.
template <int FMT, int NF, int MF>
__global__ __launch_bounds__(kMoeThreads, 2) void moe_down_kernel(const MoeArgs a) {
  constexpr int PARTS = FMT == FMT_F32 ? 1 : 2, SLOTS = 16 / PARTS;      // of a hidden row; of a fragment
  typedef MoeProduct<FMT, NF, MF, true, 160> MP;
  constexpr int TILE = 16 * NF, QUADS = TILE / 4;
  extern __shared__ __attribute__((aligned(16))) float yw[];      // [waves][T][TILE]
  __shared__ RouteOut rt;
  __shared__ int last;
  const RouteOut* ro = (const RouteOut*)a.route;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // (all of it at once, before the number of experts is known)
  const int pairs = a.T * a.top, acts = min(a.E, pairs);
  for (int p = threadIdx.x; p < pairs; p += kMoeThreads) {
    rt.tok[p] = ro->tok[p];
    rt.weight[p] = ro->weight[p];
  }
  for (int p = threadIdx.x; p <= acts; p += kMoeThreads) {
    if (p < acts) rt.act[p] = ro->act[p];
    rt.off[p] = ro->off[p];
  }
  if (threadIdx.x == 0) rt.nact = ro->nact;
  float* mine = yw + wave * a.T * TILE;
  for (int p = lane; p < a.T * QUADS; p += 64) ((f32x4_t*)mine)[p] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  __syncthreads();

  const int tile = blockIdx.x / a.S, s = blockIdx.x - tile * a.S, n0 = tile * TILE;
  const int nk = max(1, ceil_div(a.H, MP::KE));
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(rt.nact) * nk, parts = (int64_t)a.S * kMoeWaves;
  int st = (int)(total * (s * kMoeWaves + wave) / parts);
  const int end = (int)(total * (s * kMoeWaves + wave + 1) / parts);
  MP mp;
  mp.K = a.H;
  while (st < end) {
    const int ai = __builtin_amdgcn_readfirstlane(st / nk), k0 = st - ai * nk, k1 = min(nk, k0 + end - st);
    const int e = __builtin_amdgcn_readfirstlane(rt.act[ai]), lo = __builtin_amdgcn_readfirstlane(rt.off[ai]);
    const int hi = __builtin_amdgcn_readfirstlane(rt.off[ai + 1]);
#pragma unroll
    for (int f = 0; f < NF; ++f) mp.weights(f, a.W2, a.s2, e, a.D, min(n0 + f * 16, a.D - 1), a.D);
    mp.x = uniform_global((const char*)a.hidden + (int64_t)lo * a.ldh * 4);
    for (int s0 = lo; s0 < hi; s0 += SLOTS * MF) {
      f32x4_t acc[NF][MF];
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int m = 0; m < MF; ++m) acc[f][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      mp.frags = ceil_div(hi - s0, SLOTS);
#pragma unroll
      for (int m = 0; m < MF; ++m)
        mp.token(m, s0 + m * SLOTS + i / PARTS < hi, (min(s0 + m * SLOTS + i / PARTS, hi - 1) - lo) * PARTS + i % PARTS, (uint32_t)a.ldh * (4 / PARTS));
      mp.run(k0, k1, (blockIdx.x + wave) & 7, acc);
      // into this wave's sums of the tokens (a token has one slot of an expert)
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        const int slot = s0 + m * SLOTS + i / PARTS;
        if constexpr (PARTS == 2) {
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              // The low part's sum, of the next lane.  It is finite where the high
              // part's is, or else met an infinite weight: that is the high part's to
              // show, with h's sign (a low part of zero, or of the other sign, would
              // make NaN of it).
              const float low = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(acc[f][m][r]), 0xB1, 0xf, 0xf, true));
              acc[f][m][r] += __builtin_isfinite(low) ? low : 0.0f;
            }
        }
        if (slot >= hi || i % PARTS != 0) continue;
        const float wt = rt.weight[slot];
        float* y = mine + rt.tok[slot] * TILE + g * 4;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          f32x4_t v = acc[f][m];
          if (a.b2 && k0 == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int n = n0 + f * 16 + g * 4 + r;
              if (n < a.D) v[r] += value_at<FMT>(a.b2, (int64_t)e * a.D + n);
            }
          }
          f32x4_t o = *(f32x4_t*)(y + f * 16);
#pragma unroll
          for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(wt, v[r], o[r]);
          *(f32x4_t*)(y + f * 16) = o;
        }
      }
    }
    st += k1 - k0;
  }
  __syncthreads();

  const int quads = a.T * QUADS;      // four columns of a token
  auto store = [&](int q, f32x4_t v) {
    const int t = q / QUADS, n = n0 + q % QUADS * 4;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < a.D) {
        const int64_t at = (int64_t)t * a.D + n + r;
        if constexpr (FMT == FMT_F32) ((float*)a.Y)[at] = v[r];
        else ((uint16_t*)a.Y)[at] = (uint16_t)pack_bf16x2(v[r], 0.0f);
      }
  };
  f32x4_t* ws = (f32x4_t*)a.partials + (int64_t)tile * a.S * quads;
  for (int q = threadIdx.x; q < quads; q += kMoeThreads) {
    f32x4_t v = ((f32x4_t*)yw)[q];
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w) v = add4(v, ((f32x4_t*)yw)[w * quads + q]);
    if (a.S == 1) store(q, v);
    else store_shared(ws + (int64_t)s * quads + q, v);
  }
  if (a.S == 1) return;
  // the last block of the tile adds the ranges in their order; every wave's
  // stores have arrived before its block counts itself
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(a.counters + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.S - 1;
  __syncthreads();
  if (!last) return;
  for (int q = threadIdx.x; q < quads; q += kMoeThreads) {
    // (eight loads at a time: one after the other they cost a trip to memory each)
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int p0 = 0; p0 < a.S; p0 += 8) {
      f32x4_t o[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) o[p] = load_shared(ws + (int64_t)min(p0 + p, a.S - 1) * quads + q);
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p0 + p < a.S) v = add4(v, o[p]);
    }
    store(q, v);
  }
}

// Ranges of K that the second kernel's tiles are cut into: about one block for
// every CU (two: one token 23.3 us, 21.7 with one; the others equal).
int moe_ranges(int64_t tiles) { return (int)((kCus + tiles - 1) / tiles); }

// UF, DF: token fragments at a time in the first and the second kernel; NF: weight
// fragments of a wave in the second.
template <int FMT, int UF, int NF, int DF>
int launch_pair(MoeArgs& a, int64_t steps, hipStream_t s) {
  a.tiles = ceil_div(a.D, 16 * NF);
  // no more ranges than give every wave a step
  int64_t S = moe_ranges(a.tiles);
  while (S > 1 && S * kMoeWaves > steps) S = (S + 1) / 2;
  a.S = (int)S;

  // (the up rows of a gated W1 start anywhere in a block of scales)
  if (FMT == FMT_FP8X && a.gated && a.H % 16 != 0)
    hipLaunchKernelGGL((moe_up_kernel<FMT, UF, FMT != FMT_FP8X>), dim3(a.up_blocks), dim3(kMoeThreads), 0, s, a);
  else
    hipLaunchKernelGGL((moe_up_kernel<FMT, UF, true>), dim3(a.up_blocks), dim3(kMoeThreads), 0, s, a);
  int rc = (int)hipGetLastError();
  if (rc) return rc;
  hipLaunchKernelGGL((moe_down_kernel<FMT, NF, DF>), dim3(a.tiles * a.S), dim3(kMoeThreads),
                     kMoeWaves * a.T * 16 * NF * 4, s, a);
  return (int)hipGetLastError();
}

// More than 16 tokens: four weight fragments a wave, 64 columns of Y, where that
// still leaves every wave four steps: the tokens' pieces then serve twice as many
// weights (64 tokens, 8 of 64 bf16 experts of 1024 x 2048: 174 us, 182 with two;
// 4 of 32 e4m3 experts of 512 x 1024, one step a wave: 35.9 us, 30.5 with two).
// Up to 16 tokens both widths take the same time.
template <int FMT, int UF, int DF>
int launch(MoeArgs& a, hipStream_t s) {
  const int64_t experts = a.E < a.T * a.top ? a.E : a.T * a.top;
  const int64_t steps = experts * (((int64_t)a.H * FmtOps<FMT>::ESZ + 127) / 128);
  if constexpr (UF > 1) {
    if (steps >= (int64_t)4 * kMoeWaves * moe_ranges(ceil_div(a.D, 64)))
      return launch_pair<FMT, UF, 4, DF>(a, steps, s);
  }
  return launch_pair<FMT, UF, 2, DF>(a, steps, s);
}

constexpr int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

// Workspace: routing, counters, hidden rows, partial sums.
struct MoePlan {
  int64_t counters, hidden, partials, bytes, ldh;
};
static MoePlan moe_plan(int64_t T, int64_t D, int64_t H, int64_t top) {
  MoePlan p;
  p.ldh = (H + 63) / 64 * 64;
  p.counters = up16(sizeof(RouteOut));
  p.hidden = p.counters + up16((D + 31) / 32 * 4);
  p.partials = p.hidden + up16(T * top * p.ldh * 4);
  const int64_t narrow = (D + 31) / 32, wide = (D + 63) / 64;
  const int64_t a = moe_ranges(narrow) * narrow * 32, b = moe_ranges(wide) * wide * 64;
  p.bytes = p.partials + (a > b ? a : b) * T * 4;
  return p;
}
size_t moe_workspace_bytes(int64_t T, int64_t D, int64_t H, int64_t E, int64_t top) {
  (void)E;
  return (size_t)moe_plan(T, D, H, top).bytes;
}

int launch_moe(MoeArgs& a, void* workspace, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  const MoePlan p = moe_plan(a.T, a.D, a.H, a.top);
  char* ws = (char*)workspace;
  a.route = ws;
  a.counters = (int*)(ws + p.counters);
  a.hidden = ws + p.hidden;
  a.partials = (float*)(ws + p.partials);
  a.ldh = p.ldh;
  const int64_t experts = a.E < a.T * a.top ? a.E : a.T * a.top;
  const int esz = a.w_dt == DT_F32 ? 4 : a.w_dt == DT_BF16 ? 2 : 1;
  const int nk = (int)(((int64_t)a.D * esz + 127) / 128);
  a.slices = 1;
  while (a.slices < kMoeWaves && a.slices < nk) a.slices *= 2;
  const int64_t units = experts * ceil_div(ceil_div(a.H, a.gated ? 16 : 32), kMoeWaves / a.slices);
  a.up_blocks = 1 + (int)(units < 2 * kCus ? units : 2 * kCus);
  // As many token fragments as one expert can need, two at most (then in passes),
  // four in the second kernel for bf16 (64 tokens over 4 experts of 4096 x 2048:
  // 95 us, 102 with two; e4m3 spills with four)
  if (a.w_dt == DT_F32) return a.T > 16 ? launch<FMT_F32, 2, 2>(a, s) : launch<FMT_F32, 1, 1>(a, s);
  if (a.w_dt == DT_BF16)
    return a.T > 16 ? launch<FMT_BF16, 2, 4>(a, s) : a.T > 8 ? launch<FMT_BF16, 1, 2>(a, s) : launch<FMT_BF16, 1, 1>(a, s);
  return a.T > 16 ? launch<FMT_FP8X, 2, 2>(a, s) : a.T > 8 ? launch<FMT_FP8X, 1, 2>(a, s) : launch<FMT_FP8X, 1, 1>(a, s);
}

}  // namespace ox
