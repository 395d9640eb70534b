// gdp_select_common.h -- device helpers of the selective scan's kernels
// (gdp_select.hip, gdp_select_bwd.hip) and the layout of its workspace.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp_block.h"
#include "gdp_block_common.h"

namespace gdp {

// states of a channel as the kernels hold them: zeros behind the last one
inline int padded_states(int64_t S) { return S <= 4 ? 4 : (S <= 8 ? 8 : (S <= 16 ? 16 : 32)); }

// 64 channels of one group per wave
struct SelectGrid {
  int blocks, per_group, shift;  // channel blocks, those of one group, log2 of a chunk's rows
  int64_t numbers;               // of chunks
  int64_t slots;                 // for what one chunk hands to another
};
inline SelectGrid select_grid(int64_t T, int64_t N, int64_t D, int64_t G, int64_t want, int least, int most) {
  SelectGrid g;
  g.per_group = (int)((D / G + 63) / 64);
  g.blocks = (int)(G * g.per_group);
  g.shift = most;
  while (g.shift > least && (T >> g.shift) * g.blocks < want) --g.shift;
  g.numbers = chunk_numbers(T, N, g.shift);
  g.slots = hand_over_slots(T, g.shift);
  return g;
}

inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Chunk numbers, long chunks first, where that many fit: the numbers' order in which the
// waves take them.  Few waves of uneven chunks leave compute units idle at the end otherwise
// (33824 x 4096 in 68 sequences: 549 us, and 806 without); of even ones the order costs its
// launch (4 sequences of 2048 x 2048, forward and gradients: 457 us, and 455 without).
constexpr int64_t MOST_ORDERED = 1024;

// The workspace's first part: the states [slots, padded S, D] and sums of steps [slots, D]
// that chunks hand on, and the chunks' order.  (As numbers, not pointers: the sizes are
// asked for without a workspace.)
struct SelectSpace {
  float *states, *sums;
  int *order;  // [numbers], or null
  size_t bytes;
};
inline SelectSpace select_space(void *ws, int64_t D, int64_t S, const SelectGrid &g) {
  SelectSpace s;
  const uintptr_t p = (uintptr_t)ws;
  size_t at = 0;
  s.states = (float *)p;
  at += round256((size_t)g.slots * padded_states(S) * D * 4);
  s.sums = (float *)(p + at);
  at += round256((size_t)g.slots * D * 4);
  s.order = nullptr;
  if (g.numbers <= MOST_ORDERED) {
    s.order = (int *)(p + at);
    at += round256((size_t)g.numbers * 4);
  }
  s.bytes = at;
  return s;
}

// Row t of a group's B or C, element n
template <typename T> struct Shares {
  const T *p; int64_t st;
};
template <typename T> __device__ __forceinline__ Shares<T> shares_of(const SelectArgs &a, int which, int group) {
  return which ? Shares<T>{(const T *)a.C + group * a.C_sg, a.C_st} : Shares<T>{(const T *)a.B + group * a.B_sg, a.B_st};
}

// M rows of B (WHICH 0), C (1) or both (2), held by a wave until it lays them as floats,
// with zeros behind the last state, into its own LDS, [M, P] or [M, 2, P], where every lane
// reads all of them.  (As scalar loads they miss the scalar cache row by row, 600 cycles
// each, and every wait is one for all of them.)
template <typename T, int M, int P, int WHICH> struct Shared {
  static constexpr int N = WHICH == 2 ? 2 * P : P, EACH = (M * N + 63) / 64, STEP = 64 / N;  // STEP: rows between a lane's
  T v[EACH];
  // rows t, t + dir, ..
  __device__ __forceinline__ void load(const SelectArgs &a, int group, int64_t t, int dir) {
    const int lane = threadIdx.x & 63, n = lane % P;
    const Shares<T> s = shares_of<T>(a, WHICH == 2 ? lane / P & 1 : WHICH, group);
    const bool on = n < a.S && (M * N >= 64 || lane < M * N);
#pragma unroll
    for (int i = 0; i < EACH; ++i) v[i] = on ? s.p[(t + dir * (lane / N + i * STEP)) * s.st + n] : (T)0.f;
  }
  __device__ __forceinline__ void lay(float *lds) const {
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < EACH; ++i)
      if (M * N >= 64 || lane < M * N) lds[lane + i * 64] = (float)v[i];
    // (a wave's LDS accesses are done in their order; this keeps the compiler to it)
    __builtin_amdgcn_wave_barrier();
  }
};

// log(1 + e) for e in [0, 1]: 2 atanh(q), q = e / (2 + e) <= 1/3, as q times a polynomial
// in q^2 of five coefficients, the first exactly 2.  With them as float32 holds them the
// polynomial's largest relative error over [0, 1/9] is 2^-26.9; evaluated in float32,
// log(1 + e) is good to 4 units of 2^-24.
__device__ __forceinline__ float log1p_of(float e) {
  const float q = e * __builtin_amdgcn_rcpf(2.f + e), q2 = q * q;
  float p = 0.2817833524993873f;
  p = fmaf(p, q2, 0.27960602677791624f);
  p = fmaf(p, q2, 0.4002491028745423f);
  p = fmaf(p, q2, 0.6666631468186291f);
  p = fmaf(p, q2, 2.f);
  return q * p;
}
// softplus(v) = max(v, 0) + log(1 + exp(-|v|)).  (The median of three, as max() first
// brings its operand into canonical form.)
__device__ __forceinline__ float softplus_of(float v) {
  return __builtin_amdgcn_fmed3f(v, 0.f, __builtin_inff()) + log1p_of(__builtin_amdgcn_exp2f(-fabsf(v) * LOG2E_L));
}

// a channel's S states in a row of memory, or (null) zeros; zeros behind the last one
template <int P> __device__ __forceinline__ void load_states(float (&x)[P], const float *p, int S) {
  if (p && S == P) {
#pragma unroll
    for (int n = 0; n < P; n += 4) {
      const Piece<float, 4> v = *(const Piece<float, 4> *)(p + n);
#pragma unroll
      for (int c = 0; c < 4; ++c) x[n + c] = v.v[c];
    }
  } else {
#pragma unroll
    for (int n = 0; n < P; ++n) x[n] = p && n < S ? p[n] : 0.f;
  }
}
template <int P> __device__ __forceinline__ void store_states(float *p, const float (&x)[P], int S) {
  if (S == P) {
#pragma unroll
    for (int n = 0; n < P; n += 4) *(Piece<float, 4> *)(p + n) = Piece<float, 4>{{x[n], x[n + 1], x[n + 2], x[n + 3]}};
  } else {
#pragma unroll
    for (int n = 0; n < P; ++n)
      if (n < S) p[n] = x[n];
  }
}
// A[ch] as base-2 exponents; zeros behind the last state
template <int P> __device__ __forceinline__ void load_rates(float (&A2)[P], const SelectArgs &a, int ch) {
  load_states<P>(A2, a.A + (int64_t)ch * a.S, a.S);
#pragma unroll
  for (int n = 0; n < P; ++n) A2[n] *= LOG2E_L;
}

template <typename F> hipError_t select_types(int ut, int dt, F f) {
  if (ut == EL_F32) return f((float)0, (float)0);
  if (ut == EL_BF16) return dt == EL_F32 ? f((bf16)0, (float)0) : f((bf16)0, (bf16)0);
  return dt == EL_F32 ? f((_Float16)0, (float)0) : f((_Float16)0, (_Float16)0);
}
template <int P> struct States { static constexpr int value = P; };
template <typename F> hipError_t by_states(int64_t S, F f) {
  switch (padded_states(S)) {
    case 4: return f(States<4>());
    case 8: return f(States<8>());
    case 16: return f(States<16>());
    default: return f(States<32>());
  }
}

// The forward pass's chunks: short enough for 4096 waves; but where the sequences are as
// many as fill the chip by themselves, as long as twice their mean length, so that most
// are one chunk and take part in neither of the first two kernels (33824 x 4096 in 68
// sequences: 549 us, and 768 without that).
inline SelectGrid forward_grid(int64_t T, int64_t N, int64_t D, int64_t G) {
  SelectGrid g = select_grid(T, N, D, G, 4096, 4, 11);
  if (N * g.blocks >= 2048)
    while (g.shift < 11 && ((int64_t)1 << g.shift) * N < 2 * T) ++g.shift;
  g.numbers = chunk_numbers(T, N, g.shift);
  g.slots = hand_over_slots(T, g.shift);
  return g;
}
// ... and those of the gradients: enough for 2048 workgroups
inline SelectGrid backward_grid(int64_t T, int64_t N, int64_t D, int64_t G) {
  return select_grid(T, N, D, G, 2048, 6, 11);
}
}  // namespace gdp
