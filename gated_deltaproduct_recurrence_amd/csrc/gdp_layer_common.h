// gdp_layer_common.h -- device helpers shared by the layers' kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp_chunks.h"

namespace gdp {

typedef __bf16 bf16;

__device__ __forceinline__ int64_t index_at(const void *p, int is64, int64_t i) {
  return is64 ? ((const int64_t *)p)[i] : (int64_t)((const int32_t *)p)[i];
}

// cu_seqlens[i] clamped to [0, T]
__device__ __forceinline__ int64_t bound_at(const void *cu, int is64, int64_t i, int64_t T) {
  return clamp_bound(index_at(cu, is64, i), T);
}

// N neighbouring elements
template <typename T, int N> struct alignas(sizeof(T) * N) Pack { T v[N]; };

// Loads and stores of a stream that is larger than the memory-side cache (256 MB):
// nothing of it can stay there for a later reader, and marked so it does not push
// out what can.  Smaller ones are left to the caches: a product that reads the
// norm's 33 MB output took 2 to 3 us longer after marked stores.
constexpr int64_t STREAM_BYTES = (int64_t)256 << 20;
template <typename T, int N> __device__ __forceinline__ Pack<T, N> load_streamed(const T *p) {
  typedef T vec __attribute__((ext_vector_type(N)));
  const vec v = __builtin_nontemporal_load((const vec *)p);
  return *(const Pack<T, N> *)&v;
}
template <typename T, int N> __device__ __forceinline__ void store_streamed(T *p, const Pack<T, N> &s) {
  typedef T vec __attribute__((ext_vector_type(N)));
  __builtin_nontemporal_store(*(const vec *)&s, (vec *)p);
}

constexpr float LOG2E_L = 1.4426950408889634f;

// exp(g) by the hardware's base-2 exponential (1 ulp; its result below 2^-126 is
// 0, that of -inf is 0).  The product's rounding adds |g| 2^-24 relative, which
// is below an ulp of the result's effect on a state while |g| < 1 and concerns
// decays below 0.4 otherwise.
__device__ __forceinline__ float decay(float g) { return __builtin_amdgcn_exp2f(g * LOG2E_L); }

// s = sigmoid(v): the hardware's exponential and reciprocal, each good to one step;
// the product before them is rounded, which adds |v| 2^-24 relative to exp(-v).  The
// reciprocal of an infinite sum is 0.
__device__ __forceinline__ float sigmoid_of(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -LOG2E_L));
}

// 1 - exp(g): the Taylor polynomial of degree 8 for |g| < 1/2 (its first omitted
// term is g^9 / 9!, below 2^-26 of the result there), else the difference, whose
// rounding is 2^-25 of a value above 0.39.  `a` is decay(g).
__device__ __forceinline__ float one_minus_decay(float g, float a) {
  float p = 1.f / 40320.f;
  p = fmaf(p, g, 1.f / 5040.f);
  p = fmaf(p, g, 1.f / 720.f);
  p = fmaf(p, g, 1.f / 120.f);
  p = fmaf(p, g, 1.f / 24.f);
  p = fmaf(p, g, 1.f / 6.f);
  p = fmaf(p, g, 0.5f);
  p = fmaf(p, g * g, g);
  return fabsf(g) < 0.5f ? -p : 1.f - a;
}

// Sum over the lanes of an aligned team of LPG <= 64 lanes, in every lane: DPP
// moves within 16 lanes, then the row swaps.
template <int CTRL> __device__ __forceinline__ float dpp_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float team_sum(float x, int lpg) {
  if (lpg > 1) x = dpp_add<0xb1>(x);   // quad_perm 1,0,3,2
  if (lpg > 2) x = dpp_add<0x4e>(x);   // quad_perm 2,3,0,1
  if (lpg > 4) x = dpp_add<0x141>(x);  // row_half_mirror
  if (lpg > 8) x = dpp_add<0x140>(x);  // row_mirror
  if (lpg > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (lpg > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

// ... of a team of whole waves (LPG > 64): the waves' sums through LDS.  `turn`
// alternates the slots, so one barrier per sum is enough.
template <int WIDE> struct Team {
  int lpg, lane, first_wave;  // lanes per team, lane within it, its first wave in the workgroup
  float (*slots)[16];         // [2][16]
  int turn = 0;
  __device__ float sum(float x) {
    x = team_sum(x, WIDE ? 64 : lpg);
    if constexpr (WIDE) {
      if ((lane & 63) == 0) slots[turn][first_wave + (lane >> 6)] = x;
      __syncthreads();
      x = 0.f;
      for (int v = 0; v < lpg >> 6; ++v) x += slots[turn][first_wave + v];
      turn ^= 1;
    }
    return x;
  }
};

}  // namespace gdp
