// gdp_layer_common.h -- device helpers shared by the recurrence (gdp_scan.hip)
// and the norm (gdp_norm.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdp {

typedef __bf16 bf16;

__device__ __forceinline__ int64_t index_at(const void *p, int is64, int64_t i) {
  return is64 ? ((const int64_t *)p)[i] : (int64_t)((const int32_t *)p)[i];
}

// cu_seqlens[i] clamped to [0, T]
__device__ __forceinline__ int64_t bound_at(const void *cu, int is64, int64_t i, int64_t T) {
  const int64_t v = index_at(cu, is64, i);
  return v < 0 ? 0 : (v > T ? T : v);
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

}  // namespace gdp
