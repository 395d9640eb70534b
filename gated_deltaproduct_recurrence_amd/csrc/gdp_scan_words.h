// gdp_scan_words.h -- what the workgroups of the recurrence (gdp_scan.hip) hand on:
// the affine map h -> A h + B of a run of rows in an 8-byte word, and how the words
// before a tile give the state that enters it.  Functions of values only; nothing
// here reads or writes memory of the device.
//
// A tile's word holds A and B in float32.  A group's word covers up to 2048 rows,
// whose decays can multiply to far less, or (positive log decays) far more, than a
// float32 although every state on the way is one.  Its A is kept as m 2^e with m in
// [1/2, 1): 23 bits of m and 9 of e, which leaves 2^-255 .. 2^255.
// A = 0 says that nothing before matters; all-ones bits mean not yet written.  Read as
// a pair those are (not 0, NaN): a word that is missing where a state is formed
// makes it NaN, unless a nearer word drops what was before.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdp {

constexpr uint64_t NOT_WRITTEN = ~0ull;
constexpr uint32_t QUIET_NAN = 0x7fc00000u;  // a NaN that is not NOT_WRITTEN's

__host__ __device__ __forceinline__ uint32_t bits_of(float x) { return __builtin_bit_cast(uint32_t, x); }
__host__ __device__ __forceinline__ float float_of(uint32_t x) { return __builtin_bit_cast(float, x); }

__host__ __device__ __forceinline__ float part_a(uint64_t word) { return float_of((uint32_t)(word >> 32)); }
__host__ __device__ __forceinline__ float part_b(uint64_t word) { return float_of((uint32_t)word); }

// the map (A, B) applied to h; A = 0 drops h, also one that is not finite
__host__ __device__ __forceinline__ float apply(float A, float h, float B) {
  return A == 0.f ? B : __builtin_fmaf(A, h, B);
}

__host__ __device__ __forceinline__ uint64_t make_word(float A, float B) {
  return ((uint64_t)(A != A ? QUIET_NAN : bits_of(A)) << 32) | bits_of(B);
}

// The map h -> m 2^e h + B of neighbouring tiles; m = 0 where h does not matter, else
// in [1/2, 1) once it is `normal`.  The product of a group's 16 mantissas stays above
// 2^-17, so the sum over tiles is one product, one sum and one fma a tile.
struct Span { float m; int e; float B; };

__host__ __device__ __forceinline__ Span no_rows() { return Span{1.f, 0, 0.f}; }

// s, then the map (A, B)
__host__ __device__ __forceinline__ Span then(Span s, float A, float B) {
  int e = 0;
  const float m = __builtin_frexpf(A, &e);
  return Span{A == 0.f ? 0.f : s.m * m, s.e + e, apply(A, s.B, B)};
}
__host__ __device__ __forceinline__ Span normal(Span s) {
  int e = 0;
  const float m = __builtin_frexpf(s.m, &e);
  return Span{m, s.e + e, s.B};
}

// m 2^e h is rounded once, with B, as apply does: 2^(e-1) h is exact above 2^-126, and
// no larger than the product with 2 m
__host__ __device__ __forceinline__ float apply(Span s, float h) {
  return s.m == 0.f ? s.B : __builtin_fmaf(s.m + s.m, __builtin_ldexpf(h, s.e - 1), s.B);
}

// A group's word.  A state of less than 2^128 that A < 2^-126 leaves below half a
// step of B is dropped here, by values alone: then the groups behind do not wait for
// it.  (So is what would be below 2^-126, past the exponents' end; past the other
// end the largest A is kept: it takes 0 to 0 and the rest to infinity.)
__host__ __device__ __forceinline__ uint64_t make_word(Span s) {
  const bool number = __builtin_fabsf(s.m) < 1.f;
  const bool gone = s.e < -254 || (s.e <= -126 && __builtin_ldexpf(s.m, s.e + 153) <= __builtin_fabsf(s.B));
  const uint32_t a = s.e > 255 ? 0xff7fffffu : ((uint32_t)(s.e + 255) << 23) | (bits_of(s.m) & 0x7fffffu);
  return ((uint64_t)(!number || s.m == 0.f || gone ? 0u : a) << 32) | (number ? bits_of(s.B) : QUIET_NAN);
}
__host__ __device__ __forceinline__ Span span_of(uint64_t word) {
  const uint32_t a = (uint32_t)(word >> 32);
  return Span{a == 0 ? 0.f : float_of((a & 0x7fffffu) | 0x3f000000u), (int)(a >> 23) - 255, part_b(word)};
}

__host__ __device__ __forceinline__ bool drops_all(uint64_t word) { return (uint32_t)(word >> 32) == 0; }

// The state behind the words v[N - 1] .. v[0]: known if one of them drops what was
// before and all nearer ones are written, else NaN.
template <bool GROUP_WORDS, int N> __host__ __device__ __forceinline__ float fold(const uint64_t (&v)[N]) {
  float h = float_of(QUIET_NAN);
#pragma unroll
  for (int i = N - 1; i >= 0; --i)
    h = GROUP_WORDS ? apply(span_of(v[i]), h) : apply(part_a(v[i]), h, part_b(v[i]));
  return h;
}

// The map of the tiles of the words v[N - 1] .. v[0].  NOTHING is the word of no rows.
constexpr uint64_t NOTHING = 0x3f800000ull << 32;
template <int N> __host__ __device__ __forceinline__ Span span_over(const uint64_t (&v)[N]) {
  Span s = no_rows();
#pragma unroll
  for (int i = N - 1; i >= 0; --i) s = then(s, part_a(v[i]), part_b(v[i]));
  return normal(s);
}

}  // namespace gdp
