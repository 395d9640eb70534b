// gdp_block_common.h -- device helpers shared by the short convolution, the selective
// scan and the norms around a block.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp.h"
#include "gdp_chunks.h"
#include "gdp_launch.h"
#include "gdp_layer_common.h"

namespace gdp {

template <bool B> struct Flag { static constexpr bool value = B; };

__device__ __forceinline__ int uniform_of(int x) { return __builtin_amdgcn_readfirstlane(x); }

// N neighbouring elements at any element's alignment: the memory instructions take
// every alignment, so rows of odd lengths and views that start anywhere are read
// and written in whole pieces too.
template <typename T, int N> struct __attribute__((packed, aligned(sizeof(T)))) Piece { T v[N]; };

// channels ch .. ch + N - 1 of a row of D; those behind its end read as 0 and are not
// written.  STREAMED: past the caches (gdp_layer_common.h).
template <typename T, int N, bool STREAMED = false>
__device__ __forceinline__ Piece<T, N> load_piece(const T *row, int ch, int D) {
  if (ch + N <= D) {
    // (as a vector: copies of the struct itself take the compiler more registers)
    typedef T vec __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    const vec *at = (const vec *)(row + ch);
    const vec v = STREAMED ? __builtin_nontemporal_load(at) : *at;
    Piece<T, N> p;
#pragma unroll
    for (int c = 0; c < N; ++c) p.v[c] = v[c];
    return p;
  }
  Piece<T, N> p;
#pragma unroll
  for (int c = 0; c < N; ++c) p.v[c] = ch + c < D ? row[ch + c] : (T)0.f;
  return p;
}
template <typename T, int N, bool STREAMED = false>
__device__ __forceinline__ void store_piece(T *row, int ch, int D, const Piece<T, N> &p) {
  if (ch + N <= D) {
    typedef T vec __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    vec v;
#pragma unroll
    for (int c = 0; c < N; ++c) v[c] = p.v[c];
    if (STREAMED) __builtin_nontemporal_store(v, (vec *)(row + ch));
    else *(vec *)(row + ch) = v;
    return;
  }
#pragma unroll
  for (int c = 0; c < N; ++c)
    if (ch + c < D) row[ch + c] = p.v[c];
}
template <typename T, int N, bool STREAMED = false>
__device__ __forceinline__ void store_floats(T *row, int ch, int D, const float (&x)[N]) {
  Piece<T, N> p;
#pragma unroll
  for (int c = 0; c < N; ++c) p.v[c] = (T)x[c];
  store_piece<T, N, STREAMED>(row, ch, D, p);
}
// element i of a parameter of type `type` (float32 or T)
template <typename T> __device__ __forceinline__ float param_at(const void *p, int type, int64_t i) {
  return type == EL_F32 ? ((const float *)p)[i] : (float)((const T *)p)[i];
}

__device__ __forceinline__ float act_of(int act, float v) {
  if (act == GDP_ACT_NONE) return v;
  const float s = sigmoid_of(v);
  return act == GDP_ACT_SILU ? v * s : s;
}
// act(v) and act'(v)
__device__ __forceinline__ float act_of(int act, float v, float *slope) {
  if (act == GDP_ACT_NONE) {
    *slope = 1.f;
    return v;
  }
  const float s = sigmoid_of(v);
  if (act == GDP_ACT_SILU) {
    const float f = v * s;
    *slope = fmaf(f, 1.f - s, s);  // s (1 + v (1 - s))
    return f;
  }
  *slope = s * (1.f - s);
  return s;
}

// The chunk of a number (gdp_chunks.h), found by a whole wave (all 64 lanes): false where it
// names none.
__device__ __forceinline__ bool find_chunk(Chunk *k, const void *cu, int is64, int T, int N, int shift, int number) {
  const int lane = threadIdx.x & 63;
  const int seq = uniform_of(sequence_of(N, [&](int lo, int hi, int step) {
    const int i = lo + lane * step;
    return __popcll(__ballot(i < hi && chunk_number((int)bound_at(cu, is64, i, T), i, shift) <= number));
  }));
  if (seq < 0) return false;
  const int first = uniform_of((int)bound_at(cu, is64, seq, T)), last = uniform_of((int)bound_at(cu, is64, seq + 1, T));
  return chunk_of(k, number, shift, seq, first, last);
}

}  // namespace gdp
