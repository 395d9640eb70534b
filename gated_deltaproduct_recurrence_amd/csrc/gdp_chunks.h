// gdp_chunks.h -- how sequences are cut into chunks, and where what belongs to a chunk lies:
// the numbers alone, for kernels and for the host.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdp {

// a boundary from cu_seqlens, clamped to [0, T]
__host__ __device__ inline int64_t clamp_bound(int64_t v, int64_t T) { return v < 0 ? 0 : (v > T ? T : v); }

// A piece of one sequence: rows [begin, end) of sequence `seq`, whose rows are
// [first, last).  Sequences are cut into chunks of 2^shift rows from their first
// row on, so no chunk holds rows of two sequences.  Chunk c of sequence i has number
//     (cu[i] >> shift) + i + c:
// sequence i + 1 starts at least that many numbers later as sequence i has chunks, so
// numbers are unique, rise with the rows, and lie below (T >> shift) + N; some name
// no chunk.  An empty sequence has one chunk, without rows.
struct Chunk {
  int begin, end, first, last, seq, index;
};
__host__ __device__ inline int64_t chunk_numbers(int64_t T, int64_t N, int shift) { return (T >> shift) + N; }
// of chunk 0 of a sequence
__host__ __device__ inline int chunk_number(int first, int seq, int shift) { return (first >> shift) + seq; }

// The last sequence whose numbers begin at or before a number, or -1: in steps of 64,
// count(lo, hi, step) being the number of sequences lo, lo + step, .. of 64 and below hi
// of which that holds.
template <typename Count> __host__ __device__ __forceinline__ int sequence_of(int N, Count count) {
  int lo = 0, hi = N, step;
  do {
    step = (hi - lo + 63) >> 6;
    const int c = count(lo, hi, step);
    if (c == 0) return -1;
    lo += (c - 1) * step;
    hi = hi < lo + step ? hi : lo + step;
  } while (step > 1);
  return lo;
}
// The chunk of a number that belongs to sequence `seq` of rows [first, last): false where it
// names none.  Boundaries that do not rise give chunks that overlap or leave out rows, all
// within [0, T) and [0, N).
__host__ __device__ __forceinline__ bool chunk_of(Chunk *k, int number, int shift, int seq, int first, int last) {
  k->seq = seq;
  k->first = first;
  k->last = first > last ? first : last;
  k->index = number - chunk_number(first, seq, shift);
  const int64_t rows = (int64_t)1 << shift, begin = k->first + k->index * rows, end = begin + rows;
  if (k->index < 0 || (k->index > 0 && begin >= k->last)) return false;
  k->begin = (int)begin;
  k->end = (int)(end < k->last ? end : k->last);
  return true;
}

// What chunks hand on stands in the place first row >> shift of the chunk before the boundary: such
// a chunk is full and at least a row behind it lies in [0, T), so its place is its own and
// below (T - 1) >> shift, however many sequences there are.
__host__ __device__ inline int64_t hand_over_slots(int64_t T, int shift) { return T > 0 ? (T - 1) >> shift : 0; }
__host__ __device__ inline int64_t slot_behind(const Chunk &k, int shift) { return k.begin >> shift; }
__host__ __device__ inline int64_t slot_before(const Chunk &k, int shift) { return (k.begin >> shift) - 1; }
// Chunks of a sequence that another follows; their places are neighbours from first >> shift on.
__host__ __device__ inline int64_t followed_chunks(int64_t rows, int shift) {
  return ((rows + ((int64_t)1 << shift) - 1) >> shift) - 1;
}

// The checkpoint before row t, the first of 2^shift, of sequence `seq`: of the rows of
// [chunk_numbers(T, N, shift), ..].
__host__ __device__ inline int64_t checkpoint_row(int first, int seq, int t, int shift) {
  return chunk_number(first, seq, shift) + ((t - first) >> shift);
}

}  // namespace gdp
