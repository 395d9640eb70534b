// The cutting of sequences into chunks (csrc/gdp_chunks.h) on the host, for tests/test_chunks_cpu.py.
#include "gdp_chunks.h"

using namespace gdp;

namespace {
// find_chunk of a wave, its 64 lanes one after another
bool find(Chunk *k, const int64_t *cu, int T, int N, int shift, int number) {
  const int seq = sequence_of(N, [&](int lo, int hi, int step) {
    int count = 0;
    for (int lane = 0; lane < 64; ++lane) {
      const int i = lo + lane * step;
      count += i < hi && chunk_number((int)clamp_bound(cu[i], T), i, shift) <= number;
    }
    return count;
  });
  if (seq < 0) return false;
  return chunk_of(k, number, shift, seq, (int)clamp_bound(cu[seq], T), (int)clamp_bound(cu[seq + 1], T));
}
}  // namespace

extern "C" {

int64_t numbers(int64_t T, int64_t N, int shift) { return chunk_numbers(T, N, shift); }
int64_t slots(int64_t T, int shift) { return hand_over_slots(T, shift); }
int64_t followed(int64_t rows, int shift) { return followed_chunks(rows, shift); }
int64_t checkpoint(int first, int seq, int t, int shift) { return checkpoint_row(first, seq, t, shift); }

// the chunks of all numbers: [begin, end, first, last, seq, index, slot behind, slot before], or begin = -1
void chunks(const int64_t *cu, int T, int N, int shift, int64_t (*out)[8]) {
  for (int64_t number = 0; number < chunk_numbers(T, N, shift); ++number) {
    Chunk k;
    int64_t *o = out[number];
    o[0] = -1;
    if (!find(&k, cu, T, N, shift, (int)number)) continue;
    const int64_t row[8] = {k.begin, k.end, k.first, k.last, k.seq, k.index, slot_behind(k, shift), slot_before(k, shift)};
    for (int i = 0; i < 8; ++i) o[i] = row[i];
  }
}
}
