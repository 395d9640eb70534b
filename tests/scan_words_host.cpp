// The recurrence's words (csrc/gdp_scan_words.h) on the host, for tests/test_scan_words_cpu.py.
#include "gdp_scan_words.h"

using namespace gdp;

extern "C" {

uint64_t tile_word(float A, float B) { return make_word(A, B); }

// the word of the tiles' words w[count - 1] .. w[0]
uint64_t group_word(const uint64_t *w, int count) {
  Span s = no_rows();
  for (int i = count - 1; i >= 0; --i) s = then(s, part_a(w[i]), part_b(w[i]));
  return make_word(normal(s));
}

uint64_t span_word(const uint64_t (&v)[15]) { return make_word(span_over(v)); }
float span_applied(const uint64_t (&v)[15], float h) { return apply(span_over(v), h); }
float group_word_applied(uint64_t word, float h) { return apply(span_of(word), h); }
int drops(uint64_t word) { return drops_all(word); }
float fold_tiles(const uint64_t (&v)[8]) { return fold<false>(v); }
float fold_groups(const uint64_t (&v)[8]) { return fold<true>(v); }
}
