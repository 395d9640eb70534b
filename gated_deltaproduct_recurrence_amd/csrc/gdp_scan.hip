// gdp_scan.hip -- gfx950 kernels of the gated linear recurrence
//     h_t = a_t h_{t-1} + u_t,  a_t = exp(g_t),  u_t = x_t or (1 - a_t) x_t
// per channel over packed sequences, of its gradients, and of its single-token
// step.
//
// The recurrence is a composition of affine maps h -> A h + B, so a block of rows
// can be reduced to one pair (A, B) per channel before the state that enters it is
// known.  The token stream (all sequences end to end) is cut into tiles of 8 R rows;
// a workgroup of 8 waves takes one tile of one channel block, wave w rows R w ..
// R w + R - 1, a lane VEC neighbouring channels.  Every input is loaded once into
// registers and every output written once:
//   1. the rows' decays and terms, and their maps composed: per wave, then (through
//      LDS) per tile;
//   2. the tile's pair is published in an 8-byte word per channel, and the state
//      entering the tile is formed from the words of the tiles before it (below);
//   3. the rows again from the entering state, out of registers, to the outputs.
// A sequence that starts inside a tile cuts the chain there: its first row takes
// initial_state in place of the state before it, and the map's A is 0.
//
// Handing on the states.  A word holds (A, B) of one tile; a tile that knows its
// entering state h, or needs none, holds (0, A h + B) instead: A = 0 says that
// nothing before the tile matters.  A lane reads the words of the WINDOW tiles
// before its own until it has found one with A = 0 and all those between, and
// composes them from that one forward.  That is the sequential fold, whichever tile
// the fold starts from, so the result does not depend on timing.  While none has
// A = 0 only the farthest is read again: the known states reach it first.
// With few channel blocks (GROUPS) the known states come that way through groups of
// 16 tiles instead, each with a word of its own: a tile reads the pairs of the tiles
// before it in its group, other lanes the state entering the group, and the group's
// last tile publishes the group's pair and then its state.  There the tiles' words
// are pairs only, so that the order of the sums is fixed here too.  A group's pair
// keeps its A with an exponent of its own (gdp_scan_words.h): 2048 rows of decays
// leave float32 in both directions while the states between them do not.
// The words are written and read with relaxed agent-scope atomics (8 bytes, so a
// pair is whole), which go past the XCDs' own caches; all-ones bits (two NaNs that
// no published pair has) mean not yet written, and a fill kernel sets them before.
// Tiles are handed out by an atomic counter, rows ascending, so a workgroup waits
// only for tiles whose workgroups are running, and those publish their pairs before
// they wait themselves; with all pairs there, a group's pair waits for nothing else,
// and the first of the waiting tiles (or groups) finds its predecessor's word at
// A = 0: every wait ends.  (It is bounded all the same, at 2^21 looks, seconds:
// when calls on two streams share a workspace against the contract, tickets can be
// lost.  The lost tiles' rows are then left as they are, and the sequences' rows behind
// become NaN, instead of the GPU hanging.)
//
// What bounds it, measured on MI355X (a 1 GiB copy reaches 5.0 TB/s).  32768 x 2048
// bfloat16 with float32 gates: 112 us, 4.8 TB/s of the operands' bytes; 131104 x 4096
// of bfloat16 in 68 sequences, complement form: 704 us, 4.6 TB/s; forward and gradients
// of 8 x 4096 x 2048: 122 + 205 us, 4.4 and 4.6 TB/s.  The words add 7% to the bytes
// read and 6% to those written.  Of a workgroup's 11.5 us on the second shape, 4 us are
// its loads, 3 us the decays and maps (the vector units are issuing 60% of the time),
// 2.5 us the hand-over and 0.7 us the stores; two workgroups per CU overlap them.
//   Tile: 128 rows x 128 channels (16 rows and a pair of channels per lane).  With 64
// rows the second shape took 1045 us instead of 743 (twice the words, twice the hops);
// 4 channels per lane and 8 rows 838; one channel per lane 1012.
//   Window: 8 tiles; 16 cost 3% (registers, words read), 4 gained 1% on the wide shapes
// and cost 25% at 1024 channels.
//   Three workgroups per CU (80 registers) spill: 1650 us.  Workgroups that stay and
// draw their next ticket ahead: 853 us.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp_layer.h"
#include "gdp_layer_common.h"
#include "gdp_scan_words.h"

namespace gdp {
namespace {

constexpr int WAVES = 8, THREADS = 64 * WAVES;
constexpr int VEC = 2, NCH = 64 * VEC;  // channels per lane and per workgroup
constexpr int GROUP = 16;               // tiles per group
constexpr int WINDOW = 8;               // words before its own that a lane looks at
constexpr int MOST_LOOKS = 1 << 21;

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Channels ch, ch + 1 of a row: the row's address is the same for a whole wave
// (scalar registers), the lane's part a 32-bit byte offset.  The pair need not be
// aligned: rows of an odd number of channels, or of a view that starts anywhere,
// are read and written in pairs all the same, but for the last block of an odd D
// (`tail`), which goes channel by channel.
template <typename T> struct __attribute__((packed, aligned(sizeof(T)))) Pair { T v[VEC]; };
template <typename T> __device__ __forceinline__ T *at(T *row, uint32_t ch) {
  return (T *)((char *)row + (uint32_t)(ch * sizeof(T)));
}
template <typename T> __device__ __forceinline__ const T *at(const T *row, uint32_t ch) {
  return (const T *)((const char *)row + (uint32_t)(ch * sizeof(T)));
}
template <typename T> __device__ __forceinline__ Pair<T> load_pair(const T *row, uint32_t ch) {
  return *(const Pair<T> *)at(row, ch);
}
template <typename T> __device__ __forceinline__ Pair<T> load_streamed(const T *row, uint32_t ch) {
  typedef T vec __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
  const vec v = __builtin_nontemporal_load((const vec *)at(row, ch));
  return Pair<T>{{v.x, v.y}};
}
template <typename T> __device__ __forceinline__ void store_pair(T *row, uint32_t ch, const float (&x)[VEC]) {
  *(Pair<T> *)at(row, ch) = Pair<T>{{(T)x[0], (T)x[1]}};
}
struct Tail { bool on; uint32_t last; };  // last: the tensor's last channel
template <typename T> __device__ __forceinline__ Pair<T> load_pair(const T *row, uint32_t ch, Tail tail) {
  if (!tail.on) return load_pair(row, ch);
  return Pair<T>{{*at(row, ch), *at(row, ch < tail.last ? ch + 1 : ch)}};
}
template <typename T>
__device__ __forceinline__ void store_pair(T *row, uint32_t ch, const float (&x)[VEC], Tail tail) {
  if (!tail.on) return store_pair(row, ch, x);
  *at(row, ch) = (T)x[0];
  if (ch < tail.last) *at(row, ch + 1) = (T)x[1];
}

// R rows from t0 on; rows behind the last one read that row again
template <int R, typename T>
__device__ __forceinline__ void load_rows(Pair<T> (&v)[R], const T *base, int64_t stride, int64_t t0, int64_t rows,
                                          uint32_t ch, Tail tail, int streamed) {
  const T *row = base + t0 * stride;
  if (t0 + R > rows || tail.on) {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = load_pair(base + (t0 + r < rows ? t0 + r : rows - 1) * stride, ch, tail);
  } else if (streamed) {
#pragma unroll
    for (int r = 0; r < R; ++r, row += stride) v[r] = load_streamed(row, ch);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r, row += stride) v[r] = load_pair(row, ch);
  }
}

template <int R> struct Shared {
  static constexpr int ROWS = WAVES * R;
  float A[WAVES][NCH], B[WAVES][NCH];
  float state[NCH];                  // the state entering the tile's group ...
  int there[VEC];                    // ... and whether it is there, of each half of the channels
  int start_id[ROWS], end_id[ROWS];  // sequence that starts / ends at a row of the tile, or -1
  int ticket;
};

// Marks the tile's rows where sequences start and end (nonempty ones), in LDS.
// Boundaries are read 512 at a time; with more sequences, the one that holds the
// first row r0 is found first in 512-way steps.  Bad contents give wrong marks,
// with ids in [0, N).
template <typename S> __device__ __forceinline__ void mark_rows(S &sh, const ScanArgs &a, int64_t r0, int tid) {
  int64_t lo = 0, hi = a.N;
  while (hi - lo > THREADS) {  // the last sequence that starts at or before r0
    const int64_t step = (hi - lo + THREADS - 1) / THREADS, i = lo + tid * step;
    const int c = __syncthreads_count(i < hi && bound_at(a.cu, a.cu_is64, i, a.T) <= r0);
    if (c == 0) {
      hi = lo + 1;
    } else {
      lo += (c - 1) * step;
      hi = hi < lo + step ? hi : lo + step;
    }
  }
  for (int64_t base = lo; base < a.N; base += THREADS) {
    const int64_t i = base + tid;
    bool past = true;
    if (i < a.N) {
      const int64_t s = bound_at(a.cu, a.cu_is64, i, a.T) - r0, e = bound_at(a.cu, a.cu_is64, i + 1, a.T) - r0 - 1;
      if (e >= s) {
        if (s >= 0 && s < S::ROWS) sh.start_id[s] = (int)i;
        if (e >= 0 && e < S::ROWS) sh.end_id[e] = (int)i;
      }
      past = s >= S::ROWS;
    }
    if (__syncthreads_or(past)) break;
  }
}
// a wave's rows that are marked, as a mask
template <int R> __device__ __forceinline__ uint32_t marked(const int *ids, int w, int lane) {
  return (uint32_t)__ballot(lane < R && ids[w * R + (lane & (R - 1))] >= 0);
}

__device__ __forceinline__ uint64_t read_word(const uint64_t *w) {
  return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void write_word(uint64_t *w, uint64_t word) {
  __hip_atomic_store(w, word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that the `count` words before hand on, of one channel: `word` is the
// nearest one, the others lie `step` words apart.  NaN where the wait is given up.
template <bool GROUP_WORDS>
__device__ __forceinline__ float entering(const uint64_t *word, int64_t step, int count, bool live) {
  uint64_t v[WINDOW];
  auto read = [&](const uint64_t *w, int i) {  // before the first there is a state of 0
    return live && i < count ? read_word(w + i * step) : 0;
  };
  bool found;  // a word with A = 0 and all before it are there
  auto look = [&](int n) {
    bool open = true;
    found = false;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool there = v[i] != NOT_WRITTEN;
      found = found || (open && there && drops_all(v[i]));
      open = open && there && !found;
    }
  };
  // the nearer half first: mostly it is enough
  constexpr int NEAR = WINDOW / 2;
#pragma unroll
  for (int i = 0; i < WINDOW; ++i) v[i] = i < NEAR ? read(word, i) : NOT_WRITTEN;
  look(NEAR);
  if (!__all(found)) {
#pragma unroll
    for (int i = NEAR; i < WINDOW; ++i) v[i] = read(word, i);
    for (int looks = 0;; ++looks) {
      look(WINDOW);
      if (__all(found) || looks == MOST_LOOKS) break;
      __builtin_amdgcn_s_sleep(1);
      asm volatile("" : "+v"(word));  // or every word's address is kept in registers over the loop
#pragma unroll
      for (int i = 0; i < WINDOW; ++i)
        if (i == WINDOW - 1 || v[i] == NOT_WRITTEN) v[i] = read(word, i);
    }
  }
  return fold<GROUP_WORDS>(v);
}

// The map of the `count` tiles before this one in its group, of one channel; its B is
// NaN where the wait is given up.
__device__ __forceinline__ Span group_so_far(const uint64_t *word, int64_t step, int count, bool live) {
  uint64_t v[GROUP - 1];
#pragma unroll
  for (int i = 0; i < GROUP - 1; ++i) v[i] = i < count ? NOT_WRITTEN : NOTHING;
  for (int looks = 0;; ++looks) {
#pragma unroll
    for (int i = 0; i < GROUP - 1; ++i)
      if (v[i] == NOT_WRITTEN) v[i] = live ? read_word(word + i * step) : 0;
    bool open = true, there = true;  // all that matter: up to the nearest with A = 0
#pragma unroll
    for (int i = 0; i < GROUP - 1; ++i) {
      there = there && (!open || v[i] != NOT_WRITTEN);
      open = open && !(v[i] != NOT_WRITTEN && drops_all(v[i]));
    }
    if (__all(there) || looks == MOST_LOOKS) break;
    __builtin_amdgcn_s_sleep(1);
    asm volatile("" : "+v"(word));
  }
  return span_over(v);
}

// The waves' maps in sh.A, sh.B: composes the tile's, publishes it, and leaves in
// sh.A the state entering each wave's rows (of the channels first + 0 .. NCH - 1).
// REVERSE: from the last tile and wave to the first.
template <bool GROUPS, bool REVERSE, typename S>
__device__ __forceinline__ void hand_over(S &sh, const ScanArgs &a, int tile, int tiles, bool needs, int first, int tid) {
  const int c = tid % NCH, role = tid / NCH;
  if (role > (GROUPS ? 1 : 0)) return;
  const int64_t step = REVERSE ? a.D : -a.D;  // to the tile before, in this direction
  const int before = REVERSE ? tiles - 1 - tile : tile;
  const int group = before / GROUP, place = before % GROUP;
  const bool live = first + c < a.D;
  uint64_t *words = (uint64_t *)((char *)a.ws + 256);
  uint64_t *mine = at(words + (int64_t)tile * a.D, first + c);
  uint64_t *groups = at(words + ((int64_t)tiles + group) * a.D, first + c);
  if (GROUPS && role == 1) {  // the state entering the group
    if (needs && tiles > 1) {
      sh.state[c] = entering<true>(groups - a.D, -a.D, group, live);
      __hip_atomic_store(&sh.there[c >> 6], 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    return;
  }
  float carry = 0.f;
  if (tiles > 1) {
    float A = 1.f, B = 0.f;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) {
      const int w = REVERSE ? WAVES - 1 - v : v;
      B = apply(sh.A[w][c], B, sh.B[w][c]);
      A = sh.A[w][c] == 0.f ? 0.f : A * sh.A[w][c];  // also where A is not finite: another sequence's decays
    }
    if (!needs) A = 0.f;
    if (live && before + 1 < tiles) write_word(mine, make_word(A, B));
    if (!GROUPS) {
      if (needs) {
        carry = entering<false>(mine + step, step, before, live);
        if (live && before + 1 < tiles && A != 0.f) write_word(mine, make_word(0.f, fmaf(A, carry, B)));
      }
    } else {
      const bool last = place == GROUP - 1 && before + 1 < tiles && live;
      Span sofar{0.f, 0, 0.f};
      if (needs) sofar = group_so_far(mine + step, step, place, live);
      const Span group_map = normal(then(sofar, A, B));
      const uint64_t word = make_word(group_map);
      if (last) write_word(groups, word);
      if (needs) {
        while (!__hip_atomic_load(&sh.there[c >> 6], __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP))
          __builtin_amdgcn_s_sleep(1);
        const float state = sh.state[c];
        carry = apply(sofar, state);
        if (last && !drops_all(word)) write_word(groups, make_word(0.f, apply(group_map, state)));
      }
    }
  }
  float h = carry;
#pragma unroll
  for (int v = 0; v < WAVES; ++v) {
    const int w = REVERSE ? WAVES - 1 - v : v;
    const float next = apply(sh.A[w][c], h, sh.B[w][c]);
    sh.A[w][c] = h;
    h = next;
  }
}

// The workgroup's job: its ticket (the counter starts at -1), or the block's own
// index when nothing is handed on.  Clears the row marks.
template <typename S> __device__ __forceinline__ int take_ticket(S &sh, const ScanArgs &a, bool hand_on, int tid) {
  if (tid < S::ROWS) sh.start_id[tid] = sh.end_id[tid] = -1;
  if (tid < VEC) sh.there[tid] = 0;
  if (!hand_on) {
    __syncthreads();
    return (int)blockIdx.x;
  }
  if (tid == 0) sh.ticket = atomicAdd((int *)a.ws, 1) + 1;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(sh.ticket);
}

// The jobs behind the tiles: 64 sequences each, whose empty ones hand src (or
// zeros) to dst (and to the state cache).
__device__ __forceinline__ void empty_sequences(const ScanArgs &a, int64_t job, const float *src, float *dst, int tid) {
  for (int64_t i = job * 64; i < (job + 1) * 64 && i < a.N; ++i) {
    if (bound_at(a.cu, a.cu_is64, i + 1, a.T) > bound_at(a.cu, a.cu_is64, i, a.T)) continue;
    int64_t slot = -1;
    if (a.cache) {
      slot = index_at(a.slots, a.slots_is64, i);
      if (slot >= a.num_slots) slot = -1;
    }
    for (int64_t ch = tid; ch < a.D; ch += THREADS) {
      const float h = src ? src[i * a.D + ch] : 0.f;
      if (dst) dst[i * a.D + ch] = h;
      if (slot >= 0) a.cache[slot * a.D + ch] = h;
    }
  }
}

template <typename XT, typename GT, int R, bool COMPL, bool GROUPS>
__global__ void __launch_bounds__(THREADS, 4) gdp_scan_kernel(ScanArgs a, int tiles, int blocks) {
  using S = Shared<R>;
  __shared__ S sh;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool hand_on = tiles > 1;
  const int ticket = take_ticket(sh, a, hand_on, tid);
  const int tile = ticket / blocks;
  if (tile >= tiles) {
    empty_sequences(a, ticket - tiles * blocks, a.s0, a.final_state, tid);
    return;
  }
  const int first = (ticket % blocks) * NCH;  // the block's first channel
  const int64_t r0 = (int64_t)tile * S::ROWS;
  const bool mine = first + lane * VEC < a.D;
  const uint32_t ch = mine ? first + lane * VEC : 0;
  const Tail tail{first + NCH > a.D && (a.D & 1), (uint32_t)a.D - 1};
  const int64_t t0 = r0 + w * R;

  Pair<GT> graw[R];
  Pair<XT> xraw[R];
  load_rows<R>(graw, (const GT *)a.g, a.g_st, t0, a.T, ch, tail, a.streamed);
  load_rows<R>(xraw, (const XT *)a.x, a.x_st, t0, a.T, ch, tail, a.streamed);
  const int64_t c0 = bound_at(a.cu, a.cu_is64, 0, a.T), cN = bound_at(a.cu, a.cu_is64, a.N, a.T);
  mark_rows(sh, a, r0, tid);
  const uint32_t starts = marked<R>(sh.start_id, w, lane), ends = marked<R>(sh.end_id, w, lane);

  float d[R][VEC], u[COMPL ? R : 1][VEC], sum[VEC] = {}, h[VEC] = {};
  auto restart = [&](int r) {  // a sequence's first row
    if (a.s0) {
      const Pair<float> s0 = load_pair(a.s0 + (int64_t)uniform(sh.start_id[w * R + r]) * a.D, ch, tail);
#pragma unroll
      for (int c = 0; c < VEC; ++c) h[c] = s0.v[c];
    } else {
#pragma unroll
      for (int c = 0; c < VEC; ++c) h[c] = 0.f;
    }
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const float g = (float)graw[r].v[c];
      d[r][c] = decay(g);
      if (COMPL) u[r][c] = one_minus_decay(g, d[r][c]) * (float)xraw[r].v[c];
      sum[c] += g;
    }
  }
  auto advance = [&](int r) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) h[c] = fmaf(d[r][c], h[c], COMPL ? u[r][c] : (float)xraw[r].v[c]);
  };
  if (starts == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) advance(r);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (starts >> r & 1) restart(r);
      advance(r);
    }
  }
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    sh.A[w][lane * VEC + c] = starts ? 0.f : decay(sum[c]);
    sh.B[w][lane * VEC + c] = h[c];
  }
  __syncthreads();

  hand_over<GROUPS, false>(sh, a, tile, tiles, tile > 0 && sh.start_id[0] < 0 && r0 >= c0 && r0 < cN, first, tid);
  __syncthreads();

  if (a.checkpoints && tid < NCH && first + tid < a.D) {
#pragma unroll
    for (int v = 0; v < WAVES; v += SCAN_ROWS / R)
      if (r0 + v * R >= c0 && r0 + v * R < cN)
        a.checkpoints[(r0 + v * R) / SCAN_ROWS * a.D + first + tid] = sh.A[v][tid];
  }
  if (!a.o) return;  // states only
#pragma unroll
  for (int c = 0; c < VEC; ++c) h[c] = sh.A[w][lane * VEC + c];
  XT *out = (XT *)a.o + t0 * a.o_st;
  if ((starts | ends) == 0 && t0 >= c0 && t0 + R <= cN && !tail.on) {
#pragma unroll
    for (int r = 0; r < R; ++r, out += a.o_st) {
      advance(r);
      if (mine) store_pair(out, ch, h);
    }
    return;
  }
#pragma unroll
  for (int r = 0; r < R; ++r, out += a.o_st) {
    if (starts >> r & 1) restart(r);
    advance(r);
    if (mine && t0 + r >= c0 && t0 + r < cN) store_pair(out, ch, h, tail);
    if (ends >> r & 1) {
      const int64_t i = uniform(sh.end_id[w * R + r]);
      if (a.final_state && mine) store_pair(a.final_state + i * a.D, ch, h, tail);
      if (a.cache) {
        const int64_t slot = index_at(a.slots, a.slots_is64, i);
        if (slot >= 0 && slot < a.num_slots && mine) store_pair(a.cache + slot * a.D, ch, h, tail);
      }
    }
  }
}

// Gradients, tiles handed out from the last rows to the first.  The gradient e of
// a row's state follows the recurrence in reverse, e <- a (d_o + e) from the row
// behind, cut at the sequences' last rows (where d_final_state enters), and is
// handed on between tiles the same way.  The states are formed again from the
// checkpoint at the tile's first row.  Tiles of 64 rows: a lane holds the decays, the
// factors of dg, d_o and (complement form) 1 - a of its rows, 107 to 128 registers for
// 8 rows of a pair (78 to 97 without 1 - a; the float32 complement form for few channel
// blocks spills one); at 80 registers, for three workgroups per CU, the complement form
// spills (491 us instead of 328 for a training step).
template <typename XT, typename GT, bool COMPL, bool GROUPS>
__global__ void __launch_bounds__(THREADS, 4) gdp_scan_backward_kernel(ScanArgs a, int tiles, int blocks) {
  constexpr int R = SCAN_ROWS / WAVES;
  using S = Shared<R>;
  __shared__ S sh;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool hand_on = tiles > 1;
  const int ticket = take_ticket(sh, a, hand_on, tid);
  const int tile = tiles - 1 - ticket / blocks;
  if (tile < 0) {
    empty_sequences(a, ticket - tiles * blocks, a.dfinal, a.ds0, tid);
    return;
  }
  const int first = (ticket % blocks) * NCH;
  const int64_t r0 = (int64_t)tile * SCAN_ROWS;
  const bool mine = first + lane * VEC < a.D;
  const uint32_t ch = mine ? first + lane * VEC : 0;
  const Tail tail{first + NCH > a.D && (a.D & 1), (uint32_t)a.D - 1};
  const int64_t t0 = r0 + w * R;

  Pair<GT> graw[R];
  Pair<XT> xraw[R], draw[R];
  load_rows<R>(graw, (const GT *)a.g, a.g_st, t0, a.T, ch, tail, a.streamed);
  load_rows<R>(xraw, (const XT *)a.x, a.x_st, t0, a.T, ch, tail, a.streamed);
  load_rows<R>(draw, (const XT *)a.dout, a.do_st, t0, a.T, ch, tail, a.streamed);
  const bool live = tid < NCH && first + tid < a.D;  // lane tid < NCH: channel first + tid of the hand-over
  float state = 0.f;
  if (live) state = a.checkpoints[(int64_t)tile * a.D + first + tid];
  const int64_t c0 = bound_at(a.cu, a.cu_is64, 0, a.T), cN = bound_at(a.cu, a.cu_is64, a.N, a.T);
  mark_rows(sh, a, r0, tid);
  const uint32_t starts = marked<R>(sh.start_id, w, lane), ends = marked<R>(sh.end_id, w, lane);

  // the states before the wave's rows: the forward maps of the waves, composed
  float d[R][VEC], m[COMPL ? R : 1][VEC], h[VEC] = {}, sum[VEC] = {};
  auto restart = [&](int r) {  // a sequence's first row
    if (a.s0) {
      const Pair<float> s0 = load_pair(a.s0 + (int64_t)uniform(sh.start_id[w * R + r]) * a.D, ch, tail);
#pragma unroll
      for (int c = 0; c < VEC; ++c) h[c] = s0.v[c];
    } else {
#pragma unroll
      for (int c = 0; c < VEC; ++c) h[c] = 0.f;
    }
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const float g = (float)graw[r].v[c];
      d[r][c] = decay(g);
      if (COMPL) m[r][c] = one_minus_decay(g, d[r][c]);
      sum[c] += g;
    }
  }
  auto advance = [&](int r) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const float x = (float)xraw[r].v[c];
      h[c] = fmaf(d[r][c], h[c], COMPL ? m[r][c] * x : x);
    }
  };
  if (starts == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) advance(r);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (starts >> r & 1) restart(r);
      advance(r);
    }
  }
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    sum[c] = decay(sum[c]);  // the product of the wave's decays, forward and in reverse
    sh.A[w][lane * VEC + c] = starts ? 0.f : sum[c];
    sh.B[w][lane * VEC + c] = h[c];
  }
  __syncthreads();
  if (tid < NCH) {
#pragma unroll
    for (int v = 0; v < WAVES; ++v) {
      const float next = apply(sh.A[v][tid], state, sh.B[v][tid]);
      sh.A[v][tid] = state;
      state = next;
    }
  }
  __syncthreads();
  // p = a (h before [- x]), by which e gives dg; then the wave's map of e
  float p[R][VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) h[c] = sh.A[w][lane * VEC + c];
  auto weigh = [&](int r) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) p[r][c] = d[r][c] * (COMPL ? h[c] - (float)xraw[r].v[c] : h[c]);
    advance(r);
  };
  if (starts == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) weigh(r);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (starts >> r & 1) restart(r);
      weigh(r);
    }
  }
  float e[VEC] = {};
  auto last_row = [&](int r, float (&e)[VEC]) {  // a sequence's last row: e comes from d_final_state
    if (a.dfinal) {
      const Pair<float> f = load_pair(a.dfinal + (int64_t)uniform(sh.end_id[w * R + r]) * a.D, ch, tail);
#pragma unroll
      for (int c = 0; c < VEC; ++c) e[c] = f.v[c];
    } else {
#pragma unroll
      for (int c = 0; c < VEC; ++c) e[c] = 0.f;
    }
  };
  auto retreat = [&](int r) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) e[c] = d[r][c] * ((float)draw[r].v[c] + e[c]);
  };
  if (ends == 0) {
#pragma unroll
    for (int r = R - 1; r >= 0; --r) retreat(r);
  } else {
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      if (ends >> r & 1) last_row(r, e);
      retreat(r);
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    sh.A[w][lane * VEC + c] = ends ? 0.f : sum[c];
    sh.B[w][lane * VEC + c] = e[c];
  }
  __syncthreads();

  const int64_t rl = r0 + SCAN_ROWS - 1;  // the tile's last row
  hand_over<GROUPS, true>(sh, a, tile, tiles, tile + 1 < tiles && sh.end_id[SCAN_ROWS - 1] < 0 && rl >= c0 && rl < cN,
                         first, tid);
  __syncthreads();

#pragma unroll
  for (int c = 0; c < VEC; ++c) e[c] = sh.A[w][lane * VEC + c];
  float dx[VEC], dg[VEC];
  auto gradients = [&](int r) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      e[c] += (float)draw[r].v[c];
      dx[c] = COMPL ? m[r][c] * e[c] : e[c];
      dg[c] = e[c] * p[r][c];
      e[c] *= d[r][c];
    }
  };
  // the rows' gradients, stored as float32 or as the inputs' types
  auto rows = [&](auto dx_type, auto dg_type) {
    using DX = decltype(dx_type);
    using DG = decltype(dg_type);
    DX *dx_row = (DX *)a.dx + (t0 + R - 1) * a.dx_st;
    DG *dg_row = (DG *)a.dg + (t0 + R - 1) * a.dg_st;
    if ((starts | ends) == 0 && t0 >= c0 && t0 + R <= cN && !tail.on) {
#pragma unroll
      for (int r = R - 1; r >= 0; --r, dx_row -= a.dx_st, dg_row -= a.dg_st) {
        gradients(r);
        if (mine) {
          store_pair(dx_row, ch, dx);
          store_pair(dg_row, ch, dg);
        }
      }
      return;
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r, dx_row -= a.dx_st, dg_row -= a.dg_st) {
      if (ends >> r & 1) last_row(r, e);
      gradients(r);
      if (t0 + r < c0 || t0 + r >= cN) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) dx[c] = dg[c] = 0.f;
      }
      if (mine && t0 + r < a.T) {
        store_pair(dx_row, ch, dx, tail);
        store_pair(dg_row, ch, dg, tail);
      }
      if ((starts >> r & 1) && a.ds0 && mine)
        store_pair(a.ds0 + (int64_t)uniform(sh.start_id[w * R + r]) * a.D, ch, e, tail);
    }
  };
  if (a.dx_f32) {
    if (a.dg_f32) rows(0.f, 0.f);
    else rows(0.f, (GT)0);
  } else {
    if (a.dg_f32) rows((XT)0, 0.f);
    else rows((XT)0, (GT)0);
  }
}

// The single-token step: a stream over the states that are named, 4.3 us for 256
// entries of 4096 channels (3.9 TB/s).
template <typename XT, typename GT>
__global__ void __launch_bounds__(256) gdp_scan_decode_kernel(ScanDecodeArgs a) {
  const int64_t i = blockIdx.x, ch = (int64_t)blockIdx.y * 256 + threadIdx.x;
  if (ch >= a.D) return;
  const int64_t slot = index_at(a.slots, a.slots_is64, i);
  XT *o = (XT *)a.o + i * a.o_st + ch;
  if (slot < 0 || slot >= a.num_slots) {
    *o = (XT)0.f;
    return;
  }
  const float g = (float)((const GT *)a.g)[i * a.g_st + ch], x = (float)((const XT *)a.x)[i * a.x_st + ch];
  const float d = decay(g);
  float *s = a.cache + slot * a.D + ch;
  const float h = fmaf(d, *s, a.complement ? one_minus_decay(g, d) * x : x);
  *s = h;
  *o = (XT)h;
}

template <typename F> hipError_t by_types(int xt, int gt, F f) {
  if (xt == EL_F32) return f((float)0, (float)0);
  if (xt == EL_BF16) return gt == EL_F32 ? f((bf16)0, (float)0) : f((bf16)0, (bf16)0);
  return gt == EL_F32 ? f((_Float16)0, (float)0) : f((_Float16)0, (_Float16)0);
}

// the counter and the words: everything to all-ones bits
__global__ void __launch_bounds__(256) gdp_scan_fill_kernel(uint4 *p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

struct Grid { int tiles, blocks; unsigned jobs; };

Grid grid_of(const ScanArgs &a, int rows, bool empties) {
  Grid g;
  g.tiles = (int)((a.T + rows - 1) / rows);
  g.blocks = (int)((a.D + NCH - 1) / NCH);
  g.jobs = (unsigned)((int64_t)g.tiles * g.blocks + (empties ? (a.N + 63) / 64 : 0));
  return g;
}

// Channel blocks up to which the states are handed on through groups of tiles.  The
// workgroups that run at once then work on more tiles of each block, and how far the
// known states come per look bounds the rate, not the memory: 131072 rows of 64, 256
// and 512 channels take 39, 74 and 120 us through groups and 139, 155 and 167 without;
// 1024 channels 220 and 216, and 131104 rows of 4096 channels 761 and 704.
constexpr int NARROW = 4;

hipError_t fill_words(const ScanArgs &a, const Grid &g, hipStream_t stream) {
  if (g.tiles <= 1) return hipSuccess;
  const int64_t words = g.tiles + (g.blocks <= NARROW ? g.tiles / GROUP : 0);
  const int64_t n = (256 + words * a.D * 8 + 15) / 16, want = (n + 255) / 256;
  hipLaunchKernelGGL(gdp_scan_fill_kernel, dim3((unsigned)(want < 2048 ? want : 2048)), dim3(256), 0, stream,
                     (uint4 *)a.ws, n);
  return hipGetLastError();
}

template <typename XT, typename GT> hipError_t run_scan(ScanArgs a, hipStream_t stream) {
  constexpr int R = SCAN_FORWARD_ROWS / WAVES;
  a.streamed = a.T * a.D * (int64_t)(2 * sizeof(XT) + sizeof(GT)) > STREAM_BYTES;
  const Grid k = grid_of(a, WAVES * R, a.N > 0 && (a.final_state || a.cache));
  if (k.jobs == 0) return hipSuccess;
  if (hipError_t e = fill_words(a, k, stream)) return e;
  auto *kernel = k.blocks <= NARROW ? (a.complement ? gdp_scan_kernel<XT, GT, R, true, true>
                                                    : gdp_scan_kernel<XT, GT, R, false, true>)
                                    : (a.complement ? gdp_scan_kernel<XT, GT, R, true, false>
                                                    : gdp_scan_kernel<XT, GT, R, false, false>);
  hipLaunchKernelGGL(kernel, dim3(k.jobs), dim3(THREADS), 0, stream, a, k.tiles, k.blocks);
  return hipGetLastError();
}

template <typename XT, typename GT> hipError_t run_backward(ScanArgs a, hipStream_t stream) {
  a.streamed = a.T * a.D * (int64_t)(3 * sizeof(XT) + 2 * sizeof(GT)) > STREAM_BYTES;
  const Grid k = grid_of(a, SCAN_ROWS, a.N > 0 && a.ds0);
  if (k.jobs == 0) return hipSuccess;
  if (hipError_t e = fill_words(a, k, stream)) return e;
  auto *kernel = k.blocks <= NARROW ? (a.complement ? gdp_scan_backward_kernel<XT, GT, true, true>
                                                    : gdp_scan_backward_kernel<XT, GT, false, true>)
                                    : (a.complement ? gdp_scan_backward_kernel<XT, GT, true, false>
                                                    : gdp_scan_backward_kernel<XT, GT, false, false>);
  hipLaunchKernelGGL(kernel, dim3(k.jobs), dim3(THREADS), 0, stream, a, k.tiles, k.blocks);
  return hipGetLastError();
}

}  // namespace

size_t scan_state_bytes(int64_t T, int64_t D, int rows) {
  const int64_t tiles = (T + rows - 1) / rows;
  return tiles <= 1 ? 0 : (256 + (size_t)(tiles + tiles / GROUP) * D * 8 + 255) & ~(size_t)255;
}

// A launch holds less than 2^32 threads: one workgroup per 64 rows and 128 channels at
// most, and one per 64 sequences; a decode step 256 threads per entry.  A row's
// channels are reached by 32-bit byte offsets.
bool scan_served(int64_t T, int64_t N, int64_t D) {
  if (T >= (int64_t)1 << 36 || N >= (int64_t)1 << 24 || D >= ((int64_t)1 << 24) - 256) return false;
  return (T / SCAN_ROWS + 1) * (D / NCH + 1) + N / 64 + 1 < ((int64_t)1 << 32) / THREADS;
}

hipError_t launch_scan(const ScanArgs &a, int xt, int gt, hipStream_t stream) {
  return by_types(xt, gt, [&](auto x, auto g) { return run_scan<decltype(x), decltype(g)>(a, stream); });
}

hipError_t launch_scan_backward(const ScanArgs &a, int xt, int gt, hipStream_t stream) {
  return by_types(xt, gt, [&](auto x, auto g) { return run_backward<decltype(x), decltype(g)>(a, stream); });
}

hipError_t launch_scan_decode(const ScanDecodeArgs &a, int xt, int gt, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  return by_types(xt, gt, [&](auto x, auto g) {
    hipLaunchKernelGGL((gdp_scan_decode_kernel<decltype(x), decltype(g)>),
                       dim3((unsigned)a.N, (unsigned)((a.D + 255) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace gdp
