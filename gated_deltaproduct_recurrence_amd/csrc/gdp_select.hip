// gdp_select.hip -- gfx950 kernels of the selective state space scan over packed
// sequences, per channel with S states,
//     delta_t = softplus(dt_t + bias)  (or dt_t + bias),
//     h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,
//     o_t = (C_t . h_t + skip u_t) silu(z_t),
// and of its single-token step.  B and C are shared by the channels of a group.
//
// What bounds it is the vector units: per element and state one exponential and four
// float32 operations, against 6 to 10 bytes per element.  So a lane holds a channel
// with all its states in registers, and B_t and C_t, the same for a whole wave, come to it
// from the wave's own LDS, four states per read.
//
// The time axis: a wave walks one chunk of a sequence (gdp_block_common.h).  Where a call has few
// channels and long sequences, chunks are short enough to fill the chip, and the
// states that enter them come from two kernels before: the chunks' own ends (from a state
// of 0; the decay over a chunk is exp(A sum delta), one sum per channel), and a walk over
// the chunks of each sequence.  A sequence's last chunk takes no part in the first of them;
// sequences of one chunk in neither.  Uneven chunks are handed out longest first.
//
// Measured on MI355X, 16 states, bfloat16 with a gate.  An exponential takes two issue slots
// and everything else one (counters), so a row of 64 channels has 140 slots in the main kernel
// and 104 in the one before it; the vector units are busy 94% of the time in both on 32768 x 2048
// in one sequence (254 + 185 us and 18 for the walk between, the call 452).  33824 x 4096 in 68
// sequences of 1 to 1024 rows: 549 us; 812 x 512 in 4: 25 us, latency of three launches.
// (A process's first calls take a quarter longer, until the clocks have risen.)
//   4096 waves wanted; 2048 and 8192: 482 and 466 us on the first shape instead of 450.
//   Of forms that are no longer there: B and C as scalar operands missed the scalar cache row by
// row (571 us on the first shape, 456 out of LDS); delta u B added by a matrix instruction (one
// for four states) saved 12 slots per row and was slower (466 instead of 456).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp.h"
#include "gdp_block.h"
#include "gdp_block_common.h"
#include "gdp_select_common.h"

namespace gdp {
namespace {

constexpr int WAVES = 4, ROWS = 4;  // waves per workgroup (or one), rows in flight

// Sorts the chunk numbers by their chunks' lengths, in 64 classes, longest first (those that
// name no chunk last).  Within a class they stand as their counters give them,
// which changes no result.
__global__ void __launch_bounds__(256) gdp_select_order_kernel(SelectArgs a, int shift, int numbers, int *order) {
  __shared__ int count[64], start[64];
  constexpr int EACH = (int)(MOST_ORDERED / 256);
  int cls[EACH];
  if (threadIdx.x < 64) count[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int number = j * 256 + threadIdx.x;
    cls[j] = -1;
    if (number >= numbers) continue;
    int lo = 0, hi = a.N;  // the last sequence whose numbers begin at or before it
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (chunk_number((int)bound_at(a.cu, a.cu_is64, mid, a.T), mid, shift) <= number) lo = mid;
      else hi = mid;
    }
    const int first = (int)bound_at(a.cu, a.cu_is64, lo, a.T), last = (int)bound_at(a.cu, a.cu_is64, lo + 1, a.T);
    const int64_t at = (int64_t)(number - chunk_number(first, lo, shift)) * ((int64_t)1 << shift);
    const int64_t left = at < 0 ? 0 : last - first - at;
    const int64_t rows = left < 0 ? 0 : (left < (int64_t)1 << shift ? left : (int64_t)1 << shift);
    cls[j] = 63 - (int)(rows * 63 >> shift);
    atomicAdd(&count[cls[j]], 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int sum = 0;
    for (int c = 0; c < 64; ++c) {
      start[c] = sum;
      sum += count[c];
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < EACH; ++j)
    if (cls[j] >= 0) order[atomicAdd(&start[cls[j]], 1)] = j * 256 + threadIdx.x;
}

// A wave's chunk and channels
struct Place { Chunk k; int number, ch, group; bool live; };
__device__ __forceinline__ bool place_of(Place *p, const SelectArgs &a, const SelectGrid &g, const int *order,
                                         int64_t jobs) {
  const int64_t id = (int64_t)blockIdx.x * (blockDim.x >> 6) + uniform_of(threadIdx.x >> 6);
  if (id >= jobs) return false;
  p->number = (int)(id / g.blocks);
  if (order) p->number = uniform_of(order[p->number]);
  if (!find_chunk(&p->k, a.cu, a.cu_is64, a.T, a.N, g.shift, p->number)) return false;
  const int b = (int)(id % g.blocks), per = a.D / a.G;
  p->group = b / g.per_group;
  const int at = (b % g.per_group) * 64 + (threadIdx.x & 63);
  p->live = at < per;
  p->ch = p->group * per + min(at, per - 1);  // lanes without a channel work on the last one's, and write nothing
  return true;
}

// M neighbouring rows of a lane's channel: raw, then as steps, weighted inputs and gates
template <typename UT, typename DT, int M> struct Rows {
  UT u[M], z[M];
  DT dt[M];
  __device__ __forceinline__ void load(const SelectArgs &a, int64_t t, int ch, bool gate) {
#pragma unroll
    for (int r = 0; r < M; ++r) {
      u[r] = ((const UT *)a.u)[(t + r) * a.u_st + ch];
      dt[r] = ((const DT *)a.dt)[(t + r) * a.dt_st + ch];
      if (gate) z[r] = ((const UT *)a.z)[(t + r) * a.z_st + ch];
    }
  }
  __device__ __forceinline__ void steps(float (&delta)[M], float bias, int softplus) const {
#pragma unroll
    for (int r = 0; r < M; ++r) delta[r] = (float)dt[r] + bias;
    if (softplus) {
#pragma unroll
      for (int r = 0; r < M; ++r) delta[r] = softplus_of(delta[r]);
    }
  }
};

// The states at the ends of the chunks that another chunk follows, from initial_state
// in a sequence's first chunk and from 0 elsewhere, and the sums of the steps.
template <typename UT, typename DT, int P>
__global__ void __launch_bounds__(64 * WAVES) gdp_select_ends_kernel(SelectArgs a, SelectGrid g, SelectSpace s,
                                                                     int64_t jobs) {
  __shared__ __attribute__((aligned(16))) float lds[WAVES][ROWS * P];
  Place p;
  if (!place_of(&p, a, g, s.order, jobs) || p.k.end == p.k.last) return;
  const int ch = p.ch;
  float A2[P], h[P];
  load_rates<P>(A2, a, ch);
  load_states<P>(h, a.s0 && p.k.index == 0 ? a.s0 + ((int64_t)p.k.seq * a.D + ch) * a.S : nullptr, a.S);
  const float bias = a.bias ? a.bias[ch] : 0.f;
  float *mine = lds[threadIdx.x >> 6];
  Rows<UT, DT, ROWS> next = {};
  Shared<UT, ROWS, P, 0> next_b;
  next.load(a, p.k.begin, ch, false);
  next_b.load(a, p.group, p.k.begin, 1);
  float sum = 0.f;
  // (a chunk that another follows is full: a multiple of ROWS rows)
  for (int t = p.k.begin; t < p.k.end; t += ROWS) {
    const Rows<UT, DT, ROWS> now = next;
    next_b.lay(mine);
    if (t + ROWS < p.k.end) {
      next.load(a, t + ROWS, ch, false);
      next_b.load(a, p.group, t + ROWS, 1);
    }
    float delta[ROWS], part = 0.f;
    now.steps(delta, bias, a.softplus);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float w = delta[r] * (float)now.u[r];
      part += delta[r];
#pragma unroll
      for (int n = 0; n < P; n += 4) {
        const float4 B = *(const float4 *)(mine + r * P + n);
        h[n] = fmaf(__builtin_amdgcn_exp2f(delta[r] * A2[n]), h[n], w * B.x);
        h[n + 1] = fmaf(__builtin_amdgcn_exp2f(delta[r] * A2[n + 1]), h[n + 1], w * B.y);
        h[n + 2] = fmaf(__builtin_amdgcn_exp2f(delta[r] * A2[n + 2]), h[n + 2], w * B.z);
        h[n + 3] = fmaf(__builtin_amdgcn_exp2f(delta[r] * A2[n + 3]), h[n + 3], w * B.w);
      }
    }
    sum += part;
  }
  if (!p.live) return;
  const int64_t slot = slot_behind(p.k, g.shift);
  float *out = s.states + slot * P * a.D + ch;
#pragma unroll
  for (int n = 0; n < P; ++n) out[(int64_t)n * a.D] = h[n];
  s.sums[slot * a.D + ch] = sum;
}

// The states behind the chunks that another follows, in place of those from 0: a lane walks
// these chunks of a sequence for one state of one channel.
template <int P>
__global__ void __launch_bounds__(256) gdp_select_enter_kernel(SelectArgs a, SelectGrid g, SelectSpace s) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;  // n D + ch
  if (at >= (int64_t)P * a.D) return;
  const int n = (int)(at / a.D), ch = (int)(at % a.D);
  const float A2 = n < a.S ? a.A[(int64_t)ch * a.S + n] * LOG2E_L : 0.f;
  for (int i = blockIdx.y; i < a.N; i += gridDim.y) {
    const int64_t first = bound_at(a.cu, a.cu_is64, i, a.T), len = bound_at(a.cu, a.cu_is64, i + 1, a.T) - first;
    const int64_t full = followed_chunks(len, g.shift);
    if (full < 2) continue;
    const int64_t step = (int64_t)P * a.D, slot = first >> g.shift;
    float *state = s.states + slot * step + at;
    const float *sum = s.sums + slot * a.D + ch;
    float h = *state;
    constexpr int AHEAD = 8;
    for (int64_t c = 1; c < full; c += AHEAD) {
      float end[AHEAD], d[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        end[j] = d[j] = 0.f;
        if (c + j < full) {
          end[j] = state[(c + j) * step];
          d[j] = sum[(c + j) * a.D];
        }
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        h = fmaf(__builtin_amdgcn_exp2f(A2 * d[j]), h, end[j]);
        if (c + j < full) state[(c + j) * step] = h;
      }
    }
  }
}

// ZEROS: there is no skip, or there are fewer states than P.  The zeros in their place times an
// infinite input would be NaN, so they are selected, not multiplied, and groups of four states
// behind the last one left out.  Otherwise that would cost 1 to 3%: 8192 x 2048 in 4 sequences
// take 69, 87, 125 and 210 us with 4, 8, 16 and 32 states, and 71, 88, 128 and 214 that way.
template <typename UT, typename DT, int P, bool ZEROS>
__global__ void __launch_bounds__(64 * WAVES) gdp_select_kernel(SelectArgs a, SelectGrid g, SelectSpace s,
                                                                int64_t jobs) {
  __shared__ __attribute__((aligned(16))) float lds[WAVES][ROWS * 2 * P];
  Place p;
  if (!place_of(&p, a, g, s.order, jobs)) return;
  const Chunk k = p.k;
  const int ch = p.ch;
  float A2[P], h[P];
  load_rates<P>(A2, a, ch);
  if (k.index > 0) {
    const float *enter = s.states + slot_before(k, g.shift) * P * a.D + ch;
#pragma unroll
    for (int n = 0; n < P; ++n) h[n] = enter[(int64_t)n * a.D];
  } else {
    load_states<P>(h, a.s0 ? a.s0 + ((int64_t)k.seq * a.D + ch) * a.S : nullptr, a.S);
  }
  if (k.begin < k.end) {
    const float bias = a.bias ? a.bias[ch] : 0.f, skip = a.skip ? a.skip[ch] : 0.f;
    const bool gate = a.z != nullptr;
    float *mine = lds[threadIdx.x >> 6];
    UT *o = (UT *)a.o + k.begin * a.o_st + ch;
    // M rows of the recurrence
    auto run = [&](const auto &x) {
      constexpr int M = sizeof(x.u) / sizeof(UT);
      float delta[M], y[M];
      x.steps(delta, bias, a.softplus);
      // states n .. n + 3 of row r, all of them or (at least one) up to the last one
      auto four = [&](auto all, int r, int n, float w, float (&s)[2]) {
        const float4 Bv = *(const float4 *)(mine + r * 2 * P + n), Cv = *(const float4 *)(mine + (r * 2 + 1) * P + n);
        const float B[4] = {Bv.x, Bv.y, Bv.z, Bv.w}, C[4] = {Cv.x, Cv.y, Cv.z, Cv.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float after = fmaf(__builtin_amdgcn_exp2f(delta[r] * A2[n + c]), h[n + c], w * B[c]);
          h[n + c] = decltype(all)::value || c == 0 || n + c < a.S ? after : 0.f;
          s[c & 1] = fmaf(h[n + c], C[c], s[c & 1]);
        }
      };
      if constexpr (!ZEROS) {
#pragma unroll
        for (int r = 0; r < M; ++r) {
          const float u = (float)x.u[r], w = delta[r] * u;
          float s[2] = {skip * u, 0.f};
#pragma unroll
          for (int n = 0; n < P; n += 4) four(Flag<true>(), r, n, w, s);
          y[r] = s[0] + s[1];
        }
      } else {
        float w[M], s[M][2];
#pragma unroll
        for (int r = 0; r < M; ++r) {
          const float u = (float)x.u[r];
          w[r] = delta[r] * u;
          s[r][0] = a.skip ? skip * u : 0.f;
          s[r][1] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < P; n += 4) {
          // (with half of the P states or fewer, the next smaller P were taken)
          if ((P > 4 && n < P / 2) || n + 4 <= a.S) {
#pragma unroll
            for (int r = 0; r < M; ++r) four(Flag<true>(), r, n, w[r], s[r]);
          } else if (n < a.S) {
#pragma unroll
            for (int r = 0; r < M; ++r) four(Flag<false>(), r, n, w[r], s[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < M; ++r) y[r] = s[r][0] + s[r][1];
      }
      if (gate) {
#pragma unroll
        for (int r = 0; r < M; ++r) y[r] *= act_of(GDP_ACT_SILU, (float)x.z[r]);
      }
      if (a.o && p.live) {
#pragma unroll
        for (int r = 0; r < M; ++r) o[r * a.o_st] = (UT)y[r];
      }
      o += M * a.o_st;
    };
    Rows<UT, DT, ROWS> next = {};
    Shared<UT, ROWS, P, 2> next_bc;
    const int whole = k.begin + ((k.end - k.begin) & ~(ROWS - 1));
    if (k.begin < whole) {
      next.load(a, k.begin, ch, gate);
      next_bc.load(a, p.group, k.begin, 1);
    }
    auto point = [&](int t) {  // before row t, the first of 16
      float *out = a.points + checkpoint_row(k.first, k.seq, t, SELECT_SHIFT) * a.S * a.D + ch;
#pragma unroll
      for (int n = 0; n < P; ++n)
        if (n < a.S && p.live) out[(int64_t)n * a.D] = h[n];
    };
    int t = k.begin;
    for (; t < whole; t += ROWS) {
      if (a.points && ((t - k.begin) & (SELECT_ROWS - 1)) == 0) point(t);
      const Rows<UT, DT, ROWS> now = next;
      next_bc.lay(mine);
      if (t + ROWS < whole) {
        next.load(a, t + ROWS, ch, gate);
        next_bc.load(a, p.group, t + ROWS, 1);
      }
      run(now);
    }
    if (a.points && t < k.end && ((t - k.begin) & (SELECT_ROWS - 1)) == 0) point(t);
    for (; t < k.end; ++t) {
      Rows<UT, DT, 1> one = {};
      Shared<UT, 1, P, 2> one_bc;
      one.load(a, t, ch, gate);
      one_bc.load(a, p.group, t, 1);
      one_bc.lay(mine);
      run(one);
    }
  }
  if (k.end != k.last || !p.live) return;
  if (a.final_state) store_states<P>(a.final_state + ((int64_t)k.seq * a.D + ch) * a.S, h, a.S);
  if (a.cache) {
    const int64_t slot = index_at(a.slots, a.slots_is64, k.seq);
    if (slot >= 0 && slot < a.num_slots) store_states<P>(a.cache + (slot * a.D + ch) * a.S, h, a.S);
  }
}

// One token: a stream over the states that are named, four states per lane.  The
// workgroups walk the channels of an entry before the next entry, so a state is read from end
// to end: 256 entries of 4096 channels of 16 states take 32 us (4.3 TB/s).  When this took 34, the
// entries walked first took 40, two entries per lane 33 and four 44.
template <typename UT, typename DT, int P>
__global__ void __launch_bounds__(256) gdp_select_decode_kernel(SelectArgs a, int blocks) {
  constexpr int LANES = P / 4;  // of one channel
  const int64_t i = blockIdx.x / (unsigned)blocks;
  const int ch = (int)(blockIdx.x % (unsigned)blocks) * (256 / LANES) + threadIdx.x / LANES;
  const int n0 = (threadIdx.x % LANES) * 4;
  if (ch >= a.D) return;
  const int64_t slot = index_at(a.slots, a.slots_is64, i);
  UT *o = (UT *)a.o + i * a.o_st + ch;
  if (slot < 0 || slot >= a.num_slots) {
    if (n0 == 0) *o = (UT)0.f;
    return;
  }
  const int group = ch / (a.D / a.G);
  float *state = a.cache + (slot * a.D + ch) * a.S;
  Piece<float, 4> h = load_piece<float, 4>(state, n0, a.S);
  const Piece<float, 4> A = load_piece<float, 4>(a.A + (int64_t)ch * a.S, n0, a.S);
  const Piece<UT, 4> B = load_piece<UT, 4>((const UT *)a.B + i * a.B_st + group * a.B_sg, n0, a.S),
                     C = load_piece<UT, 4>((const UT *)a.C + i * a.C_st + group * a.C_sg, n0, a.S);
  const float u = (float)((const UT *)a.u)[i * a.u_st + ch];
  const float v = (float)((const DT *)a.dt)[i * a.dt_st + ch] + (a.bias ? a.bias[ch] : 0.f);
  const float delta = a.softplus ? softplus_of(v) : v, w = delta * u;
  float y = 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    h.v[c] = fmaf(__builtin_amdgcn_exp2f(delta * (A.v[c] * LOG2E_L)), h.v[c], w * (float)B.v[c]);
    if (n0 + c < a.S) y = fmaf(h.v[c], (float)C.v[c], y);
  }
  store_piece<float, 4>(state, n0, a.S, h);
  y = team_sum(y, LANES);
  if (n0 == 0) {
    y += a.skip ? a.skip[ch] * u : 0.f;
    if (a.z) y *= act_of(GDP_ACT_SILU, (float)((const UT *)a.z)[i * a.z_st + ch]);
    *o = (UT)y;
  }
}

}  // namespace

// A launch holds less than 2^32 threads: a wave per chunk and block of 64 channels forward, up
// to 8 in the gradients; the decode step 256 threads per entry and at least 32 channels.
bool select_served(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S) {
  if (T > BLOCK_MAX_ROWS || N > BLOCK_MAX_SEQS || D > BLOCK_MAX_CHANNELS) return false;
  const SelectGrid f = forward_grid(T, N, D, G), b = backward_grid(T, N, D, G);
  const int64_t most = (int64_t)1 << 32;
  return f.numbers * f.blocks + WAVES < most / 64 && b.numbers * b.blocks < most / 512 && N * ((D + 31) / 32) < most / 256;
}

size_t select_bytes(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S) {
  return select_space(nullptr, D, S, forward_grid(T, N, D, G)).bytes;
}

hipError_t launch_select(const SelectArgs &a, int ut, int dt, hipStream_t stream) {
  const SelectGrid g = forward_grid(a.T, a.N, a.D, a.G);
  const int64_t jobs = g.numbers * g.blocks;
  if (jobs == 0 || a.N == 0) return hipSuccess;
  SelectSpace s = select_space(a.ws, a.D, a.S, g);
  // one wave per workgroup while that leaves compute units without one: 812 rows of 512
  // channels take 26.2 us so and 26.8 with four, 32768 of 2048 take 483 and 450
  const int waves = jobs <= 1024 ? 1 : WAVES;
  // (the chunks of one sequence stand in order, and few waves all run at once)
  if (a.N == 1 || waves == 1) s.order = nullptr;
  if (s.order) {
    hipLaunchKernelGGL(gdp_select_order_kernel, dim3(1), dim3(256), 0, stream, a, g.shift, (int)g.numbers, s.order);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return select_types(ut, dt, [&](auto u, auto d) {
    using UT = decltype(u);
    using DT = decltype(d);
    return by_states(a.S, [&](auto n) {
      constexpr int P = decltype(n)::value;
      const dim3 grid((unsigned)((jobs + waves - 1) / waves)), threads(64 * waves);
      if (a.T > (int64_t)1 << g.shift) {  // else no sequence has two chunks
        hipLaunchKernelGGL((gdp_select_ends_kernel<UT, DT, P>), grid, threads, 0, stream, a, g, s, jobs);
        if (hipError_t e = hipGetLastError()) return e;
        const dim3 lanes((unsigned)(((int64_t)P * a.D + 255) / 256), (unsigned)(a.N < 32 ? a.N : 32));
        hipLaunchKernelGGL(gdp_select_enter_kernel<P>, lanes, dim3(256), 0, stream, a, g, s);
        if (hipError_t e = hipGetLastError()) return e;
      }
      auto *kernel = !a.skip || a.S < P ? gdp_select_kernel<UT, DT, P, true> : gdp_select_kernel<UT, DT, P, false>;
      hipLaunchKernelGGL(kernel, grid, threads, 0, stream, a, g, s, jobs);
      return hipGetLastError();
    });
  });
}

hipError_t launch_select_decode(const SelectArgs &a, int ut, int dt, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  return select_types(ut, dt, [&](auto u, auto d) {
    return by_states(a.S, [&](auto n) {
      constexpr int P = decltype(n)::value, channels = 256 / (P / 4);
      const int64_t blocks = (a.D + channels - 1) / channels;
      hipLaunchKernelGGL((gdp_select_decode_kernel<decltype(u), decltype(d), P>), dim3((unsigned)(a.N * blocks)),
                         dim3(256), 0, stream, a, (int)blocks);
      return hipGetLastError();
    });
  });
}

}  // namespace gdp
