// gdp_select_bwd.hip -- gfx950 kernels of the selective scan's gradients
// (gdp_select.hip has the recurrence).  With gy_t = d_o_t silu(z_t) and e_t the gradient
// of the state after token t, walking back,
//     e_t = C_t gy_t + a_{t+1} e_{t+1},   a_t = exp(delta_t A),
//     du_t = skip gy_t + delta_t (e_t . B_t),
//     ddelta_t = e_t . (A a_t h_{t-1} + u_t B_t),  d dt_t = ddelta_t softplus'(dt_t + bias),
//     dA = sum_t delta_t a_t e_t h_{t-1},  dskip = sum gy u,  dbias = sum d dt,
//     dB_t = sum over channels of e_t delta_t u_t,  dC_t = sum of gy_t h_t,
//     dz_t = d_o_t silu'(z_t) (C_t . h_t + skip u_t),  d_initial_state = a_0 e_0.
//
// Blocks of 16 rows, last to first: the states within a block are formed again from
// the forward pass's checkpoint at its first row and stay in registers, with their
// decays, for the way back, so each exponential is taken once.  16 rows of S states are
// too many for one lane; a workgroup's waves share 64 channels, four states each, and
// what is summed over the states (three values per row) meets in LDS.  What is
// summed over channels, 8 values per row and wave, is reduced over the lanes by
// exchanging halves: each step adds two values into one register, so 64 sums of 64
// lanes cost two instructions each and no LDS.  Their partial sums per 64 channels
// go to the workspace, and a last kernel adds them in a fixed order.
//
// The time axis is cut into chunks as in the forward pass; the gradients that enter them
// from behind come from two kernels before.
//
// Measured on MI355X, 8192 x 2048 in 4 sequences, 16 states, bfloat16 with a gate: 230 us, the
// vector units busy 77% of the time (the kernels before it 62 and 7 us, the sums 20), at
// 250 registers and two waves per SIMD.  1024 and 4096 workgroups wanted in place of 2048:
// the training step takes 518 and 463 us instead of 457.
//   With 4, 8, 24 and 32 states 168, 268, 443 and 445 us: up to 8 states a wave holds 8 or 16 rows of
// a block and loads none ahead, up to 4 a workgroup is one wave, from 17 on some registers spill.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp.h"
#include "gdp_block.h"
#include "gdp_block_common.h"
#include "gdp_select_common.h"

namespace gdp {
namespace {

constexpr int WAVES = 4, ROWS = 4;           // of the kernel over whole channels
constexpr int R = SELECT_ROWS, HALF = R / 2;
constexpr int OWN = 4;                       // states per wave

struct BackwardSpace {
  SelectSpace s;     // states: the gradients behind the chunks that another follows
  float *points;     // checkpoints of a call without them
  float *shares;     // [blocks, T, 2, padded S]: dB and dC over 64 channels
  float *sums;       // [numbers, waves OWN + 2, D]: dA, dskip, dbias over chunks
  size_t bytes;
};
BackwardSpace backward_space(void *ws, int64_t T, int64_t N, int64_t D, int64_t G, int64_t S, const SelectGrid &g,
                             bool with_points) {
  BackwardSpace b;
  const int64_t P = padded_states(S);
  b.s = select_space(ws, D, S, g);
  size_t at = b.s.bytes;
  if (!with_points) {  // the forward pass's space comes first, in the same place
    const size_t forward = select_space(ws, D, S, forward_grid(T, N, D, G)).bytes;
    at = forward > at ? forward : at;
  }
  b.points = (float *)((uintptr_t)ws + at);
  if (!with_points) at += round256((size_t)chunk_numbers(T, N, SELECT_SHIFT) * S * D * 4);
  b.shares = (float *)((uintptr_t)ws + at);
  at += round256((size_t)g.blocks * T * 2 * P * 4);
  b.sums = (float *)((uintptr_t)ws + at);
  at += round256((size_t)g.numbers * (P + 2) * D * 4);
  b.bytes = at;
  return b;
}
template <typename UT, typename DT, int M> struct Back {
  UT d_o[M], z[M];
  DT dt[M];
};

// The gradients of the states entering the chunks that follow another, of what the chunk's
// own rows (and in a sequence's last chunk d_final_state) contribute, and the sums of
// the steps.
template <typename UT, typename DT, int P>
__global__ void __launch_bounds__(64 * WAVES) gdp_select_starts_kernel(SelectArgs a, SelectGrid g, SelectSpace s,
                                                                       int64_t jobs) {
  const int64_t id = (int64_t)blockIdx.x * WAVES + uniform_of(threadIdx.x >> 6);
  if (id >= jobs) return;
  const int number = (int)(id / g.blocks), b = (int)(id % g.blocks), per = a.D / a.G, group = b / g.per_group;
  const int at = (b % g.per_group) * 64 + (threadIdx.x & 63), ch = group * per + min(at, per - 1);
  __shared__ __attribute__((aligned(16))) float lds[WAVES][ROWS * P];
  float *mine = lds[threadIdx.x >> 6];
  Chunk k;
  if (!find_chunk(&k, a.cu, a.cu_is64, a.T, a.N, g.shift, number) || k.index == 0) return;
  float A2[P], e[P];
  load_rates<P>(A2, a, ch);
  load_states<P>(e, k.end == k.last && a.dfinal ? a.dfinal + ((int64_t)k.seq * a.D + ch) * a.S : nullptr, a.S);
  const float bias = a.bias ? a.bias[ch] : 0.f;
  const bool gate = a.z != nullptr;
  // rows t, t - 1, ..
  auto load = [&](auto &x, int t) {
    constexpr int M = sizeof(x.d_o) / sizeof(UT);
#pragma unroll
    for (int r = 0; r < M; ++r) {
      x.d_o[r] = ((const UT *)a.d_o)[(t - r) * a.do_st + ch];
      x.dt[r] = ((const DT *)a.dt)[(t - r) * a.dt_st + ch];
      if (gate) x.z[r] = ((const UT *)a.z)[(t - r) * a.z_st + ch];
    }
  };
  float sum = 0.f;
  auto run = [&](const auto &x) {
    constexpr int M = sizeof(x.d_o) / sizeof(UT);
    float delta[M], gy[M], part = 0.f;
#pragma unroll
    for (int r = 0; r < M; ++r) {
      delta[r] = (float)x.dt[r] + bias;
      gy[r] = (float)x.d_o[r];
    }
    if (a.softplus) {
#pragma unroll
      for (int r = 0; r < M; ++r) delta[r] = softplus_of(delta[r]);
    }
    if (gate) {
#pragma unroll
      for (int r = 0; r < M; ++r) gy[r] *= act_of(GDP_ACT_SILU, (float)x.z[r]);
    }
#pragma unroll
    for (int r = 0; r < M; ++r) {
      part += delta[r];
#pragma unroll
      for (int n = 0; n < P; n += 4) {
        const float4 v = *(const float4 *)(mine + r * P + n);
        const float C[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          e[n + c] = __builtin_amdgcn_exp2f(delta[r] * A2[n + c]) * fmaf(C[c], gy[r], e[n + c]);
      }
    }
    sum += part;
  };
  int t = k.end - 1;
  Back<UT, DT, ROWS> next = {};
  Shared<UT, ROWS, P, 1> next_c;
  if (t - ROWS + 1 >= k.begin) {
    load(next, t);
    next_c.load(a, group, t, -1);
  }
  for (; t - ROWS + 1 >= k.begin; t -= ROWS) {
    const Back<UT, DT, ROWS> now = next;
    next_c.lay(mine);
    if (t - 2 * ROWS + 1 >= k.begin) {
      load(next, t - ROWS);
      next_c.load(a, group, t - ROWS, -1);
    }
    run(now);
  }
  for (; t >= k.begin; --t) {
    Back<UT, DT, 1> one = {};
    Shared<UT, 1, P, 1> one_c;
    load(one, t);
    one_c.load(a, group, t, -1);
    one_c.lay(mine);
    run(one);
  }
  if (at >= per) return;
  const int64_t slot = slot_before(k, g.shift);
  float *out = s.states + slot * P * a.D + ch;
#pragma unroll
  for (int n = 0; n < P; ++n) out[(int64_t)n * a.D] = e[n];
  s.sums[slot * a.D + ch] = sum;
}

// The gradients behind the chunks that another follows, in place of what the chunk behind
// contributes: a lane walks these chunks of a sequence, last to first, for one state of one
// channel.
template <int P>
__global__ void __launch_bounds__(256) gdp_select_behind_kernel(SelectArgs a, SelectGrid g, SelectSpace s) {
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
    float e = state[(full - 1) * step];
    constexpr int AHEAD = 8;
    for (int64_t c = full - 2; c >= 0; c -= AHEAD) {
      float own[AHEAD], d[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        own[j] = d[j] = 0.f;
        if (c - j >= 0) {
          own[j] = state[(c - j) * step];
          d[j] = sum[(c - j) * a.D];
        }
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        e = fmaf(__builtin_amdgcn_exp2f(A2 * d[j]), e, own[j]);
        if (c - j >= 0) state[(c - j) * step] = e;
      }
    }
  }
}

// x and y summed over pairs of lanes: the lower half of the lanes (of 64, of each 32)
// gets x's sums, the upper half y's
__device__ __forceinline__ float add_halves(float x, float y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_quarters(float x, float y) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// ... within 16 lanes: lanes without `upper` get x's sums, those with it y's; CTRL moves a
// lane's value to one on the other side
template <int CTRL> __device__ __forceinline__ float add_within(float x, float y, bool upper) {
  const float keep = upper ? y : x, give = upper ? x : y;
  return keep + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(give), CTRL, 0xf, 0xf, true));
}

// LDS: five values per row and channel, B and C, then the waves' sums over their states
template <int P> struct alignas(16) Tile {
  float bc[R][2][P];
  float delta[R][64], u[R][64], gy[R][64];
  float zs[R][64];  // d_o silu'(z)
  float ds[R][64];  // softplus'
};
struct Part { float through[R][64], carried[R][64], y[R][64]; };

template <typename UT, typename DT, int P>
__global__ void __launch_bounds__(64 * (P / OWN)) __attribute__((amdgpu_waves_per_eu(P > 4 ? 2 : 1)))
gdp_select_backward_kernel(SelectArgs a, SelectGrid g, BackwardSpace b) {
  constexpr int W = P / OWN, MINE = R / W;  // waves, rows of a block that a wave loads and finishes: w, w + W, ..
  __shared__ Tile<P> tile;
  __shared__ Part parts[W];
  const int w = uniform_of(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int number = (int)(blockIdx.x / (unsigned)g.blocks), blk = (int)(blockIdx.x % (unsigned)g.blocks);
  const int per = a.D / a.G, group = blk / g.per_group, at = (blk % g.per_group) * 64 + lane;
  const bool live = at < per;
  const int ch = group * per + (live ? at : per - 1);  // lanes without a channel hold the last one's, as zeros
  Chunk k;
  const bool some = find_chunk(&k, a.cu, a.cu_is64, a.T, a.N, g.shift, number);
  // the wave's places in LDS, as vector registers (as scalars every row's address is a
  // scalar of its own, and they spill)
  int mine = w;
  asm("" : "+v"(mine));
  const float *my_bc = &tile.bc[0][0][mine * OWN];
  Part *my_part = (Part *)&parts[mine].through[0][lane];
  float A[OWN], A2[OWN], e[OWN], dA[OWN] = {}, dskip = 0.f, dbias = 0.f;
  const float skip = a.skip ? a.skip[ch] : 0.f;
#pragma unroll
  for (int n = 0; n < OWN; ++n) {
    A[n] = w * OWN + n < a.S ? a.A[(int64_t)ch * a.S + w * OWN + n] : 0.f;
    A2[n] = A[n] * LOG2E_L;
    e[n] = 0.f;
  }
  if (some) {
    const float bias = a.bias ? a.bias[ch] : 0.f;
    const bool gate = a.z != nullptr;
    if (k.end < k.last) {
      const float *behind = b.s.states + (slot_behind(k, g.shift) * P + w * OWN) * a.D + ch;
#pragma unroll
      for (int n = 0; n < OWN; ++n) e[n] = live ? behind[(int64_t)n * a.D] : 0.f;
    } else if (a.dfinal) {
#pragma unroll
      for (int n = 0; n < OWN; ++n)
        if (live && w * OWN + n < a.S) e[n] = a.dfinal[((int64_t)k.seq * a.D + ch) * a.S + w * OWN + n];
    }
    // a block's inputs, loaded a block ahead where a wave holds few rows of them
    constexpr bool AHEAD = MINE <= 4;
    UT u_[MINE] = {}, z_[MINE] = {}, do_[MINE] = {};
    DT dt_[MINE] = {};
    float point[OWN] = {};
    UT bc_[2] = {};  // 2 P values per row: two of a block's per lane of the workgroup, HALF rows apart
    const Shares<UT> mine_bc = shares_of<UT>(a, threadIdx.x / P & 1, group);
    const int bc_n = threadIdx.x % P, bc_r = threadIdx.x / (2 * P);
    auto fetch = [&](int t0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t t = t0 + bc_r + i * HALF;
        if (t < k.end && bc_n < a.S) bc_[i] = mine_bc.p[t * mine_bc.st + bc_n];
      }
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int64_t t = t0 + w + i * W;
        if (t < k.end) {
          u_[i] = ((const UT *)a.u)[t * a.u_st + ch];
          dt_[i] = ((const DT *)a.dt)[t * a.dt_st + ch];
          do_[i] = ((const UT *)a.d_o)[t * a.do_st + ch];
          if (gate) z_[i] = ((const UT *)a.z)[t * a.z_st + ch];
        }
      }
      const int64_t row = checkpoint_row(k.first, k.seq, t0, SELECT_SHIFT);
      const float *p = a.points + (row * a.S + w * OWN) * a.D + ch;
#pragma unroll
      for (int n = 0; n < OWN; ++n)
        if (w * OWN + n < a.S) point[n] = p[(int64_t)n * a.D];
    };
    int t0 = k.begin + ((k.end - k.begin - 1) & ~(R - 1));
    if (AHEAD && k.begin < k.end) fetch(t0);
    for (; t0 >= k.begin && k.begin < k.end; t0 -= R) {
      const int rows = min(R, k.end - t0);
      if (!AHEAD) fetch(t0);
      // the rows' steps, inputs and output gradients, and the slopes for what follows
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int r = w + i * W;
        float delta = 0.f, u = 0.f, gy = 0.f, zs = 0.f, ds = 0.f;
        if (r < rows) {
          const float v = (float)dt_[i] + bias;
          u = live ? (float)u_[i] : 0.f;
          gy = live ? (float)do_[i] : 0.f;
          delta = a.softplus ? softplus_of(v) : v;
          ds = a.softplus ? sigmoid_of(v) : 1.f;
          if (gate) {
            const float f = act_of(GDP_ACT_SILU, (float)z_[i], &zs);
            zs *= gy;
            gy *= f;
          }
        }
        tile.delta[r][lane] = live ? delta : 0.f;
        tile.u[r][lane] = u;
        tile.gy[r][lane] = live ? gy : 0.f;
        tile.zs[r][lane] = zs;
        tile.ds[r][lane] = ds;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) (&tile.bc[0][0][0])[threadIdx.x + i * 64 * W] = (float)bc_[i];
      float h[R][OWN], d[R][OWN], last[OWN];  // states before the rows, decays; the state behind the block
#pragma unroll
      for (int n = 0; n < OWN; ++n) last[n] = live ? point[n] : 0.f;
      __syncthreads();
      if (AHEAD && t0 > k.begin) fetch(t0 - R);
      auto four = [&](float (&x)[OWN], int r, int which) {
        const float4 v = *(const float4 *)(my_bc + (r * 2 + which) * P);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
      };
      auto forward = [&](int r) {
        float B[OWN];
        four(B, r, 0);
        const float delta = tile.delta[r][lane], x = delta * tile.u[r][lane];
#pragma unroll
        for (int n = 0; n < OWN; ++n) {
          h[r][n] = last[n];
          d[r][n] = __builtin_amdgcn_exp2f(delta * A2[n]);
          last[n] = fmaf(d[r][n], last[n], x * B[n]);
        }
        if (r % 2 == 1) __builtin_amdgcn_sched_barrier(0);  // or more rows' operands are read ahead than fit
      };
      float share[2 * HALF];
      auto backward = [&](int r) {
        float B[OWN], C[OWN];
        four(B, r, 0);
        four(C, r, 1);
        const int i = r & (HALF - 1);
        const float delta = tile.delta[r][lane], x = delta * tile.u[r][lane], gy = tile.gy[r][lane];
        float q[2 * OWN], s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int n = 0; n < OWN; ++n) {
          const float after = r + 1 < R ? h[r + 1 < R ? r + 1 : r][n] : last[n];
          s3 = fmaf(C[n], after, s3);
          q[OWN + n] = gy * after;
          e[n] = fmaf(C[n], gy, e[n]);
          s1 = fmaf(e[n], B[n], s1);
          q[n] = e[n] * x;
          e[n] *= d[r][n];
          const float c = e[n] * h[r][n];
          s2 = fmaf(c, A[n], s2);
          dA[n] = fmaf(c, delta, dA[n]);
        }
        my_part->through[r][0] = s1;
        my_part->carried[r][0] = s2;
        my_part->y[r][0] = s3;
        // 16 lanes each of (q0, q2, q1, q3), and of (q4, q6, q5, q7)
        share[2 * i] = add_quarters(add_halves(q[0], q[1]), add_halves(q[2], q[3]));
        share[2 * i + 1] = add_quarters(add_halves(q[4], q[5]), add_halves(q[6], q[7]));
        if (r % 2 == 0) __builtin_amdgcn_sched_barrier(0);
      };
      // the sums over lanes of rows [first, first + HALF)
      auto store_shares = [&](int first) {
        const bool b3 = lane & 8, b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
        float s[HALF], s4[HALF / 2], s2[HALF / 4];
#pragma unroll
        for (int i = 0; i < HALF; ++i) s[i] = add_within<0x140>(share[2 * i], share[2 * i + 1], b3);  // row_mirror
#pragma unroll
        for (int i = 0; i < HALF / 2; ++i) s4[i] = add_within<0x141>(s[2 * i], s[2 * i + 1], b2);  // row_half_mirror
#pragma unroll
        for (int i = 0; i < HALF / 4; ++i) s2[i] = add_within<0x4e>(s4[2 * i], s4[2 * i + 1], b1);  // quad 2, 3, 0, 1
        const float one = add_within<0xb1>(s2[0], s2[1], b0);                                       // quad 1, 0, 3, 2
        const int row = (b2 ? 1 : 0) + (b1 ? 2 : 0) + (b0 ? 4 : 0), part = lane >> 4;
        const int n = part == 1 ? 2 : (part == 2 ? 1 : part);
        if (first + row < rows)
          b.shares[(((int64_t)blk * a.T + t0 + first + row) * 2 + (b3 ? 1 : 0)) * P + w * OWN + n] = one;
      };
      if (rows == R) {
#pragma unroll
        for (int r = 0; r < R; ++r) forward(r);
#pragma unroll
        for (int r = R - 1; r >= HALF; --r) backward(r);
        store_shares(HALF);
#pragma unroll
        for (int r = HALF - 1; r >= 0; --r) backward(r);
        store_shares(0);
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (r < rows) {
            forward(r);
          } else {  // the state behind the last row, for that row
#pragma unroll
            for (int n = 0; n < OWN; ++n) h[r][n] = last[n];
          }
        }
#pragma unroll
        for (int i = 0; i < 2 * HALF; ++i) share[i] = 0.f;
        if (rows > HALF) {
#pragma unroll
          for (int r = R - 2; r >= HALF; --r)
            if (r < rows) backward(r);
          store_shares(HALF);
        }
#pragma unroll
        for (int r = HALF - 1; r >= 0; --r)
          if (r < rows) backward(r);
        store_shares(0);
      }
      __syncthreads();
      // a wave's rows; it alone writes them in the tile again
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int r = w + i * W;
        if (r >= rows) continue;
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int v = 0; v < W; ++v) {
          s1 += parts[v].through[r][lane];
          s2 += parts[v].carried[r][lane];
          s3 += parts[v].y[r][lane];
        }
        const int64_t t = t0 + r;
        const float u = tile.u[r][lane], gy = tile.gy[r][lane];
        const float ddt = fmaf(u, s1, s2) * tile.ds[r][lane];
        dskip = fmaf(gy, u, dskip);
        dbias += ddt;
        if (!live) continue;
        ((UT *)a.du)[t * a.du_st + ch] = (UT)fmaf(tile.delta[r][lane], s1, a.skip ? skip * gy : 0.f);
        ((DT *)a.ddt)[t * a.ddt_st + ch] = (DT)ddt;
        if (gate) ((UT *)a.dz)[t * a.dz_st + ch] = (UT)(tile.zs[r][lane] * (a.skip ? fmaf(skip, u, s3) : s3));
      }
    }
    if (k.index == 0 && a.ds0 && live) {
#pragma unroll
      for (int n = 0; n < OWN; ++n)
        if (w * OWN + n < a.S) a.ds0[((int64_t)k.seq * a.D + ch) * a.S + w * OWN + n] = e[n];
    }
  }
  // sums over the chunk; a number that names none has zeros
  float *sums = b.sums + (int64_t)number * (P + 2) * a.D + ch;
  if (live) {
#pragma unroll
    for (int n = 0; n < OWN; ++n) sums[(int64_t)(w * OWN + n) * a.D] = dA[n];
  }
  __syncthreads();
  parts[w].through[0][lane] = dskip;
  parts[w].carried[0][lane] = dbias;
  __syncthreads();
  if (w == 0 && live) {
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      s1 += parts[v].through[0][lane];
      s2 += parts[v].carried[0][lane];
    }
    sums[(int64_t)P * a.D] = s1;
    sums[(int64_t)(P + 1) * a.D] = s2;
  }
}

// dB and dC from the channel blocks' shares; zeros in all rows that no sequence covers
template <typename UT, typename DT>
__global__ void __launch_bounds__(256) gdp_select_rows_kernel(SelectArgs a, SelectGrid g, BackwardSpace b, int P) {
  const int64_t c0 = bound_at(a.cu, a.cu_is64, 0, a.T), cN = a.N > 0 ? bound_at(a.cu, a.cu_is64, a.N, a.T) : 0;
  // four states per lane, eight blocks' loads ahead
  const int64_t all = (int64_t)a.T * a.G * 2 * P, block = (int64_t)a.T * 2 * P;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < all; i += (int64_t)gridDim.x * 1024) {
    const int n = (int)(i & (P - 1)), which = (int)(i / P & 1);
    const int64_t group = i / block, t = i / (2 * P) % a.T;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (t >= c0 && t < cN) {
      const float *p = b.shares + group * g.per_group * block + i % block;
      int j = 0;
      for (; j + 8 <= g.per_group; j += 8) {
        float4 x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = *(const float4 *)(p + (j + q) * block);
#pragma unroll
        for (int q = 0; q < 8; ++q) s[0] += x[q].x, s[1] += x[q].y, s[2] += x[q].z, s[3] += x[q].w;
      }
      for (; j < g.per_group; ++j) {
        const float4 x = *(const float4 *)(p + j * block);
        s[0] += x.x, s[1] += x.y, s[2] += x.z, s[3] += x.w;
      }
    }
    UT *out = (UT *)(which ? a.dC : a.dB) + (t * a.G + group) * a.S + n;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (n + c < a.S) out[c] = (UT)s[c];
  }
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (t >= c0 && t < cN) continue;
    for (int ch = threadIdx.x; ch < a.D; ch += 256) {
      ((UT *)a.du)[t * a.du_st + ch] = (UT)0.f;
      ((DT *)a.ddt)[t * a.ddt_st + ch] = (DT)0.f;
      if (a.dz) ((UT *)a.dz)[t * a.dz_st + ch] = (UT)0.f;
    }
  }
}

}  // namespace

size_t select_backward_bytes(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S, bool with_points) {
  return backward_space(nullptr, T, N, D, G, S, backward_grid(T, N, D, G), with_points).bytes;
}

hipError_t launch_select_backward(const SelectArgs &given, int ut, int dt, hipStream_t stream) {
  SelectArgs a = given;
  const SelectGrid g = backward_grid(a.T, a.N, a.D, a.G);
  const BackwardSpace b = backward_space(a.ws, a.T, a.N, a.D, a.G, a.S, g, a.points != nullptr);
  if (!a.points) {  // the checkpoints again, into the workspace (which begins as the forward pass's)
    a.points = b.points;
    if (hipError_t e = launch_select(a, ut, dt, stream)) return e;
  }
  const int64_t jobs = g.numbers * g.blocks;
  return select_types(ut, dt, [&](auto u, auto d) {
    using UT = decltype(u);
    using DT = decltype(d);
    return by_states(a.S, [&](auto n) {
      constexpr int P = decltype(n)::value;
      if (a.T > (int64_t)1 << g.shift && a.N > 0) {  // else no sequence has two chunks
        hipLaunchKernelGGL((gdp_select_starts_kernel<UT, DT, P>), dim3((unsigned)((jobs + WAVES - 1) / WAVES)),
                           dim3(64 * WAVES), 0, stream, a, g, b.s, jobs);
        if (hipError_t e = hipGetLastError()) return e;
        const dim3 lanes((unsigned)(((int64_t)P * a.D + 255) / 256), (unsigned)(a.N < 32 ? a.N : 32));
        hipLaunchKernelGGL(gdp_select_behind_kernel<P>, lanes, dim3(256), 0, stream, a, g, b.s);
        if (hipError_t e = hipGetLastError()) return e;
      }
      if (jobs > 0) {
        hipLaunchKernelGGL((gdp_select_backward_kernel<UT, DT, P>), dim3((unsigned)jobs), dim3(64 * (P / OWN)), 0,
                           stream, a, g, b);
        if (hipError_t e = hipGetLastError()) return e;
      }
      if (a.T > 0) {
        const int64_t want = ((int64_t)a.T * a.G * 2 * P + 1023) / 1024;
        hipLaunchKernelGGL((gdp_select_rows_kernel<UT, DT>), dim3((unsigned)(want < 4096 ? want : 4096)), dim3(256), 0,
                           stream, a, g, b, P);
        if (hipError_t e = hipGetLastError()) return e;
      }
      SumArgs sums{b.sums, (int64_t)(P + 2) * a.D, (int)g.numbers, a.D, P, a.S, a.dA, a.dskip, a.dbias};
      return launch_sums(sums, stream);
    });
  });
}

}  // namespace gdp
