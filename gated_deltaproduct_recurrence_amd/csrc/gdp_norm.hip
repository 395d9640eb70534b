// gdp_norm.hip -- gfx950 kernels of the group norm with an activation over the
// channels of each (token, group), and of its gradients.
//
//     n = (x - mean) rstd w + b,   y = act(n)  or  n act(z)
//     q = dn w:   dx = rstd (q - mean(q) - xhat mean(q xhat)),   xhat = (x - mean) rstd
//     dw = sum dn xhat,  db = sum dn,   dn = d_y act'(n)  or  d_y act(z),
//     dz = d_y n act'(z)
//
// Both directions are streams: each input is read once, each output written once.
// A team of LPG lanes (a power of two) holds one (token, group) in registers, E
// pieces of VEC neighbouring channels per lane, so that the two passes of the
// statistics (mean, then the squares of x - mean: no cancellation under a large
// mean) and the gradient's sums take no second read.  A workgroup holds S teams;
// the teams of the whole grid step through the tokens together, by a number of
// (token, group) pairs that is a multiple of G: a team keeps its group, hence its
// weights and, in the backward pass, its partial sums of dw and db, in registers.
// The raw values of a team's next token are loaded before the current one is
// computed.
//
// What bounds it, measured on MI355X (a 1 GiB copy reaches 5.0 TB/s): the memory.
// 65536 x 32 x 128 bfloat16 with a gate: 266 us, 6.0 TB/s; the gradients of 32768 x 16
// x 128: 118 us, 5.7 TB/s.  Operands that fit the memory-side cache and are left to it
// stay below that: 8195 x 8 x 512 float16 without a gate 34 us, 3.9 TB/s (dropping the
// reductions or the sigmoid changes it by 1 to 2 us).
//   Grid: 1024 workgroups forward and 768 backward, half and three quarters of what a
// round holds (8 and 4 per compute unit at 54 and 127 registers).  512, 1024 and 2048
// forward: 276, 270 and 314 us on the first shape; 512, 768 and 1024 backward: the
// training step of the second 191, 194 and 206 us, 4099 x 5 x 100 float32 29 and 27 us.
// Two tokens per step and team cost 20%.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp.h"
#include "gdp_layer.h"
#include "gdp_layer_common.h"

namespace gdp {
namespace {

constexpr int MAX_VALUES = 16;  // values a lane holds of one group

// E pieces of one (token, group)
template <typename T, int VEC, int E> struct Values {
  Pack<T, VEC> p[E];
  template <bool STREAMED> __device__ __forceinline__ void load(const T *row, int lane, int lpg, int V) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int v = (e * lpg + lane) * VEC;
      p[e] = {};
      if (v < V) p[e] = STREAMED ? load_streamed<T, VEC>(row + v) : *(const Pack<T, VEC> *)(row + v);
    }
  }
};

template <bool STREAMED, typename T, int VEC, int E>
__device__ __forceinline__ void store_values(T *row, const float (&y)[E][VEC], int lane, int lpg, int V) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int v = (e * lpg + lane) * VEC;
    Pack<T, VEC> s;
#pragma unroll
    for (int c = 0; c < VEC; ++c) s.v[c] = (T)y[e][c];
    if (v < V) {
      if (STREAMED) store_streamed<T, VEC>(row + v, s);
      else *(Pack<T, VEC> *)(row + v) = s;
    }
  }
}

// a group's weights or biases (or `other` without any)
template <typename T, int VEC, int E>
__device__ __forceinline__ void load_params(float (&w)[E][VEC], const void *p, int type, int64_t at, float other,
                                            int lane, int lpg, int V) {
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const int v = (e * lpg + lane) * VEC + c;
      w[e][c] = !p || v >= V ? other : (type == EL_F32 ? ((const float *)p)[at + v] : (float)((const T *)p)[at + v]);
    }
}

// xhat of a group in place of its values; returns rstd.  Lanes past V hold zeros.
template <typename T, int VEC, int E, int WIDE>
__device__ __forceinline__ float normalise(float (&xhat)[E][VEC], const Values<T, VEC, E> &x, const NormArgs &a,
                                           Team<WIDE> &team, float inv_v) {
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int c = 0; c < VEC; ++c) xhat[e][c] = (float)x.p[e].v[c];
  if (a.center) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) s += xhat[e][c];
    const float mean = team.sum(s) * inv_v;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) xhat[e][c] = (e * team.lpg + team.lane) * VEC < a.V ? xhat[e][c] - mean : 0.f;
  }
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int c = 0; c < VEC; ++c) ss = fmaf(xhat[e][c], xhat[e][c], ss);
  const float rstd = __builtin_amdgcn_rsqf(fmaf(team.sum(ss), inv_v, a.eps));
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int c = 0; c < VEC; ++c) xhat[e][c] *= rstd;
  return rstd;
}

// The team's place: its group and first token.
struct Place { int q, g; int64_t t, t_block, step; };  // step >= T where a team has one pair
__device__ __forceinline__ Place place_of(const NormArgs &a, int teams, int team) {
  Place p;
  p.q = (int)blockIdx.x * teams + team;
  p.g = p.q % a.G;
  p.t = p.q / a.G;
  p.t_block = (int)blockIdx.x * teams / a.G;  // the block's earliest token: a loop bound its waves share
  p.step = (int64_t)gridDim.x * teams / a.G;
  return p;
}

template <typename T, int VEC, int E, int WIDE, bool STREAMED>
__global__ void __launch_bounds__(WIDE == 0 ? 256 : 512 * WIDE) gdp_norm_kernel(NormArgs a, int lpg) {
  __shared__ float slots[WIDE ? 2 : 1][16];
  const int tid = threadIdx.x;
  Team<WIDE> team{lpg, tid & (lpg - 1), (tid & ~(lpg - 1)) >> 6, slots};
  const Place at = place_of(a, (int)blockDim.x / lpg, tid / lpg);
  const float inv_v = 1.f / (float)a.V;
  const T *x = (const T *)a.x + at.g * a.x_sh, *z = (const T *)a.z + at.g * a.z_sh;
  T *y = (T *)a.y + at.g * a.y_sh;
  float w[E][VEC], b[E][VEC];
  load_params<T, VEC, E>(w, a.w, a.w_type, at.g * a.w_sh, 1.f, team.lane, lpg, a.V);
  load_params<T, VEC, E>(b, a.b, a.w_type, at.g * a.w_sh, 0.f, team.lane, lpg, a.V);
  Values<T, VEC, E> xv{}, zv{}, xn{}, zn{};
  auto fetch = [&](int64_t t) {
    if (t < a.T) {
      xn.template load<STREAMED>(x + t * a.x_st, team.lane, lpg, a.V);
      if (a.z) zn.template load<STREAMED>(z + t * a.z_st, team.lane, lpg, a.V);
    }
  };
  int64_t t = at.t;
  fetch(t);
  for (int64_t tb = at.t_block; tb < a.T; tb += at.step, t += at.step) {
    xv = xn;
    zv = zn;
    fetch(t + at.step);
    float n[E][VEC];
    normalise<T, VEC, E, WIDE>(n, xv, a, team, inv_v);
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) n[e][c] = fmaf(n[e][c], w[e][c], b[e][c]);
    if (a.z) {
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const float v = (float)zv.p[e].v[c];
          n[e][c] *= a.act == GDP_ACT_NONE ? v : (a.act == GDP_ACT_SILU ? v * sigmoid_of(v) : sigmoid_of(v));
        }
    } else if (a.act != GDP_ACT_NONE) {
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const float s = sigmoid_of(n[e][c]);
          n[e][c] = a.act == GDP_ACT_SILU ? n[e][c] * s : s;
        }
    }
    if (t < a.T) store_values<STREAMED, T, VEC, E>(y + t * a.y_st, n, team.lane, lpg, a.V);
  }
}

// The gradients; partial sums of dw and db to the workspace: one row [2][V] per
// workgroup when the groups share their weights (the teams' sums added in LDS),
// else one per team.
template <typename T, int VEC, int E, int WIDE, bool STREAMED>
__global__ void __launch_bounds__(WIDE == 0 ? 256 : 512 * WIDE) gdp_norm_backward_kernel(NormArgs a, int lpg) {
  __shared__ float slots[WIDE ? 2 : 1][16];
  __shared__ float part[WIDE ? 1 : 256 * MAX_VALUES];
  const int tid = threadIdx.x, teams = (int)blockDim.x / lpg;
  Team<WIDE> team{lpg, tid & (lpg - 1), (tid & ~(lpg - 1)) >> 6, slots};
  const Place at = place_of(a, teams, tid / lpg);
  const float inv_v = 1.f / (float)a.V;
  const T *x = (const T *)a.x + at.g * a.x_sh, *z = (const T *)a.z + at.g * a.z_sh,
          *dy = (const T *)a.dy + at.g * a.dy_sh;
  T *dx = (T *)a.dx + at.g * a.dx_sh, *dz = (T *)a.dz + at.g * a.dz_sh;
  float w[E][VEC], b[E][VEC], dw[E][VEC] = {}, db[E][VEC] = {};
  load_params<T, VEC, E>(w, a.w, a.w_type, at.g * a.w_sh, 1.f, team.lane, lpg, a.V);
  load_params<T, VEC, E>(b, a.b, a.w_type, at.g * a.w_sh, 0.f, team.lane, lpg, a.V);
  Values<T, VEC, E> xv{}, zv{}, dv{}, xn{}, zn{}, dn_{};
  auto fetch = [&](int64_t t) {
    if (t < a.T) {
      xn.template load<STREAMED>(x + t * a.x_st, team.lane, lpg, a.V);
      dn_.template load<STREAMED>(dy + t * a.dy_st, team.lane, lpg, a.V);
      if (a.z) zn.template load<STREAMED>(z + t * a.z_st, team.lane, lpg, a.V);
    }
  };
  int64_t t = at.t;
  fetch(t);
  for (int64_t tb = at.t_block; tb < a.T; tb += at.step, t += at.step) {
    xv = xn;
    zv = zn;
    dv = dn_;
    fetch(t + at.step);
    float xhat[E][VEC], dn[E][VEC], g[E][VEC];  // g: dz
    const float rstd = normalise<T, VEC, E, WIDE>(xhat, xv, a, team, inv_v);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        const float n = fmaf(xhat[e][c], w[e][c], b[e][c]), d = (float)dv.p[e].v[c];
        const float v = a.z ? (float)zv.p[e].v[c] : n;
        float f = v, df = 1.f;
        if (a.act != GDP_ACT_NONE) {
          const float s = sigmoid_of(v);
          if (a.act == GDP_ACT_SILU) {
            f = v * s;
            df = fmaf(f, 1.f - s, s);  // s (1 + v (1 - s))
          } else {
            f = s;
            df = s * (1.f - s);
          }
        }
        dn[e][c] = d * (a.z ? f : df);
        g[e][c] = d * n * df;
        s1 = fmaf(dn[e][c], w[e][c], s1);
        s2 = fmaf(dn[e][c] * w[e][c], xhat[e][c], s2);
      }
    s1 = a.center ? team.sum(s1) * inv_v : 0.f;
    s2 = team.sum(s2) * inv_v;
    if (t < a.T) {
      if (a.z) store_values<STREAMED, T, VEC, E>(dz + t * a.dz_st, g, team.lane, lpg, a.V);
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          dw[e][c] = fmaf(dn[e][c], xhat[e][c], dw[e][c]);
          db[e][c] += dn[e][c];
          g[e][c] = (dn[e][c] * w[e][c] - s1 - xhat[e][c] * s2) * rstd;
        }
      store_values<STREAMED, T, VEC, E>(dx + t * a.dx_st, g, team.lane, lpg, a.V);
    }
  }
  if (!a.dw && !a.db) return;
  const bool fold = !WIDE && a.w_sh == 0 && teams > 1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!(k == 0 ? a.dw : a.db)) continue;
    float *row = a.ws + ((int64_t)(fold ? (int)blockIdx.x : at.q) * 2 + k) * a.V;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        const int v = (e * lpg + team.lane) * VEC + c;
        const float s = k == 0 ? dw[e][c] : db[e][c];
        if (v < a.V) {
          if (fold) part[(tid / lpg) * a.V + v] = s;
          else row[v] = s;
        }
      }
    if (fold) {
      __syncthreads();
      for (int v = tid; v < a.V; v += 256) {
        float s = 0.f;
        for (int i = 0; i < teams; ++i) s += part[i * a.V + v];
        row[v] = s;
      }
      __syncthreads();
    }
  }
}

// dw (blockIdx.z = 0) and db from the partial rows of a group (row r: r * stride +
// blockIdx.y): 16 channels per workgroup, the rows dealt over 64 lane groups, eight
// loads ahead.  A fixed order: the result does not depend on timing.  With 64
// channels and 16 lane groups per workgroup the sums of 1024 rows of 128 channels
// took 23 us, waiting for 64 loads one after another.
__global__ void __launch_bounds__(1024) gdp_norm_weight_kernel(NormArgs a, int rows, int stride) {
  __shared__ float red[64][17];
  const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int v = (int)blockIdx.x * 16 + c;
  float *out = blockIdx.z == 0 ? a.dw : a.db;
  if (!out) return;
  float s = 0.f;
  if (v < a.V) {
    const float *p = a.ws + ((int64_t)blockIdx.y * 2 + blockIdx.z) * a.V + v;
    const int64_t step = (int64_t)stride * 2 * a.V;
    int r = part;
    for (; r + 64 * 7 < rows; r += 64 * 8) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[(r + 64 * i) * step];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[i];
    }
    for (; r < rows; r += 64) s += p[r * step];
  }
  red[part][c] = s;
  __syncthreads();
  for (int n = 32; n > 0; n >>= 1) {
    if (part < n) red[part][c] += red[part + n][c];
    __syncthreads();
  }
  if (part == 0 && v < a.V) out[(int64_t)blockIdx.y * a.V + v] = red[0][c];
}

// How the groups are laid over lanes.  E pieces of VEC channels per lane: one while
// a wave holds the group, then up to MAX_VALUES values per lane, then more waves.
struct Plan { int vec, pieces, lpg, threads, teams; };
Plan plan_of(int64_t V, int vec) {
  Plan p;
  p.vec = vec;
  const int64_t chunks = (V + vec - 1) / vec;
  p.pieces = 1;
  while ((chunks + p.pieces - 1) / p.pieces > 64 && p.pieces * vec < MAX_VALUES) p.pieces *= vec == 1 ? 4 : 2;
  const int64_t lanes = (chunks + p.pieces - 1) / p.pieces;
  p.lpg = 1;
  while (p.lpg < lanes) p.lpg *= 2;
  p.threads = p.lpg > 256 ? p.lpg : 256;
  p.teams = p.threads / p.lpg;
  return p;
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// Workgroups: one pair per team while that gives at most `most` / 2, then down to
// `per_team` pairs per team, at most `most`.  Teams that take more than one pair come
// in multiples that keep a team's group; no more workgroups than there are pairs for,
// however few tokens an odd number of groups has.
int64_t grid_of(const Plan &p, int64_t T, int G, int64_t per_team, int64_t most) {
  const int64_t want = (T * G + p.teams - 1) / p.teams, unit = G / gcd(G, p.teams);
  int64_t n = want;
  if (want > most / 2) {
    n = want / per_team;
    n = n < most / 2 ? most / 2 : (n > most ? most : n);
    n = (n + unit - 1) / unit * unit;
  }
  return n < want ? n : want;
}
constexpr int64_t FORWARD_GRID = 1024, BACKWARD_GRID = 768;

template <typename F> hipError_t by_type(int xt, F f) {
  if (xt == EL_F32) return f((float)0);
  return xt == EL_BF16 ? f((bf16)0) : f((_Float16)0);
}

// WIDE: 0 while a wave holds a group, 1 up to 512 lanes, 2 up to 1024.  Lanes of the
// latter have half the registers: the gradients of groups of more than 8192 channels
// spill 164 to 305 of them, and so do, less, the forms for operands that no vector width
// aligns (30 to 34 forward past 8192, 10 to 13 in the gradients past 1024).
template <int VEC, int E, int WIDE> struct Shape { static constexpr int vec = VEC, pieces = E, wide = WIDE; };

// calls f with the compile-time shape of a plan
template <int VEC, int E, typename F> hipError_t by_width(const Plan &p, F f) {
  if (p.lpg <= 64) return f(Shape<VEC, E, 0>());
  return p.lpg <= 512 ? f(Shape<VEC, E, 1>()) : f(Shape<VEC, E, 2>());
}
template <typename T, typename F> hipError_t by_plan(const Plan &p, F f) {
  if constexpr (sizeof(T) == 2) {
    if (p.vec == 8) return p.pieces == 1 ? f(Shape<8, 1, 0>()) : by_width<8, 2>(p, f);
  }
  if (p.vec == 4) {
    if (p.pieces == 1) return f(Shape<4, 1, 0>());
    return p.pieces == 2 ? f(Shape<4, 2, 0>()) : by_width<4, 4>(p, f);
  }
  if (p.pieces == 1) return f(Shape<1, 1, 0>());
  return p.pieces == 4 ? f(Shape<1, 4, 0>()) : by_width<1, 16>(p, f);
}

// whether pieces of `vec` elements of es bytes are aligned everywhere in a tensor
bool fits(const void *p, int64_t st, int64_t sh, int vec, int es) {
  return !p || (((uintptr_t)p & (vec * es - 1)) == 0 && st % vec == 0 && sh % vec == 0);
}
int vec_of(const NormArgs &a, int es, bool backward) {
  for (int vec = es == 2 ? 8 : 4; vec > 1; vec = vec == 8 ? 4 : 1) {
    bool ok = a.V % vec == 0 && fits(a.x, a.x_st, a.x_sh, vec, es) && fits(a.z, a.z_st, a.z_sh, vec, es);
    if (backward)
      ok = ok && fits(a.dy, a.dy_st, a.dy_sh, vec, es) && fits(a.dx, a.dx_st, a.dx_sh, vec, es) &&
           fits(a.dz, a.dz_st, a.dz_sh, vec, es);
    else
      ok = ok && fits(a.y, a.y_st, a.y_sh, vec, es);
    if (ok) return vec;
  }
  return 1;
}

}  // namespace

size_t norm_backward_bytes(int64_t T, int64_t G, int64_t V) {
  int64_t most = 0;  // of the plans that the alignment of a call's tensors can choose
  for (int vec : {8, 4, 1}) {
    if (V % vec) continue;
    const Plan p = plan_of(V, vec);
    const int64_t rows = grid_of(p, T, (int)G, 8, BACKWARD_GRID) * p.teams;
    most = rows > most ? rows : most;
  }
  return (size_t)most * V * 8;
}

hipError_t launch_norm(const NormArgs &a, int xt, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  return by_type(xt, [&](auto x) {
    using T = decltype(x);
    const bool streamed = a.T * a.G * a.V * (int64_t)sizeof(T) * (a.z ? 3 : 2) > STREAM_BYTES;
    const Plan p = plan_of(a.V, vec_of(a, sizeof(T), false));
    const int64_t blocks = grid_of(p, a.T, a.G, 1, FORWARD_GRID);
    return by_plan<T>(p, [&](auto s) {
      using S = decltype(s);
      auto *kernel = gdp_norm_kernel<T, S::vec, S::pieces, S::wide, false>;
      // only whole 16-byte pieces: the narrower forms are bound elsewhere
      if constexpr (S::vec * sizeof(T) == 16)
        if (streamed) kernel = gdp_norm_kernel<T, S::vec, S::pieces, S::wide, true>;
      hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(p.threads), 0, stream, a, p.lpg);
      return hipGetLastError();
    });
  });
}

hipError_t launch_norm_backward(const NormArgs &a, int xt, hipStream_t stream) {
  return by_type(xt, [&](auto x) {
    using T = decltype(x);
    const bool streamed = a.T * a.G * a.V * (int64_t)sizeof(T) * (a.z ? 5 : 3) > STREAM_BYTES;
    const Plan p = plan_of(a.V, vec_of(a, sizeof(T), true));
    const int64_t blocks = a.T ? grid_of(p, a.T, a.G, 8, BACKWARD_GRID) : 0;
    if (blocks) {
      const hipError_t e = by_plan<T>(p, [&](auto s) {
        using S = decltype(s);
        auto *kernel = gdp_norm_backward_kernel<T, S::vec, S::pieces, S::wide, false>;
        if constexpr (S::vec * sizeof(T) == 16)
          if (streamed) kernel = gdp_norm_backward_kernel<T, S::vec, S::pieces, S::wide, true>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(p.threads), 0, stream, a, p.lpg);
        return hipGetLastError();
      });
      if (e != hipSuccess) return e;
    }
    if (!a.dw && !a.db) return hipSuccess;
    const bool shared = a.w_sh == 0, fold = shared && p.lpg <= 64 && p.teams > 1;
    // the teams that had a pair: all, or (one pair each) the first T G
    const int64_t teams = blocks * p.teams < a.T * a.G ? blocks * p.teams : a.T * a.G;
    const int64_t rows = fold ? blocks : teams;
    const dim3 grid((unsigned)((a.V + 15) / 16), shared ? 1u : (unsigned)a.G, 2);
    hipLaunchKernelGGL(gdp_norm_weight_kernel, grid, dim3(1024), 0, stream, a, (int)(shared ? rows : rows / a.G),
                       shared ? 1 : a.G);
    return hipGetLastError();
  });
}

}  // namespace gdp
