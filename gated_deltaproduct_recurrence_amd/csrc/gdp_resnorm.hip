// gdp_resnorm.hip -- gfx950 kernels of the norms before and after a block, fused with
// the block's gate, the residual scale and the residual sum: from the residual
// stream x and a block's output y, per token over all D channels,
//     p = yhat w_post,  yhat = y rstd(y)  (or y without the post norm),
//     r = x + s f(z) p,                    f the gate's activation (1 without a gate)
//     n = r rstd(r) w_pre,                 the next block's input
// with rstd(v) = 1 / sqrt(mean(v^2) + eps), and of its gradients: with q = d_n w_pre,
// rhat = r rstd(r),
//     e = d_r + rstd(r) (q - rhat mean(q rhat)),   dx = e,
//     dz = s e p f'(z),  dp = s e f(z),  v = dp w_post,
//     dy = rstd(y) (v - yhat mean(v yhat))  (or v),
//     dw_post = sum dp yhat,  dw_pre = sum d_n rhat.
//
// A stream: every operand is read once and every result written once; r is formed
// again in the gradients from x, y and z (in place of r, which is as large as x), so
// its rounding in the stored stream does not enter them.  A team of LPG lanes (a power
// of two) holds a token in registers, E pieces of VEC channels per lane; the teams of
// the whole grid step through the tokens together, and the raw values of a team's
// next token are loaded before the current one is computed.
//
// What bounds it, measured on MI355X (a 1 GiB copy reaches 5.1 TB/s): the memory.
// 65536 x 4096 bfloat16 without a gate: 374 us, 5.7 TB/s; 8195 x 4096 float16 with a gate
// and a float32 stream: 89 us, 5.3 TB/s, and its gradients 174 us, 4.2 TB/s, at 241 registers
// and two waves per SIMD with four sums over the token between barriers.
//   Loads and stores past the caches where the operands exceed the memory-side one: 392 us on
// the first shape without, where this takes 372.  Grid: 1024 workgroups forward, 512 in the
// gradients; 768, 1536, 2048 and 4096 forward: 421, 440, 378 and 378 us, half and twice the
// workgroups of the gradients in the training step 369 and 299 us instead of 271.
//   Gradients of more than 8192 channels keep part of a token outside the registers and are
// slow: 4096 tokens of 8192, 12288 and 16384 channels, bfloat16 with a gate, take 194, 930 and
// 1024 us (2.8, 0.9 and 1.0 TB/s).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp.h"
#include "gdp_block.h"
#include "gdp_block_common.h"

namespace gdp {
namespace {

constexpr int MAX_VALUES = 16;  // values a lane holds of one token

template <typename T, int VEC, int E> struct Row {
  Piece<T, VEC> p[E];
  template <bool STREAMED> __device__ __forceinline__ void load(const T *row, int lane, int lpg, int D) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = (e * lpg + lane) * VEC;
      p[e] = {};
      if (ch < D) p[e] = load_piece<T, VEC, STREAMED>(row, ch, D);
    }
  }
  __device__ __forceinline__ float at(int e, int c) const { return (float)p[e].v[c]; }
};

template <bool STREAMED, typename T, int VEC, int E>
__device__ __forceinline__ void store_row(T *row, const float (&x)[E][VEC], int lane, int lpg, int D) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int ch = (e * lpg + lane) * VEC;
    if (ch < D) store_floats<T, VEC, STREAMED>(row, ch, D, x[e]);
  }
}

template <typename P, int VEC, int E>
__device__ __forceinline__ void load_pieces(float (&w)[E][VEC], const P *p, int lane, int lpg, int D) {
  Row<P, VEC, E> row;
  row.template load<false>(p, lane, lpg, D);
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int c = 0; c < VEC; ++c) w[e][c] = row.at(e, c);
}
template <typename T, int VEC, int E>
__device__ __forceinline__ void load_weights(float (&w)[E][VEC], const void *p, int type, int lane, int lpg, int D) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) w[e][c] = 1.f;
  } else if (type == EL_F32) {
    load_pieces<float, VEC, E>(w, (const float *)p, lane, lpg, D);
  } else {
    load_pieces<T, VEC, E>(w, (const T *)p, lane, lpg, D);
  }
}

template <int VEC, int E, int WIDE>
__device__ __forceinline__ float rstd_of(const float (&v)[E][VEC], Team<WIDE> &team, float inv_d, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int c = 0; c < VEC; ++c) ss = fmaf(v[e][c], v[e][c], ss);
  return __builtin_amdgcn_rsqf(fmaf(team.sum(ss), inv_d, eps));
}

// T: y, the gate and n; X: the residual stream
template <typename T, typename X, int VEC, int E, int WIDE, bool STREAMED>
__global__ void __launch_bounds__(WIDE == 0 ? 256 : 512 * WIDE) gdp_resnorm_kernel(ResNormArgs a, int lpg) {
  __shared__ float slots[WIDE ? 2 : 1][16];
  const int tid = threadIdx.x, teams = (int)blockDim.x / lpg;
  Team<WIDE> team{lpg, tid & (lpg - 1), (tid & ~(lpg - 1)) >> 6, slots};
  const int64_t step = (int64_t)gridDim.x * teams;
  const float inv_d = 1.f / (float)a.D;
  float wa[E][VEC], wb[E][VEC];
  load_weights<T, VEC, E>(wa, a.w_post, a.w_type, team.lane, lpg, a.D);
  load_weights<T, VEC, E>(wb, a.w_pre, a.w_type, team.lane, lpg, a.D);
  Row<T, VEC, E> yv{}, zv{}, yn{}, zn{};
  Row<X, VEC, E> xv{}, xn{};
  auto fetch = [&](int64_t t) {
    if (t < a.T) {
      yn.template load<STREAMED>((const T *)a.y + t * a.y_st, team.lane, lpg, a.D);
      xn.template load<STREAMED>((const X *)a.x + t * a.x_st, team.lane, lpg, a.D);
      if (a.z) zn.template load<STREAMED>((const T *)a.z + t * a.z_st, team.lane, lpg, a.D);
    }
  };
  constexpr bool AHEAD = WIDE < 2;  // lanes of the widest teams have half the registers
  int64_t t = (int64_t)blockIdx.x * teams + tid / lpg;
  if (AHEAD) fetch(t);
  // (the loop's bound is the block's: its waves meet at the sums' barriers)
  for (int64_t tb = (int64_t)blockIdx.x * teams; tb < a.T; tb += step, t += step) {
    if (!AHEAD) fetch(t);
    yv = yn;
    zv = zn;
    xv = xn;
    if (AHEAD) fetch(t + step);
    float v[E][VEC];
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) v[e][c] = yv.at(e, c);
    const float ry = (a.post ? rstd_of<VEC, E, WIDE>(v, team, inv_d, a.eps) : 1.f) * a.scale;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        float p = v[e][c] * ry * wa[e][c];
        if (a.z) p *= act_of(a.act, zv.at(e, c));
        v[e][c] = xv.at(e, c) + p;
      }
    if (t < a.T) store_row<STREAMED, X, VEC, E>((X *)a.r + t * a.r_st, v, team.lane, lpg, a.D);
    if (a.pre) {
      // lanes behind the row's end hold zeros: x and y are 0 there
      const float rr = rstd_of<VEC, E, WIDE>(v, team, inv_d, a.eps);
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) v[e][c] *= rr * wb[e][c];
      if (t < a.T) store_row<STREAMED, T, VEC, E>((T *)a.n + t * a.n_st, v, team.lane, lpg, a.D);
    }
  }
}

// The gradients; partial sums of the weights' gradients to the workspace, one row
// [2, D] per workgroup (the teams' sums added in LDS).
template <typename T, typename X, int VEC, int E, int WIDE, bool STREAMED>
__global__ void __launch_bounds__(WIDE == 0 ? 256 : 512 * WIDE) gdp_resnorm_backward_kernel(ResNormArgs a, int lpg) {
  __shared__ float slots[WIDE ? 2 : 1][16];
  __shared__ float part[WIDE ? 1 : 256 * MAX_VALUES];
  const int tid = threadIdx.x, teams = (int)blockDim.x / lpg;
  Team<WIDE> team{lpg, tid & (lpg - 1), (tid & ~(lpg - 1)) >> 6, slots};
  const int64_t step = (int64_t)gridDim.x * teams;
  const float inv_d = 1.f / (float)a.D;
  float wa[E][VEC], wb[E][VEC], dwa[E][VEC] = {}, dwb[E][VEC] = {};
  load_weights<T, VEC, E>(wa, a.w_post, a.w_type, team.lane, lpg, a.D);
  load_weights<T, VEC, E>(wb, a.w_pre, a.w_type, team.lane, lpg, a.D);
  Row<T, VEC, E> yv{}, zv{}, nv{}, yn{}, zn{}, nn{};
  Row<X, VEC, E> xv{}, rv{}, xn{}, rn{};
  // A token is loaded ahead, but the widest teams' lanes have half the registers; and in
  // float32 the output gradients are loaded with the token's first sums (70 registers
  // spill otherwise; in 16 bits, where none do, loading them late costs 2%).
  constexpr bool AHEAD = WIDE < 2, LATE = sizeof(T) == 4;
  auto fetch_outputs = [&](int64_t t) {
    if (a.pre) nn.template load<STREAMED>((const T *)a.dn + t * a.dn_st, team.lane, lpg, a.D);
    if (a.dr) rn.template load<STREAMED>((const X *)a.dr + t * a.dr_st, team.lane, lpg, a.D);
  };
  auto fetch = [&](int64_t t) {
    if (t < a.T) {
      yn.template load<STREAMED>((const T *)a.y + t * a.y_st, team.lane, lpg, a.D);
      // r is needed for its norm alone
      if (a.pre) xn.template load<STREAMED>((const X *)a.x + t * a.x_st, team.lane, lpg, a.D);
      if (a.z) zn.template load<STREAMED>((const T *)a.z + t * a.z_st, team.lane, lpg, a.D);
      if (!LATE) fetch_outputs(t);
    }
  };
  int64_t t = (int64_t)blockIdx.x * teams + tid / lpg;
  if (AHEAD) fetch(t);
  for (int64_t tb = (int64_t)blockIdx.x * teams; tb < a.T; tb += step, t += step) {
    if (!AHEAD) fetch(t);
    if (LATE && t < a.T) fetch_outputs(t);
    yv = yn;
    zv = zn;
    xv = xn;
    nv = nn;
    rv = rn;
    if (AHEAD) fetch(t + step);
    float yhat[E][VEC], e_[E][VEC];  // e_: r, then e
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) yhat[e][c] = yv.at(e, c);
    const float ry = a.post ? rstd_of<VEC, E, WIDE>(yhat, team, inv_d, a.eps) : 1.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) yhat[e][c] *= ry;
    if (a.pre) {
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          float p = yhat[e][c] * a.scale * wa[e][c];
          if (a.z) p *= act_of(a.act, zv.at(e, c));
          e_[e][c] = xv.at(e, c) + p;
        }
      const float rr = rstd_of<VEC, E, WIDE>(e_, team, inv_d, a.eps);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          e_[e][c] *= rr;
          s = fmaf(nv.at(e, c) * wb[e][c], e_[e][c], s);
        }
      s = team.sum(s) * inv_d;
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const float rhat = e_[e][c], dn = nv.at(e, c);
          if (t < a.T) dwb[e][c] = fmaf(dn, rhat, dwb[e][c]);
          e_[e][c] = fmaf(rr, fmaf(-rhat, s, dn * wb[e][c]), rv.at(e, c));
        }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) e_[e][c] = rv.at(e, c);
    }
    if (t < a.T) store_row<STREAMED, X, VEC, E>((X *)a.dx + t * a.dx_st, e_, team.lane, lpg, a.D);
    // dp in e_, then v; dz in its own
    if (a.z) {
      float dz[E][VEC];
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          float slope;
          const float f = act_of(a.act, zv.at(e, c), &slope), d = e_[e][c] * a.scale;
          dz[e][c] = d * yhat[e][c] * wa[e][c] * slope;
          e_[e][c] = d * f;
        }
      if (t < a.T) store_row<STREAMED, T, VEC, E>((T *)a.dz + t * a.dz_st, dz, team.lane, lpg, a.D);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) e_[e][c] *= a.scale;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        if (t < a.T) dwa[e][c] = fmaf(e_[e][c], yhat[e][c], dwa[e][c]);
        e_[e][c] *= wa[e][c];
        s = fmaf(e_[e][c], yhat[e][c], s);
      }
    if (a.post) {
      s = team.sum(s) * inv_d;
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int c = 0; c < VEC; ++c) e_[e][c] = ry * fmaf(-yhat[e][c], s, e_[e][c]);
    }
    if (t < a.T) store_row<STREAMED, T, VEC, E>((T *)a.dy + t * a.dy_st, e_, team.lane, lpg, a.D);
  }
  if (!a.dw_post && !a.dw_pre) return;
  const bool fold = !WIDE && teams > 1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!(k == 0 ? a.dw_post : a.dw_pre)) continue;
    float *row = a.ws + ((WIDE ? (int64_t)blockIdx.x * teams + tid / lpg : (int64_t)blockIdx.x) * 2 + k) * a.D;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        const int ch = (e * lpg + team.lane) * VEC + c;
        const float s = k == 0 ? dwa[e][c] : dwb[e][c];
        if (ch < a.D) {
          if (fold) part[(tid / lpg) * a.D + ch] = s;
          else row[ch] = s;
        }
      }
    if (fold) {
      __syncthreads();
      for (int ch = tid; ch < a.D; ch += 256) {
        float s = 0.f;
        for (int i = 0; i < teams; ++i) s += part[i * a.D + ch];
        row[ch] = s;
      }
      __syncthreads();
    }
  }
}

// How a token is laid over lanes: one piece per lane while a wave holds the token, then
// up to MAX_VALUES values per lane, then more waves.
struct Plan { int vec, pieces, lpg, threads, teams; };
Plan plan_of(int64_t D, int vec) {
  Plan p;
  p.vec = vec;
  const int64_t chunks = (D + vec - 1) / vec;
  p.pieces = 1;
  while ((chunks + p.pieces - 1) / p.pieces > 64 && p.pieces * vec < MAX_VALUES) p.pieces *= 2;
  const int64_t lanes = (chunks + p.pieces - 1) / p.pieces;
  p.lpg = 1;
  while (p.lpg < lanes) p.lpg *= 2;
  p.threads = p.lpg > 256 ? p.lpg : 256;
  p.teams = p.threads / p.lpg;
  return p;
}

constexpr int64_t FORWARD_GRID = 1024, BACKWARD_GRID = 512;
int64_t grid_of(const Plan &p, int64_t T, int64_t most) {
  const int64_t want = (T + p.teams - 1) / p.teams;
  return want < most ? want : most;
}

template <int VEC, int E, int WIDE> struct Shape { static constexpr int vec = VEC, pieces = E, wide = WIDE; };
template <int VEC, int E, typename F> hipError_t by_width(const Plan &p, F f) {
  if (p.lpg <= 64) return f(Shape<VEC, E, 0>());
  return p.lpg <= 512 ? f(Shape<VEC, E, 1>()) : f(Shape<VEC, E, 2>());
}
template <typename T> constexpr int vec_of() { return sizeof(T) == 2 ? 8 : 4; }
// calls f with the compile-time shape of a plan
template <typename T, typename F> hipError_t by_plan(const Plan &p, F f) {
  constexpr int VEC = vec_of<T>();
  if (p.pieces == 1) return f(Shape<VEC, 1, 0>());
  if constexpr (VEC == 8) {
    return by_width<8, 2>(p, f);
  } else {
    return p.pieces == 2 ? f(Shape<4, 2, 0>()) : by_width<4, 4>(p, f);
  }
}
template <typename F> hipError_t by_types(int yt, int xt, F f) {
  if (yt == EL_F32) return f((float)0, (float)0);
  if (yt == EL_BF16) return xt == EL_F32 ? f((bf16)0, (float)0) : f((bf16)0, (bf16)0);
  return xt == EL_F32 ? f((_Float16)0, (float)0) : f((_Float16)0, (_Float16)0);
}

}  // namespace

size_t resnorm_backward_bytes(int64_t T, int64_t D) {
  int64_t most = 0;  // of the two types' plans
  for (int vec : {8, 4}) {
    const Plan p = plan_of(D, vec);
    const int64_t rows = grid_of(p, T, BACKWARD_GRID) * (p.lpg > 64 ? p.teams : 1);
    most = rows > most ? rows : most;
  }
  return (size_t)most * D * 8;
}

hipError_t launch_resnorm(const ResNormArgs &a, int yt, int xt, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  return by_types(yt, xt, [&](auto y, auto x) {
    using T = decltype(y);
    using X = decltype(x);
    const Plan p = plan_of(a.D, vec_of<T>());
    const bool streamed = a.T * a.D * (int64_t)(2 * sizeof(X) + (1 + (a.z != nullptr) + a.pre) * sizeof(T)) > STREAM_BYTES;
    return by_plan<T>(p, [&](auto s) {
      using S = decltype(s);
      auto *kernel = streamed ? gdp_resnorm_kernel<T, X, S::vec, S::pieces, S::wide, true>
                              : gdp_resnorm_kernel<T, X, S::vec, S::pieces, S::wide, false>;
      hipLaunchKernelGGL(kernel, dim3((unsigned)grid_of(p, a.T, FORWARD_GRID)), dim3(p.threads), 0, stream, a, p.lpg);
      return hipGetLastError();
    });
  });
}

hipError_t launch_resnorm_backward(const ResNormArgs &a, int yt, int xt, hipStream_t stream) {
  return by_types(yt, xt, [&](auto y, auto x) {
    using T = decltype(y);
    using X = decltype(x);
    const Plan p = plan_of(a.D, vec_of<T>());
    const bool streamed =
        a.T * a.D * (int64_t)(3 * sizeof(X) + (2 + 2 * (a.z != nullptr) + a.pre) * sizeof(T)) > STREAM_BYTES;
    const int64_t blocks = grid_of(p, a.T, BACKWARD_GRID);
    if (blocks) {
      const hipError_t e = by_plan<T>(p, [&](auto s) {
        using S = decltype(s);
        auto *kernel = streamed ? gdp_resnorm_backward_kernel<T, X, S::vec, S::pieces, S::wide, true>
                                : gdp_resnorm_backward_kernel<T, X, S::vec, S::pieces, S::wide, false>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(p.threads), 0, stream, a, p.lpg);
        return hipGetLastError();
      });
      if (e != hipSuccess) return e;
    }
    SumArgs s{a.ws, (int64_t)2 * a.D, (int)(blocks * (p.lpg > 64 ? p.teams : 1)), a.D, 0, 0, nullptr, a.dw_post,
              a.dw_pre};
    return launch_sums(s, stream);
  });
}

}  // namespace gdp
