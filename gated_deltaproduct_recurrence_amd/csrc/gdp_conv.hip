// gdp_conv.hip -- gfx950 kernels of the short causal convolution over packed
// sequences, channel by channel:
//     v_t = b + sum_j w_j x_{t-W+1+j},   y_t = act(v_t),
// of its single-token step, and of its gradients:
//     dv_t = d_y_t act'(v_t),  dx_t = sum_i w_{W-1-i} dv_{t+i},
//     dw_j = sum_t dv_t x_{t-W+1+j},  db = sum_t dv_t.
// The W - 1 rows before a sequence's first are its initial state (or zeros), its last
// W - 1 rows the final state; the gradients treat both as rows of the stream.
//
// A stream: x read once, y written once, 2 W + 4 operations per element.  A wave takes
// one chunk of a sequence (gdp_block_common.h) and a block of channels, 16 bytes of a row per
// lane, and walks down the rows with the last W - 1 of them in registers, as floats;
// ROWS rows ahead are in flight.  The W - 1 rows before the chunk are read a second
// time, out of the caches.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp.h"
#include "gdp_block.h"
#include "gdp_block_common.h"

namespace gdp {
namespace {

constexpr int WAVES = 4, ROWS = 4;

// Row t >= first - (W - 1) of a chunk's sequence: those before its first lie in the initial state.
template <typename T, int W, int VEC>
__device__ __forceinline__ Piece<T, VEC> row_before(const ConvArgs &a, const Chunk &k, int64_t t, int ch) {
  if (t >= k.first) return load_piece<T, VEC>((const T *)a.x + t * a.x_st, ch, a.D);
  if (a.s0) return load_piece<T, VEC>((const T *)a.s0 + ((int64_t)k.seq * (W - 1) + (t - k.first + W - 1)) * a.D, ch, a.D);
  Piece<T, VEC> p;
#pragma unroll
  for (int c = 0; c < VEC; ++c) p.v[c] = (T)0.f;
  return p;
}

template <typename T, int W, int VEC>
__device__ __forceinline__ void load_taps(float (&w)[W][VEC], float (&b)[VEC], const ConvArgs &a, int ch) {
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    const int d = min(ch + c, a.D - 1);
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][c] = param_at<T>(a.w, a.w_type, (int64_t)d * W + j);
    b[c] = a.b ? param_at<T>(a.b, a.w_type, d) : 0.f;
  }
}

template <typename T, int N> __device__ __forceinline__ void to_floats(float (&x)[N], const Piece<T, N> &p) {
#pragma unroll
  for (int c = 0; c < N; ++c) x[c] = (float)p.v[c];
}

template <typename T, int W, int VEC, bool STREAMED>
__global__ void __launch_bounds__(64 * WAVES) gdp_conv_kernel(ConvArgs a, int shift, int blocks, int jobs) {
  const int id = (int)blockIdx.x * WAVES + uniform_of(threadIdx.x >> 6);
  if (id >= jobs) return;
  Chunk k;
  if (!find_chunk(&k, a.cu, a.cu_is64, a.T, a.N, shift, id / blocks)) return;
  const int ch = (id % blocks) * 64 * VEC + (threadIdx.x & 63) * VEC;
  if (ch >= a.D) return;
  if (k.begin < k.end) {
    float w[W][VEC], b[VEC], x[W - 1 + ROWS][VEC];
    Piece<T, VEC> next[ROWS] = {};
    const T *row = (const T *)a.x + (int64_t)k.begin * a.x_st;
    auto fetch = [&](int t) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (t + r < k.end) next[r] = load_piece<T, VEC, STREAMED>(row + (int64_t)(t + r - k.begin) * a.x_st, ch, a.D);
    };
    fetch(k.begin);
    load_taps<T, W, VEC>(w, b, a, ch);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) to_floats(x[j], row_before<T, W, VEC>(a, k, (int64_t)k.begin - (W - 1) + j, ch));
    T *out = (T *)a.y + (int64_t)k.begin * a.y_st;
    for (int t = k.begin; t < k.end; t += ROWS) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) to_floats(x[W - 1 + r], next[r]);
      fetch(t + ROWS);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (t + r < k.end) {
          float y[VEC];
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            float v = b[c];
#pragma unroll
            for (int j = 0; j < W; ++j) v = fmaf(w[j][c], x[r + j][c], v);
            y[c] = v;
          }
          if (a.act != GDP_ACT_NONE) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) y[c] = act_of(a.act, y[c]);
          }
          store_floats<T, VEC, STREAMED>(out, ch, a.D, y);
          out += a.y_st;
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int c = 0; c < VEC; ++c) x[j][c] = x[ROWS + j][c];
    }
  }
  // the chunk that ends its sequence writes the last W - 1 rows, as they are
  if (k.end != k.last || (!a.final_state && !a.cache)) return;
  T *state = (T *)a.final_state + (int64_t)k.seq * (W - 1) * a.D, *slot = nullptr;
  if (a.cache) {
    const int64_t s = index_at(a.slots, a.slots_is64, k.seq);
    if (s >= 0 && s < a.num_slots) slot = (T *)a.cache + s * (W - 1) * a.D;
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const Piece<T, VEC> p = row_before<T, W, VEC>(a, k, (int64_t)k.last - (W - 1) + j, ch);
    if (a.final_state) store_piece<T, VEC>(state + (int64_t)j * a.D, ch, a.D, p);
    if (slot) store_piece<T, VEC>(slot + (int64_t)j * a.D, ch, a.D, p);
  }
}

template <typename T, int W, int VEC>
__global__ void __launch_bounds__(256) gdp_conv_decode_kernel(ConvArgs a) {
  const int64_t i = blockIdx.x;
  const int ch = ((int)blockIdx.y * 256 + threadIdx.x) * VEC;
  if (ch >= a.D) return;
  const int64_t s = index_at(a.slots, a.slots_is64, i);
  T *out = (T *)a.y + i * a.y_st;
  float y[VEC] = {};
  if (s >= 0 && s < a.num_slots) {
    T *state = (T *)a.cache + s * (W - 1) * a.D;
    Piece<T, VEC> x[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) x[j] = load_piece<T, VEC>(state + (int64_t)j * a.D, ch, a.D);
    x[W - 1] = load_piece<T, VEC>((const T *)a.x + i * a.x_st, ch, a.D);
    float w[W][VEC];
    load_taps<T, W, VEC>(w, y, a, ch);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int c = 0; c < VEC; ++c) y[c] = fmaf(w[j][c], (float)x[j].v[c], y[c]);
#pragma unroll
    for (int c = 0; c < VEC; ++c) y[c] = act_of(a.act, y[c]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_piece<T, VEC>(state + (int64_t)j * a.D, ch, a.D, x[j + 1]);
  }
  store_floats<T, VEC>(out, ch, a.D, y);
}

// The gradients.  The wave walks W - 1 rows past its chunk (rows behind the sequence's
// end have dv = 0), and row t's dx is whole when row t + W - 1 is done.  Chunk 0
// also forms the rows of the initial state's gradient, which lie before it.  Sums
// of dw and db over the chunk go to the workspace: row `number` of [numbers, W + 2, D].
template <typename T, int W, int VEC>
__global__ void __launch_bounds__(64 * WAVES) gdp_conv_backward_kernel(ConvArgs a, int shift, int blocks, int numbers,
                                                                       int jobs) {
  const int id = (int)blockIdx.x * WAVES + uniform_of(threadIdx.x >> 6);
  if (id >= jobs) return;
  const int number = id / blocks, ch = (id % blocks) * 64 * VEC + (threadIdx.x & 63) * VEC;
  Chunk k;
  // (by the whole wave: before lanes without channels leave)
  const bool some = number < numbers && find_chunk(&k, a.cu, a.cu_is64, a.T, a.N, shift, number);
  if (ch >= a.D) return;
  if (number >= numbers) {  // rows that no sequence covers
    const int64_t r0 = (int64_t)(number - numbers) << shift, r1 = min(r0 + ((int64_t)1 << shift), (int64_t)a.T);
    const int64_t c0 = bound_at(a.cu, a.cu_is64, 0, a.T), cN = a.N > 0 ? bound_at(a.cu, a.cu_is64, a.N, a.T) : 0;
    const float zero[VEC] = {};
    for (int64_t t = r0; t < r1; ++t)
      if (t < c0 || t >= cN) store_floats<T, VEC>((T *)a.dx + t * a.dx_st, ch, a.D, zero);
    return;
  }
  float dw[W][VEC] = {}, db[VEC] = {};
  if (some) {
    float w[W][VEC], b[VEC], x[W - 1 + ROWS][VEC], dv[W - 1 + ROWS][VEC];
    Piece<T, VEC> xn[ROWS] = {}, gn[ROWS] = {};
    const int stop = k.end + W - 1;  // rows walked: [begin, stop)
    auto fetch = [&](int t) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (t + r < min(stop, k.last)) {
          xn[r] = load_piece<T, VEC>((const T *)a.x + (int64_t)(t + r) * a.x_st, ch, a.D);
          gn[r] = load_piece<T, VEC>((const T *)a.dy + (int64_t)(t + r) * a.dy_st, ch, a.D);
        }
    };
    fetch(k.begin);
    load_taps<T, W, VEC>(w, b, a, ch);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      to_floats(x[j], row_before<T, W, VEC>(a, k, (int64_t)k.begin - (W - 1) + j, ch));
#pragma unroll
      for (int c = 0; c < VEC; ++c) dv[j][c] = 0.f;
    }
    for (int t = k.begin; t < stop; t += ROWS) {
      float g[ROWS][VEC];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        to_floats(x[W - 1 + r], xn[r]);
        to_floats(g[r], gn[r]);
      }
      fetch(t + ROWS);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (t + r >= stop) continue;
        if (t + r < k.last) {
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            float v = b[c], slope;
#pragma unroll
            for (int j = 0; j < W; ++j) v = fmaf(w[j][c], x[r + j][c], v);
            act_of(a.act, v, &slope);
            dv[W - 1 + r][c] = g[r][c] * slope;
          }
          if (t + r < k.end) {
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
#pragma unroll
              for (int j = 0; j < W; ++j) dw[j][c] = fmaf(dv[W - 1 + r][c], x[r + j][c], dw[j][c]);
              db[c] += dv[W - 1 + r][c];
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < VEC; ++c) dv[W - 1 + r][c] = 0.f;
        }
        const int row = t + r - (W - 1);  // whose dx is whole now
        const bool state = row < k.begin;
        if (state && (k.index > 0 || !a.ds0)) continue;
        float dx[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < W; ++i) s = fmaf(w[W - 1 - i][c], dv[r + i][c], s);
          dx[c] = s;
        }
        const int left = row - (k.last - (W - 1));  // the row's place in the final state
        if (a.dfinal && left >= 0) {
          const Piece<float, VEC> f =
              load_piece<float, VEC>(a.dfinal + ((int64_t)k.seq * (W - 1) + left) * a.D, ch, a.D);
#pragma unroll
          for (int c = 0; c < VEC; ++c) dx[c] += f.v[c];
        }
        if (state)
          store_floats<float, VEC>(a.ds0 + ((int64_t)k.seq * (W - 1) + (row - k.first + W - 1)) * a.D, ch, a.D, dx);
        else
          store_floats<T, VEC>((T *)a.dx + (int64_t)row * a.dx_st, ch, a.D, dx);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          x[j][c] = x[ROWS + j][c];
          dv[j][c] = dv[ROWS + j][c];
        }
    }
  }
  float *sums = a.ws + (int64_t)number * (W + 2) * a.D;
#pragma unroll
  for (int j = 0; j < W; ++j) store_floats<float, VEC>(sums + (int64_t)j * a.D, ch, a.D, dw[j]);
  if (a.db) store_floats<float, VEC>(sums + (int64_t)W * a.D, ch, a.D, db);
}

// Rows per chunk: the longest of 64, 32 and 16 that gives `want` waves.
int shift_of(int64_t T, int64_t blocks, int64_t want) {
  int shift = 6;
  while (shift > 4 && (T >> shift) * blocks < want) --shift;
  return shift;
}
constexpr int64_t WANT = 2048;

template <typename F> hipError_t by_type(int xt, F f) {
  if (xt == EL_F32) return f((float)0);
  return xt == EL_BF16 ? f((bf16)0) : f((_Float16)0);
}
template <int W> struct Taps { static constexpr int value = W; };
template <typename F> hipError_t by_taps(int W, F f) {
  switch (W) {
    case 2: return f(Taps<2>());
    case 3: return f(Taps<3>());
    case 4: return f(Taps<4>());
    case 5: return f(Taps<5>());
    case 6: return f(Taps<6>());
    case 7: return f(Taps<7>());
    default: return f(Taps<8>());
  }
}

int64_t blocks_of(int64_t D, int vec) { return (D + 64 * vec - 1) / (64 * vec); }
constexpr int FORWARD_VEC = 16, BACKWARD_VEC = 4;  // bytes per lane; channels per lane

}  // namespace

// A launch holds less than 2^32 threads: per block of at least 256 channels a wave for
// 16 rows, for a sequence, and in the gradients for 16 rows that may be uncovered.
bool conv_served(int64_t T, int64_t N, int64_t D) {
  if (T > BLOCK_MAX_ROWS || N > BLOCK_MAX_SEQS || D > BLOCK_MAX_CHANNELS) return false;
  return ((T >> 3) + 1 + N) * blocks_of(D, BACKWARD_VEC) < ((int64_t)1 << 32) / 64 - WAVES &&
         N * ((D + 1023) / 1024) < ((int64_t)1 << 32) / 256;
}

size_t conv_backward_bytes(int64_t T, int64_t N, int64_t D, int64_t W) {
  return (size_t)chunk_numbers(T, N, shift_of(T, blocks_of(D, BACKWARD_VEC), WANT)) * (W + 2) * D * 4;
}

hipError_t launch_conv(const ConvArgs &a, int xt, hipStream_t stream) {
  return by_type(xt, [&](auto x) {
    using T = decltype(x);
    constexpr int VEC = FORWARD_VEC / sizeof(T);
    const int64_t blocks = blocks_of(a.D, VEC);
    const int shift = shift_of(a.T, blocks, WANT);
    const int64_t jobs = chunk_numbers(a.T, a.N, shift) * blocks;
    if (jobs == 0 || a.N == 0) return hipSuccess;
    const bool streamed = (int64_t)a.T * a.D * 2 * (int64_t)sizeof(T) > STREAM_BYTES;
    return by_taps(a.W, [&](auto w) {
      auto *kernel = streamed ? gdp_conv_kernel<T, decltype(w)::value, VEC, true>
                              : gdp_conv_kernel<T, decltype(w)::value, VEC, false>;
      hipLaunchKernelGGL(kernel, dim3((unsigned)((jobs + WAVES - 1) / WAVES)), dim3(64 * WAVES), 0, stream, a, shift,
                         (int)blocks, (int)jobs);
      return hipGetLastError();
    });
  });
}

hipError_t launch_conv_decode(const ConvArgs &a, int xt, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  return by_type(xt, [&](auto x) {
    using T = decltype(x);
    constexpr int VEC = 4;
    return by_taps(a.W, [&](auto w) {
      hipLaunchKernelGGL((gdp_conv_decode_kernel<T, decltype(w)::value, VEC>),
                         dim3((unsigned)a.N, (unsigned)((a.D + 256 * VEC - 1) / (256 * VEC))), dim3(256), 0, stream, a);
      return hipGetLastError();
    });
  });
}

hipError_t launch_conv_backward(const ConvArgs &a, int xt, hipStream_t stream) {
  const int64_t blocks = blocks_of(a.D, BACKWARD_VEC);
  const int shift = shift_of(a.T, blocks, WANT);
  const int64_t numbers = chunk_numbers(a.T, a.N, shift), jobs = (numbers + (a.T >> shift) + 1) * blocks;
  const hipError_t e = by_type(xt, [&](auto x) {
    using T = decltype(x);
    return by_taps(a.W, [&](auto w) {
      hipLaunchKernelGGL((gdp_conv_backward_kernel<T, decltype(w)::value, BACKWARD_VEC>),
                         dim3((unsigned)((jobs + WAVES - 1) / WAVES)), dim3(64 * WAVES), 0, stream, a, shift,
                         (int)blocks, (int)numbers, (int)jobs);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess) return e;
  SumArgs s{a.ws, (int64_t)(a.W + 2) * a.D, (int)numbers, a.D, a.W, a.W, a.dw, a.db, nullptr};
  return launch_sums(s, stream);
}

}  // namespace gdp
