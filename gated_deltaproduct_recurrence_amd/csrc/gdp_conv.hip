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
// one chunk of a sequence (gdp_block_common.h) and a block of channels and walks down the
// rows with the last W - 1 of them in registers, as floats; a group of rows is loaded
// while the one before is computed.  The W - 1 rows before the chunk are read a second
// time, out of the caches.  Groups that lie inside the chunk take no branch per row.
//
// What bounds it, measured on MI355X (a 1 GiB copy reaches 5.1 TB/s): the memory.
// 131104 x 4096 bfloat16 in 68 sequences, 4 taps, SiLU: 393 us, 5.5 TB/s; 32768 x 2048:
// 51 us, 5.3 TB/s.
//   Forward: 8 bytes of a row per lane, chunks of 16 rows, groups of 2.  On the first shape
// 16 bytes per lane take 405 us, chunks of 32 and 64 rows 409 and 441, groups of 1 and 4 rows
// 524 and 544, and loads and stores left to the caches 407.
//   Gradients of the second shape: 114 us, 3.5 TB/s (their sums another 7 us), the vector units
// busy 66% of the time, 6900 of 8192 waves resident: neither they nor the memory are full.
// One channel per lane, chunks of up to 128 rows, groups of 4.  2 and 4 channels per lane
// take 141 and 211 us, chunks of up to 32 and 64 rows 135 and 120.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp.h"
#include "gdp_block.h"
#include "gdp_block_common.h"

namespace gdp {
namespace {

constexpr int WAVES = 4, FORWARD_ROWS = 2, BACKWARD_ROWS = 4;  // rows: of a group, loaded a group ahead

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

template <typename P, int W, int VEC> __device__ __forceinline__ void load_rows(float (&w)[W][VEC], const P *p, int ch, int D) {
  if (ch + VEC <= D) {  // the channels' taps lie behind each other
    const Piece<P, VEC * W> all = *(const Piece<P, VEC * W> *)(p + (int64_t)ch * W);
#pragma unroll
    for (int c = 0; c < VEC; ++c)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][c] = (float)all.v[c * W + j];
    return;
  }
#pragma unroll
  for (int c = 0; c < VEC; ++c)
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][c] = ch + c < D ? (float)p[(int64_t)(ch + c) * W + j] : 0.f;
}
template <typename T, int W, int VEC>
__device__ __forceinline__ void load_taps(float (&w)[W][VEC], float (&b)[VEC], const ConvArgs &a, int ch) {
  if (a.w_type == EL_F32) load_rows<float, W, VEC>(w, (const float *)a.w, ch, a.D);
  else load_rows<T, W, VEC>(w, (const T *)a.w, ch, a.D);
#pragma unroll
  for (int c = 0; c < VEC; ++c) b[c] = a.b && ch + c < a.D ? param_at<T>(a.b, a.w_type, ch + c) : 0.f;
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
  constexpr int ROWS = FORWARD_ROWS;
  if (k.begin < k.end) {
    float w[W][VEC], b[VEC], x[W - 1 + ROWS][VEC];
    Piece<T, VEC> next[ROWS] = {};
    const T *row = (const T *)a.x + (int64_t)k.begin * a.x_st;
    auto fetch = [&](int t) {
      const T *p = row + (int64_t)(t - k.begin) * a.x_st;
      if (t + ROWS <= k.end) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) next[r] = load_piece<T, VEC, STREAMED>(p + r * a.x_st, ch, a.D);
      } else {
#pragma unroll
        for (int r = 0; r < ROWS - 1; ++r)
          if (t + r < k.end) next[r] = load_piece<T, VEC, STREAMED>(p + r * a.x_st, ch, a.D);
      }
    };
    fetch(k.begin);
    load_taps<T, W, VEC>(w, b, a, ch);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) to_floats(x[j], row_before<T, W, VEC>(a, k, (int64_t)k.begin - (W - 1) + j, ch));
    T *out = (T *)a.y + (int64_t)k.begin * a.y_st;
    // `count` rows of the group in x, all of them (without a branch per row) or fewer
    auto group = [&](auto all, int count) {
      float y[ROWS][VEC];
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          float v = b[c];
#pragma unroll
          for (int j = 0; j < W; ++j) v = fmaf(w[j][c], x[r + j][c], v);
          y[r][c] = v;
        }
      if (a.act != GDP_ACT_NONE) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
          for (int c = 0; c < VEC; ++c) y[r][c] = act_of(a.act, y[r][c]);
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (decltype(all)::value || r < count) store_floats<T, VEC, STREAMED>(out + r * a.y_st, ch, a.D, y[r]);
      out += ROWS * a.y_st;
    };
    for (int t = k.begin; t < k.end; t += ROWS) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) to_floats(x[W - 1 + r], next[r]);
      fetch(t + ROWS);
      if (t + ROWS <= k.end) group(Flag<true>(), ROWS);
      else group(Flag<false>(), k.end - t);
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
template <typename T, int W, int VEC, bool STREAMED>
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
  constexpr int ROWS = BACKWARD_ROWS;
  if (some) {
    float w[W][VEC], b[VEC], x[W - 1 + ROWS][VEC], dv[W - 1 + ROWS][VEC];
    Piece<T, VEC> xn[ROWS] = {}, gn[ROWS] = {}, g[ROWS];
    const int stop = k.end + W - 1;  // rows walked: [begin, stop)
    const int rows_in = min(stop, k.last);  // rows read: [begin, rows_in)
    auto fetch = [&](int t) {
      const T *px = (const T *)a.x + (int64_t)t * a.x_st, *pg = (const T *)a.dy + (int64_t)t * a.dy_st;
      if (t + ROWS <= rows_in) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          xn[r] = load_piece<T, VEC, STREAMED>(px + r * a.x_st, ch, a.D);
          gn[r] = load_piece<T, VEC, STREAMED>(pg + r * a.dy_st, ch, a.D);
        }
      } else {
#pragma unroll
        for (int r = 0; r < ROWS - 1; ++r)
          if (t + r < rows_in) {
            xn[r] = load_piece<T, VEC, STREAMED>(px + r * a.x_st, ch, a.D);
            gn[r] = load_piece<T, VEC, STREAMED>(pg + r * a.dy_st, ch, a.D);
          }
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
    // row t + r of a group: its dv, its share of the sums, and the dx of the row W - 1 before
    auto slope_of = [&](int r) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        float v = b[c], slope;
#pragma unroll
        for (int j = 0; j < W; ++j) v = fmaf(w[j][c], x[r + j][c], v);
        act_of(a.act, v, &slope);
        dv[W - 1 + r][c] = (float)g[r].v[c] * slope;
      }
    };
    auto sums_of = [&](int r) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][c] = fmaf(dv[W - 1 + r][c], x[r + j][c], dw[j][c]);
        db[c] += dv[W - 1 + r][c];
      }
    };
    auto dx_of = [&](float (&dx)[VEC], int r) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) s = fmaf(w[W - 1 - i][c], dv[r + i][c], s);
        dx[c] = s;
      }
    };
    for (int t = k.begin; t < stop; t += ROWS) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        to_floats(x[W - 1 + r], xn[r]);
        g[r] = gn[r];
      }
      fetch(t + ROWS);
      const int first = t - (W - 1);  // whose dx is whole with row t
      if (t + ROWS <= k.end && first >= k.begin && first + ROWS <= k.last - (W - 1)) {
        // inside the chunk, and no row of the initial or the final state among those finished
#pragma unroll
        for (int r = 0; r < ROWS; ++r) slope_of(r);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) sums_of(r);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          float dx[VEC];
          dx_of(dx, r);
          store_floats<T, VEC, STREAMED>((T *)a.dx + (int64_t)(first + r) * a.dx_st, ch, a.D, dx);
        }
      } else {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          if (t + r >= stop) continue;
          if (t + r < k.last) {
            slope_of(r);
            if (t + r < k.end) sums_of(r);
          } else {
#pragma unroll
            for (int c = 0; c < VEC; ++c) dv[W - 1 + r][c] = 0.f;
          }
          const int row = first + r;
          const bool state = row < k.begin;
          if (state && (k.index > 0 || !a.ds0)) continue;
          float dx[VEC];
          dx_of(dx, r);
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
            store_floats<T, VEC, STREAMED>((T *)a.dx + (int64_t)row * a.dx_st, ch, a.D, dx);
        }
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

// log2 of the rows per chunk: 16, or 8 (at least the W - 1 rows before it) where that
// leaves fewer than 2048 waves
int forward_shift(int64_t T, int64_t blocks) { return (T >> 4) * blocks < 2048 ? 3 : 4; }
// ... of the gradients: 128, or fewer down to 16 for at least 4096 waves
int backward_shift(int64_t T, int64_t blocks) {
  int shift = 7;
  while (shift > 4 && (T >> shift) * blocks < 4096) --shift;
  return shift;
}

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
constexpr int FORWARD_VEC = 8, BACKWARD_VEC = 1;  // bytes per lane; channels per lane

}  // namespace

// A launch holds less than 2^32 threads: in the gradients, per block of 64 channels, a wave for
// 16 rows, another for 16 rows that may be uncovered, and one for a sequence.  The forward pass has
// one for 8 rows and for a sequence, per wider block; the decode step 256 threads per entry and
// 1024 channels.
bool conv_served(int64_t T, int64_t N, int64_t D) {
  if (T > BLOCK_MAX_ROWS || N > BLOCK_MAX_SEQS || D > BLOCK_MAX_CHANNELS) return false;
  return ((T >> 3) + 1 + N) * blocks_of(D, BACKWARD_VEC) < ((int64_t)1 << 32) / 64 - WAVES &&
         N * ((D + 1023) / 1024) < ((int64_t)1 << 32) / 256;
}

size_t conv_backward_bytes(int64_t T, int64_t N, int64_t D, int64_t W) {
  return (size_t)chunk_numbers(T, N, backward_shift(T, blocks_of(D, BACKWARD_VEC))) * (W + 2) * D * 4;
}

hipError_t launch_conv(const ConvArgs &a, int xt, hipStream_t stream) {
  return by_type(xt, [&](auto x) {
    using T = decltype(x);
    constexpr int VEC = FORWARD_VEC / sizeof(T);
    const int64_t blocks = blocks_of(a.D, VEC);
    const int shift = forward_shift(a.T, blocks);
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
  const int shift = backward_shift(a.T, blocks);
  const int64_t numbers = chunk_numbers(a.T, a.N, shift), jobs = (numbers + (a.T >> shift) + 1) * blocks;
  const hipError_t e = by_type(xt, [&](auto x) {
    using T = decltype(x);
    const bool streamed = (int64_t)a.T * a.D * 3 * (int64_t)sizeof(T) > STREAM_BYTES;
    return by_taps(a.W, [&](auto w) {
      auto *kernel = streamed ? gdp_conv_backward_kernel<T, decltype(w)::value, BACKWARD_VEC, true>
                              : gdp_conv_backward_kernel<T, decltype(w)::value, BACKWARD_VEC, false>;
      hipLaunchKernelGGL(kernel, dim3((unsigned)((jobs + WAVES - 1) / WAVES)), dim3(64 * WAVES), 0, stream, a, shift,
                         (int)blocks, (int)numbers, (int)jobs);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess) return e;
  SumArgs s{a.ws, (int64_t)(a.W + 2) * a.D, (int)numbers, a.D, a.W, a.W, a.dw, a.db, nullptr};
  return launch_sums(s, stream);
}

}  // namespace gdp
