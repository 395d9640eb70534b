// gdp_scan.hip -- gfx950 kernels of the gated linear recurrence
//     h_t = a_t h_{t-1} + u_t,  a_t = exp(g_t),  u_t = x_t or (1 - a_t) x_t
// per channel over packed sequences, of its single-token step, and of its
// gradients.  One lane per (sequence, channel) walks the sequence's rows.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp_layer.h"
#include "gdp_layer_common.h"

namespace gdp {
namespace {

template <typename XT, typename GT>
__global__ void __launch_bounds__(64) gdp_scan_kernel(ScanArgs a) {
  const int64_t i = blockIdx.x, ch = (int64_t)blockIdx.y * 64 + threadIdx.x;
  if (ch >= a.D) return;
  const int64_t lo = bound_at(a.cu, a.cu_is64, i, a.T), hi = bound_at(a.cu, a.cu_is64, i + 1, a.T);
  float h = a.s0 ? a.s0[i * a.D + ch] : 0.f;
  for (int64_t t = lo; t < hi; ++t) {
    if (a.checkpoints && t % SCAN_ROWS == 0) a.checkpoints[t / SCAN_ROWS * a.D + ch] = h;
    const float g = (float)((const GT *)a.g)[t * a.g_st + ch], x = (float)((const XT *)a.x)[t * a.x_st + ch];
    const float d = decay(g);
    h = fmaf(d, h, a.complement ? one_minus_decay(g, d) * x : x);
    if (a.o) ((XT *)a.o)[t * a.o_st + ch] = (XT)h;
  }
  if (a.final_state) a.final_state[i * a.D + ch] = h;
  if (a.cache) {
    const int64_t slot = index_at(a.slots, a.slots_is64, i);
    if (slot >= 0 && slot < a.num_slots) a.cache[slot * a.D + ch] = h;
  }
}

// The rows before the first sequence and behind the last one (i = N) get zeros.
template <typename XT, typename GT>
__global__ void __launch_bounds__(64) gdp_scan_backward_kernel(ScanArgs a) {
  const int64_t i = blockIdx.x, ch = (int64_t)blockIdx.y * 64 + threadIdx.x;
  if (ch >= a.D) return;
  auto put = [&](int64_t t, float dx, float dg) {
    if (a.dx_f32) ((float *)a.dx)[t * a.dx_st + ch] = dx; else ((XT *)a.dx)[t * a.dx_st + ch] = (XT)dx;
    if (a.dg_f32) ((float *)a.dg)[t * a.dg_st + ch] = dg; else ((GT *)a.dg)[t * a.dg_st + ch] = (GT)dg;
  };
  if (i == a.N) {
    const int64_t first = bound_at(a.cu, a.cu_is64, 0, a.T), last = bound_at(a.cu, a.cu_is64, a.N, a.T);
    for (int64_t t = 0; t < first; ++t) put(t, 0.f, 0.f);
    for (int64_t t = last; t < a.T; ++t) put(t, 0.f, 0.f);
    return;
  }
  const int64_t lo = bound_at(a.cu, a.cu_is64, i, a.T), hi = bound_at(a.cu, a.cu_is64, i + 1, a.T);
  float e = a.dfinal ? a.dfinal[i * a.D + ch] : 0.f;
  float before[SCAN_ROWS];
  for (int64_t end = hi; end > lo;) {
    int64_t begin = (end - 1) / SCAN_ROWS * SCAN_ROWS;
    float h;
    if (begin <= lo) {
      begin = lo;
      h = a.s0 ? a.s0[i * a.D + ch] : 0.f;
    } else {
      h = a.checkpoints[begin / SCAN_ROWS * a.D + ch];
    }
    for (int64_t t = begin; t < end; ++t) {
      const float g = (float)((const GT *)a.g)[t * a.g_st + ch], x = (float)((const XT *)a.x)[t * a.x_st + ch];
      const float d = decay(g);
      before[t - begin] = h;
      h = fmaf(d, h, a.complement ? one_minus_decay(g, d) * x : x);
    }
    for (int64_t t = end - 1; t >= begin; --t) {
      const float g = (float)((const GT *)a.g)[t * a.g_st + ch], x = (float)((const XT *)a.x)[t * a.x_st + ch];
      const float d = decay(g), p = before[t - begin];
      e += (float)((const XT *)a.dout)[t * a.do_st + ch];
      put(t, a.complement ? one_minus_decay(g, d) * e : e, e * d * (a.complement ? p - x : p));
      e *= d;
    }
    end = begin;
  }
  if (a.ds0) a.ds0[i * a.D + ch] = e;
}

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

}  // namespace

size_t scan_state_bytes(int64_t, int64_t) { return 0; }
bool scan_served(int64_t, int64_t N, int64_t D) { return N < INT32_MAX && (D + 63) / 64 <= 65535; }

hipError_t launch_scan(const ScanArgs &a, int xt, int gt, hipStream_t stream) {
  if (a.N == 0) return hipSuccess;
  return by_types(xt, gt, [&](auto x, auto g) {
    hipLaunchKernelGGL((gdp_scan_kernel<decltype(x), decltype(g)>), dim3((unsigned)a.N, (unsigned)((a.D + 63) / 64)),
                       dim3(64), 0, stream, a);
    return hipGetLastError();
  });
}

hipError_t launch_scan_backward(const ScanArgs &a, int xt, int gt, hipStream_t stream) {
  return by_types(xt, gt, [&](auto x, auto g) {
    hipLaunchKernelGGL((gdp_scan_backward_kernel<decltype(x), decltype(g)>),
                       dim3((unsigned)(a.N + 1), (unsigned)((a.D + 63) / 64)), dim3(64), 0, stream, a);
    return hipGetLastError();
  });
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
