// gdp_norm.hip -- gfx950 kernels of the group norm with an activation over the
// channels of each (token, group), and of its gradients.  One wave per (token,
// group); the weight gradients are summed by one workgroup per channel.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp.h"
#include "gdp_layer.h"
#include "gdp_layer_common.h"

namespace gdp {
namespace {

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

template <typename T> __device__ __forceinline__ float param(const void *p, int type, int64_t i) {
  return type == EL_F32 ? ((const float *)p)[i] : (float)((const T *)p)[i];
}

// f = act(v) and its derivative
__device__ __forceinline__ void activate(int act, float v, float &f, float &df) {
  if (act == GDP_ACT_NONE) { f = v; df = 1.f; return; }
  const float s = 1.f / (1.f + expf(-v));
  if (act == GDP_ACT_SIGMOID) { f = s; df = s * (1.f - s); return; }
  f = v * s;
  df = s * (1.f + v * (1.f - s));
}

template <typename T> struct Row {
  const T *x;
  float mean, rstd;
  __device__ Row(const NormArgs &a, int64_t t, int g, int lane) {
    x = (const T *)a.x + t * a.x_st + g * a.x_sh;
    mean = 0.f;
    if (a.center) {
      float s = 0.f;
      for (int v = lane; v < a.V; v += 64) s += (float)x[v];
      mean = wave_sum(s) / a.V;
    }
    float ss = 0.f;
    for (int v = lane; v < a.V; v += 64) {
      const float d = (float)x[v] - mean;
      ss = fmaf(d, d, ss);
    }
    rstd = 1.f / sqrtf(wave_sum(ss) / a.V + a.eps);
  }
};

template <typename T> __global__ void __launch_bounds__(64) gdp_norm_kernel(NormArgs a) {
  const int64_t t = blockIdx.x / a.G;
  const int g = (int)(blockIdx.x % a.G), lane = threadIdx.x;
  const Row<T> r(a, t, g, lane);
  for (int v = lane; v < a.V; v += 64) {
    float n = ((float)r.x[v] - r.mean) * r.rstd;
    if (a.w) n *= param<T>(a.w, a.w_type, g * a.w_sh + v);
    if (a.b) n += param<T>(a.b, a.w_type, g * a.w_sh + v);
    float f, df;
    activate(a.act, a.z ? (float)((const T *)a.z)[t * a.z_st + g * a.z_sh + v] : n, f, df);
    ((T *)a.y)[t * a.y_st + g * a.y_sh + v] = (T)(a.z ? n * f : f);
  }
}

template <typename T> __global__ void __launch_bounds__(64) gdp_norm_backward_kernel(NormArgs a) {
  const int64_t t = blockIdx.x / a.G;
  const int g = (int)(blockIdx.x % a.G), lane = threadIdx.x;
  const Row<T> r(a, t, g, lane);
  const T *z = a.z ? (const T *)a.z + t * a.z_st + g * a.z_sh : nullptr;
  const T *dy = (const T *)a.dy + t * a.dy_st + g * a.dy_sh;
  float s1 = 0.f, s2 = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int v = lane; v < a.V; v += 64) {
      const float xhat = ((float)r.x[v] - r.mean) * r.rstd;
      const float w = a.w ? param<T>(a.w, a.w_type, g * a.w_sh + v) : 1.f;
      float n = xhat * w;
      if (a.b) n += param<T>(a.b, a.w_type, g * a.w_sh + v);
      float f, df;
      activate(a.act, z ? (float)z[v] : n, f, df);
      const float d = (float)dy[v], dn = d * (z ? f : df);
      if (pass == 0) {
        s1 += dn * w;
        s2 = fmaf(dn * w, xhat, s2);
      } else {
        ((T *)a.dx)[t * a.dx_st + g * a.dx_sh + v] = (T)((dn * w - s1 - xhat * s2) * r.rstd);
        if (z) ((T *)a.dz)[t * a.dz_st + g * a.dz_sh + v] = (T)(d * n * df);
      }
    }
    if (pass == 0) {
      s1 = a.center ? wave_sum(s1) / a.V : 0.f;
      s2 = wave_sum(s2) / a.V;
      if (a.ws && lane == 0) {
        a.ws[2 * (t * a.G + g)] = r.mean;
        a.ws[2 * (t * a.G + g) + 1] = r.rstd;
      }
    }
  }
}

// dw, db of channel blockIdx.x of group blockIdx.y (or of all groups)
template <typename T> __global__ void __launch_bounds__(256) gdp_norm_weight_kernel(NormArgs a) {
  const int v = blockIdx.x, tid = threadIdx.x;
  const bool shared = a.w_sh == 0;
  const int64_t rows = shared ? a.T * a.G : a.T;
  float dw = 0.f, db = 0.f;
  for (int64_t i = tid; i < rows; i += 256) {
    const int64_t t = shared ? i / a.G : i;
    const int g = shared ? (int)(i % a.G) : (int)blockIdx.y;
    const float mean = a.ws[2 * (t * a.G + g)], rstd = a.ws[2 * (t * a.G + g) + 1];
    const float xhat = ((float)((const T *)a.x)[t * a.x_st + g * a.x_sh + v] - mean) * rstd;
    float n = xhat;
    if (a.w) n *= param<T>(a.w, a.w_type, g * a.w_sh + v);
    if (a.b) n += param<T>(a.b, a.w_type, g * a.w_sh + v);
    float f, df;
    activate(a.act, a.z ? (float)((const T *)a.z)[t * a.z_st + g * a.z_sh + v] : n, f, df);
    const float dn = (float)((const T *)a.dy)[t * a.dy_st + g * a.dy_sh + v] * (a.z ? f : df);
    dw = fmaf(dn, xhat, dw);
    db += dn;
  }
  __shared__ float red[2][4];
  dw = wave_sum(dw);
  db = wave_sum(db);
  if ((tid & 63) == 0) { red[0][tid >> 6] = dw; red[1][tid >> 6] = db; }
  __syncthreads();
  if (tid == 0) {
    const int64_t at = blockIdx.y * a.w_sh + v;
    if (a.dw) a.dw[at] = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
    if (a.db) a.db[at] = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  }
}

template <typename F> hipError_t by_type(int xt, F f) {
  if (xt == EL_F32) return f((float)0);
  return xt == EL_BF16 ? f((bf16)0) : f((_Float16)0);
}

}  // namespace

size_t norm_backward_bytes(int64_t T, int64_t G, int64_t) { return (size_t)T * G * 8; }

hipError_t launch_norm(const NormArgs &a, int xt, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  if (a.T > INT32_MAX / a.G) return hipErrorInvalidValue;
  return by_type(xt, [&](auto x) {
    hipLaunchKernelGGL((gdp_norm_kernel<decltype(x)>), dim3((unsigned)(a.T * a.G)), dim3(64), 0, stream, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_backward(const NormArgs &a, int xt, hipStream_t stream) {
  if (a.T > INT32_MAX / a.G) return hipErrorInvalidValue;
  return by_type(xt, [&](auto x) {
    if (a.T > 0) {
      hipLaunchKernelGGL((gdp_norm_backward_kernel<decltype(x)>), dim3((unsigned)(a.T * a.G)), dim3(64), 0, stream, a);
      if (hipError_t e = hipGetLastError()) return e;
    }
    if (a.dw || a.db)
      hipLaunchKernelGGL((gdp_norm_weight_kernel<decltype(x)>), dim3((unsigned)a.V, a.w_sh ? (unsigned)a.G : 1u),
                         dim3(256), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace gdp
