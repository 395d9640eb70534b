// gdp_sums.hip -- sums over rows of partial sums: the last step of the weight
// gradients of the short convolution, the selective scan and the norms around a
// block.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp_block.h"

namespace gdp {
namespace {

// 16 columns of one plane per workgroup, the rows dealt over 64 lane groups, eight
// loads ahead.  A fixed order: the result does not depend on timing.
__global__ void __launch_bounds__(1024) gdp_sums_kernel(SumArgs s) {
  __shared__ float red[64][17];
  const int c = threadIdx.x & 15, part = threadIdx.x >> 4, plane = blockIdx.y;
  const int col = (int)blockIdx.x * 16 + c;
  float *out;
  int64_t at = col;
  if (plane < s.planes) {
    out = plane < s.kept ? s.a : nullptr;
    at = (int64_t)col * s.kept + plane;
  } else {
    out = plane == s.planes ? s.b : s.c;
  }
  if (!out) return;
  float sum = 0.f;
  if (col < s.cols) {
    const float *p = s.p + (int64_t)plane * s.cols + col;
    int r = part;
    for (; r + 64 * 7 < s.rows; r += 64 * 8) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[(r + 64 * i) * s.stride];
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i];
    }
    for (; r < s.rows; r += 64) sum += p[r * s.stride];
  }
  red[part][c] = sum;
  __syncthreads();
  for (int n = 32; n > 0; n >>= 1) {
    if (part < n) red[part][c] += red[part + n][c];
    __syncthreads();
  }
  if (part == 0 && col < s.cols) out[at] = red[0][c];
}

}  // namespace

hipError_t launch_sums(const SumArgs &s, hipStream_t stream) {
  if (!s.a && !s.b && !s.c) return hipSuccess;
  hipLaunchKernelGGL(gdp_sums_kernel, dim3((unsigned)((s.cols + 15) / 16), (unsigned)(s.planes + 2)), dim3(1024), 0,
                     stream, s);
  return hipGetLastError();
}

}  // namespace gdp
