// gdp_block.h -- internal interface between the C ABI (gdp_block_api.cpp) and the
// gfx950 kernels of the short convolution (gdp_conv.hip), of the selective scan
// (gdp_select.hip, gdp_select_bwd.hip) and of the norms around a block
// (gdp_resnorm.hip).  Not installed; not part of the ABI.  Strides are in elements,
// element types are ElType values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp_launch.h"

namespace gdp {

// most rows and sequences of these operators: a row's number is 32 bits wide
constexpr int64_t BLOCK_MAX_ROWS = (int64_t)1 << 30, BLOCK_MAX_SEQS = (int64_t)1 << 24,
                  BLOCK_MAX_CHANNELS = (int64_t)1 << 24;

constexpr int CONV_MAX_TAPS = 8;

struct ConvArgs {
  const void *x; int64_t x_st;          // [T, D] (decode: [N, D])
  const void *w, *b; int w_type;        // [D, W], [D] or null, float32 or x's type
  const void *cu; int cu_is64;          // [N+1]
  int T, N, D, W;
  int act;
  const void *s0;                       // [N, W-1, D] x's type, or null
  void *final_state;                    // [N, W-1, D] or null
  void *cache;                          // [num_slots, W-1, D] or null
  const void *slots; int slots_is64; int64_t num_slots;
  void *y; int64_t y_st;                // [T, D]
  // backward
  const void *dy; int64_t dy_st;        // [T, D]
  const float *dfinal;                  // [N, W-1, D] or null
  void *dx; int64_t dx_st;              // [T, D] x's type
  float *ds0;                           // [N, W-1, D] or null
  float *dw, *db;                       // [D, W], [D] or null
  float *ws;                            // conv_backward_bytes(T, N, D, W)
};
bool conv_served(int64_t T, int64_t N, int64_t D);
size_t conv_backward_bytes(int64_t T, int64_t N, int64_t D, int64_t W);
hipError_t launch_conv(const ConvArgs &a, int x_type, hipStream_t stream);
hipError_t launch_conv_decode(const ConvArgs &a, int x_type, hipStream_t stream);
hipError_t launch_conv_backward(const ConvArgs &a, int x_type, hipStream_t stream);

// states per channel at most, and rows of a sequence per checkpoint
constexpr int SELECT_MAX_STATES = 32, SELECT_SHIFT = 4, SELECT_ROWS = 1 << SELECT_SHIFT;

struct SelectArgs {
  const void *u; int64_t u_st;          // [T, D] (decode: [N, D])
  const void *dt; int64_t dt_st;        // [T, D] float32 or u's type
  const float *A;                       // [D, S]
  const void *B; int64_t B_st, B_sg;    // [T, G, S] u's type
  const void *C; int64_t C_st, C_sg;
  const float *skip, *bias;             // [D] or null
  const void *z; int64_t z_st;          // [T, D] or null
  const void *cu; int cu_is64;          // [N+1]
  int T, N, D, G, S;
  int softplus;
  const float *s0;                      // [N, D, S] or null
  float *final_state;                   // [N, D, S] or null
  float *cache;                         // [num_slots, D, S] or null
  const void *slots; int slots_is64; int64_t num_slots;
  float *points;                        // [T / SELECT_ROWS + N, S, D] or null (backward: read)
  void *o; int64_t o_st;                // [T, D], or null (states only)
  // backward
  const void *d_o; int64_t do_st;       // [T, D]
  const float *dfinal;                  // [N, D, S] or null
  void *du; int64_t du_st;              // [T, D] u's type
  void *ddt; int64_t ddt_st;            // [T, D] dt's type
  float *dA;                            // [D, S]
  void *dB, *dC;                        // [T, G, S] u's type, contiguous
  float *dskip, *dbias;                 // [D] or null
  void *dz; int64_t dz_st;              // [T, D] or null
  float *ds0;                           // [N, D, S] or null
  void *ws;
};
bool select_served(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S);
size_t select_bytes(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S);
size_t select_backward_bytes(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S, bool with_points);
hipError_t launch_select(const SelectArgs &a, int u_type, int dt_type, hipStream_t stream);
hipError_t launch_select_decode(const SelectArgs &a, int u_type, int dt_type, hipStream_t stream);
hipError_t launch_select_backward(const SelectArgs &a, int u_type, int dt_type, hipStream_t stream);

struct ResNormArgs {
  const void *x; int64_t x_st;          // [T, D] residual stream
  const void *y; int64_t y_st;          // [T, D] block's output
  const void *z; int64_t z_st;          // [T, D] gate, y's type, or null
  const void *w_post, *w_pre;           // [D] or null
  int w_type;
  int64_t T; int D;
  int act, post, pre;
  float scale, eps;
  void *r; int64_t r_st;                // [T, D] x's type
  void *n; int64_t n_st;                // [T, D] y's type, or null
  // backward
  const void *dr; int64_t dr_st;        // [T, D] x's type, or null
  const void *dn; int64_t dn_st;        // [T, D] y's type, or null
  void *dx; int64_t dx_st;              // x's type
  void *dy; int64_t dy_st;              // y's type
  void *dz; int64_t dz_st;              // y's type, or null
  float *dw_post, *dw_pre;              // [D] or null
  float *ws;                            // resnorm_backward_bytes(T, D)
};
constexpr int64_t RESNORM_MAX_CHANNELS = 16384;
size_t resnorm_backward_bytes(int64_t T, int64_t D);
hipError_t launch_resnorm(const ResNormArgs &a, int y_type, int x_type, hipStream_t stream);
hipError_t launch_resnorm_backward(const ResNormArgs &a, int y_type, int x_type, hipStream_t stream);

// Sums over the rows of p [rows, planes + 2, cols] (rows `stride` apart): the first planes
// to a[col * planes + plane], the last two to b[col] and c[col]; null outputs are skipped.
struct SumArgs {
  const float *p; int64_t stride;
  int rows, cols, planes, kept;         // kept: planes written to a, a[col * kept + plane]
  float *a, *b, *c;
};
hipError_t launch_sums(const SumArgs &s, hipStream_t stream);

}  // namespace gdp
