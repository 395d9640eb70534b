// gdp_layer.h -- internal interface between the C ABI (gdp_layer_api.cpp) and
// the gfx950 kernels of the gated linear recurrence (gdp_scan.hip) and of the
// group norm (gdp_norm.hip).  Not installed; not part of the ABI.  Strides are
// in elements, element types are ElType values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdp_launch.h"

namespace gdp {

// rows of the token stream per checkpoint and per tile of the gradients, and per tile
// of the forward pass
constexpr int SCAN_ROWS = 64, SCAN_FORWARD_ROWS = 128;

struct ScanArgs {
  const void *x; int64_t x_st;          // [T, D]
  const void *g; int64_t g_st;          // [T, D] log decays
  const void *cu; int cu_is64;          // [N+1]
  int64_t T, N, D;
  int complement;
  const float *s0;                      // [N, D] or null
  float *final_state;                   // [N, D] or null
  float *cache;                         // [num_slots, D] or null
  const void *slots; int slots_is64; int64_t num_slots;
  float *checkpoints;                   // [ceil(T / SCAN_ROWS), D] or null (backward: read)
  void *o; int64_t o_st;                // [T, D] or null (states only)
  // backward
  const void *dout; int64_t do_st;      // [T, D]
  const float *dfinal;                  // [N, D] or null
  void *dx; int64_t dx_st; int dx_f32;  // [T, D] float32 or x's type
  void *dg; int64_t dg_st; int dg_f32;  // [T, D] float32 or g's type
  float *ds0;                           // [N, D] or null
  void *ws;                             // scan_state_bytes(T, D, rows per tile)
  int streamed;                         // set by the launch: the rows' loads bypass the caches
};
// the counter and the words through which tiles of `rows` rows hand their states on
size_t scan_state_bytes(int64_t T, int64_t D, int rows);
// whether the launch grids of these sizes fit
bool scan_served(int64_t T, int64_t N, int64_t D);
hipError_t launch_scan(const ScanArgs &a, int x_type, int g_type, hipStream_t stream);
hipError_t launch_scan_backward(const ScanArgs &a, int x_type, int g_type, hipStream_t stream);

struct ScanDecodeArgs {
  const void *x; int64_t x_st;          // [N, D]
  const void *g; int64_t g_st;          // [N, D]
  int64_t N, D;
  int complement;
  float *cache; int64_t num_slots;      // [num_slots, D], read and written in place
  const void *slots; int slots_is64;    // [N]
  void *o; int64_t o_st;                // [N, D]
};
hipError_t launch_scan_decode(const ScanDecodeArgs &a, int x_type, int g_type, hipStream_t stream);

struct NormArgs {
  const void *x; int64_t x_st, x_sh;    // [T, G, V]
  const void *w, *b; int w_type;        // [V] or [G, V], float32 or x's type, or null
  int64_t w_sh;                         // stride between the groups' weights: V, or 0 when shared
  const void *z; int64_t z_st, z_sh;    // [T, G, V] or null
  int64_t T; int G, V;
  int act, center;
  float eps;
  void *y; int64_t y_st, y_sh;          // [T, G, V]
  // backward
  const void *dy; int64_t dy_st, dy_sh;
  void *dx; int64_t dx_st, dx_sh;
  void *dz; int64_t dz_st, dz_sh;
  float *dw, *db;                       // [V] or [G, V] or null
  float *ws;                            // norm_backward_bytes(T, G, V)
};
constexpr int64_t NORM_MAX_SIZE = 16384, NORM_MAX_GROUPS = 65535;
size_t norm_backward_bytes(int64_t T, int64_t G, int64_t V);
hipError_t launch_norm(const NormArgs &a, int x_type, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs &a, int x_type, hipStream_t stream);

}  // namespace gdp
