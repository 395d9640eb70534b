// gdp_layer_api.cpp -- C ABI of the gated linear recurrence and of the group
// norm (declared in include/gdp.h).  As in gdp_api.cpp: host-side validation of
// shapes, dtypes, strides and pointer ranges, then launches on the caller's
// stream.

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstring>

#include "gdp.h"
#include "gdp_check.h"
#include "gdp_layer.h"
#include "gdp_layer_check.h"

using namespace gdp;

namespace {

int check_scan_types(const gdp_tensor *x, const gdp_tensor *g) {
  if (!is_float(x->dtype)) return fail(GDP_EUNSUPPORTED, "x must be float32, bfloat16 or float16");
  if (g->dtype != GDP_F32 && g->dtype != x->dtype)
    return fail(GDP_EUNSUPPORTED, "g_log must be float32 or x's dtype");
  return GDP_OK;
}

int64_t checkpoint_rows(int64_t T) { return (T + SCAN_ROWS - 1) / SCAN_ROWS; }

bool scan_sizes_ok(int64_t T, int64_t N, int64_t D) { return T >= 0 && N >= 0 && D >= 1 && scan_served(T, N, D); }

}  // namespace

extern "C" {

size_t gdp_gated_scan_workspace_bytes(int64_t T, int64_t N, int64_t D) {
  if (!scan_sizes_ok(T, N, D)) return 0;
  return scan_state_bytes(T, D, SCAN_FORWARD_ROWS);
}

size_t gdp_gated_scan_backward_workspace_bytes(int64_t T, int64_t N, int64_t D) {
  if (!scan_sizes_ok(T, N, D)) return 0;
  return scan_state_bytes(T, D, SCAN_ROWS) + align256((size_t)checkpoint_rows(T) * D * 4);
}

int gdp_gated_scan(const gdp_tensor *x, const gdp_tensor *g_log, const gdp_tensor *cu_seqlens,
                   int32_t complement_input, const gdp_tensor *initial_state, int32_t output_final_state,
                   const gdp_tensor *state_cache, const gdp_tensor *state_indices, int32_t return_checkpoints,
                   const gdp_tensor *o, const gdp_tensor *final_state, const gdp_tensor *checkpoints,
                   void *workspace, size_t workspace_bytes, void *stream) {
  g_last_error.clear();
  if (!present(x) || !present(g_log) || !present(o)) return fail(GDP_EINVAL, "x, g_log and o are required");
  if (!present(cu_seqlens)) return fail(GDP_EINVAL, "cu_seqlens is required (varlen input only)");
  if (x->ndim != 2) return fail(GDP_EINVAL, "x must be [T, D]");
  int rc;
  if ((rc = check_cu(cu_seqlens))) return rc;
  const int64_t T = x->shape[0], D = x->shape[1], N = cu_seqlens->shape[0] - 1;
  if (D < 1) return fail(GDP_EINVAL, "x needs at least one channel");
  if ((rc = check_scan_types(x, g_log))) return rc;
  if (o->dtype != x->dtype) return fail(GDP_EUNSUPPORTED, "x and o must share one dtype");
  if ((rc = check_rows(x, "x", T, D)) || (rc = check_rows(g_log, "g_log", T, D)) || (rc = check_rows(o, "o", T, D)) ||
      (rc = check_row_overlap(o, "o")))
    return rc;
  if (!scan_served(T, N, D))
    return fail(GDP_EUNSUPPORTED, "T=%lld, N=%lld, D=%lld is past the launch limits", (long long)T, (long long)N,
                (long long)D);
  const bool init = present(initial_state), sink = present(state_cache);
  if (init && (rc = check_states(initial_state, "initial_state", N, D))) return rc;
  if (output_final_state) {
    if (!present(final_state)) return fail(GDP_EINVAL, "output_final_state needs a final_state buffer");
    if ((rc = check_states(final_state, "final_state", N, D))) return rc;
  }
  if (sink != present(state_indices)) return fail(GDP_EINVAL, "state_cache and state_indices go together");
  if (sink && (rc = check_slots(state_cache, state_indices, N, D))) return rc;
  if (return_checkpoints) {
    if (!present(checkpoints)) return fail(GDP_EINVAL, "return_checkpoints needs a checkpoints buffer");
    if ((rc = check_states(checkpoints, "checkpoints", checkpoint_rows(T), D))) return rc;
  }
  const size_t need = gdp_gated_scan_workspace_bytes(T, N, D);
  if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const Range ins[] = {range_of(x, "x"), range_of(g_log, "g_log"), range_of(cu_seqlens, "cu_seqlens"),
                       range_of(initial_state, "initial_state"), range_if(sink, state_indices, "state_indices")};
  const Range outs[] = {range_of(o, "o"), range_if(output_final_state != 0, final_state, "final_state"),
                        range_if(sink, state_cache, "state_cache"),
                        range_if(return_checkpoints != 0, checkpoints, "checkpoints"),
                        workspace_range(workspace, need)};
  if ((rc = check_alias(ins, outs))) return rc;

  ScanArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = x->data; a.x_st = x->stride[0];
  a.g = g_log->data; a.g_st = g_log->stride[0];
  a.cu = cu_seqlens->data; a.cu_is64 = cu_seqlens->dtype == GDP_I64;
  a.T = T; a.N = N; a.D = D;
  a.complement = complement_input != 0;
  a.s0 = init ? (const float *)initial_state->data : nullptr;
  a.final_state = output_final_state ? (float *)final_state->data : nullptr;
  if (sink) {
    a.cache = (float *)state_cache->data;
    a.num_slots = state_cache->shape[0];
    a.slots = state_indices->data;
    a.slots_is64 = state_indices->dtype == GDP_I64;
  }
  a.checkpoints = return_checkpoints ? (float *)checkpoints->data : nullptr;
  a.o = o->data; a.o_st = o->stride[0];
  a.ws = workspace;
  hipError_t e;
  if (debug_validate()) {
    ValidateArgs va;
    std::memset(&va, 0, sizeof va);
    va.cu = a.cu; va.cu_is64 = a.cu_is64; va.N = N; va.T = T;
    va.slots = a.slots; va.slots_is64 = a.slots_is64; va.nslots_given = sink ? N : 0; va.num_slots = a.num_slots;
    if ((e = launch_validate(va, (hipStream_t)stream)) != hipSuccess)
      return fail(GDP_EHIP, "validation launch: %s", hipGetErrorString(e));
  }
  e = launch_scan(a, float_type(x->dtype), float_type(g_log->dtype), (hipStream_t)stream);
  if (e != hipSuccess) return fail(GDP_EHIP, "scan launch: %s", hipGetErrorString(e));
  return GDP_OK;
}

int gdp_gated_scan_decode(const gdp_tensor *x, const gdp_tensor *g_log, int32_t complement_input,
                          const gdp_tensor *state_cache, const gdp_tensor *state_indices, const gdp_tensor *o,
                          void *stream) {
  g_last_error.clear();
  if (!present(x) || !present(g_log) || !present(o)) return fail(GDP_EINVAL, "x, g_log and o are required");
  if (!present(state_cache) || !present(state_indices))
    return fail(GDP_EINVAL, "state_cache and state_indices are required");
  if (x->ndim != 2) return fail(GDP_EINVAL, "x must be [N, D]");
  int rc;
  const int64_t N = x->shape[0], D = x->shape[1];
  if (D < 1) return fail(GDP_EINVAL, "x needs at least one channel");
  if ((rc = check_scan_types(x, g_log))) return rc;
  if (o->dtype != x->dtype) return fail(GDP_EUNSUPPORTED, "x and o must share one dtype");
  if ((rc = check_rows(x, "x", N, D)) || (rc = check_rows(g_log, "g_log", N, D)) || (rc = check_rows(o, "o", N, D)) ||
      (rc = check_row_overlap(o, "o")) || (rc = check_slots(state_cache, state_indices, N, D)))
    return rc;
  if (!scan_served(0, N, D))
    return fail(GDP_EUNSUPPORTED, "N=%lld, D=%lld is past the launch limits", (long long)N, (long long)D);
  const Range ins[] = {range_of(x, "x"), range_of(g_log, "g_log"), range_of(state_indices, "state_indices")};
  const Range outs[] = {range_of(o, "o"), range_of(state_cache, "state_cache")};
  if ((rc = check_alias(ins, outs))) return rc;

  ScanDecodeArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = x->data; a.x_st = x->stride[0];
  a.g = g_log->data; a.g_st = g_log->stride[0];
  a.N = N; a.D = D;
  a.complement = complement_input != 0;
  a.cache = (float *)state_cache->data;
  a.num_slots = state_cache->shape[0];
  a.slots = state_indices->data;
  a.slots_is64 = state_indices->dtype == GDP_I64;
  a.o = o->data; a.o_st = o->stride[0];
  hipError_t e;
  if (debug_validate()) {
    ValidateArgs va;
    std::memset(&va, 0, sizeof va);
    va.slots = a.slots; va.slots_is64 = a.slots_is64; va.nslots_given = N; va.num_slots = a.num_slots;
    if ((e = launch_validate(va, (hipStream_t)stream)) != hipSuccess)
      return fail(GDP_EHIP, "validation launch: %s", hipGetErrorString(e));
  }
  e = launch_scan_decode(a, float_type(x->dtype), float_type(g_log->dtype), (hipStream_t)stream);
  if (e != hipSuccess) return fail(GDP_EHIP, "decode launch: %s", hipGetErrorString(e));
  return GDP_OK;
}

int gdp_gated_scan_backward(const gdp_tensor *x, const gdp_tensor *g_log, const gdp_tensor *cu_seqlens,
                            int32_t complement_input, const gdp_tensor *initial_state,
                            const gdp_tensor *checkpoints, const gdp_tensor *d_o,
                            const gdp_tensor *d_final_state, const gdp_tensor *dx, const gdp_tensor *dg_log,
                            const gdp_tensor *d_initial_state, void *workspace, size_t workspace_bytes,
                            void *stream) {
  g_last_error.clear();
  if (!present(x) || !present(g_log) || !present(d_o)) return fail(GDP_EINVAL, "x, g_log and d_o are required");
  if (!present(dx) || !present(dg_log)) return fail(GDP_EINVAL, "dx and dg_log are required");
  if (!present(cu_seqlens)) return fail(GDP_EINVAL, "cu_seqlens is required (varlen input only)");
  if (x->ndim != 2) return fail(GDP_EINVAL, "x must be [T, D]");
  int rc;
  if ((rc = check_cu(cu_seqlens))) return rc;
  const int64_t T = x->shape[0], D = x->shape[1], N = cu_seqlens->shape[0] - 1;
  if (D < 1) return fail(GDP_EINVAL, "x needs at least one channel");
  if ((rc = check_scan_types(x, g_log))) return rc;
  if (d_o->dtype != x->dtype) return fail(GDP_EUNSUPPORTED, "x and d_o must share one dtype");
  if (dx->dtype != GDP_F32 && dx->dtype != x->dtype) return fail(GDP_EUNSUPPORTED, "dx must be float32 or x's dtype");
  if (dg_log->dtype != GDP_F32 && dg_log->dtype != g_log->dtype)
    return fail(GDP_EUNSUPPORTED, "dg_log must be float32 or g_log's dtype");
  if ((rc = check_rows(x, "x", T, D)) || (rc = check_rows(g_log, "g_log", T, D)) ||
      (rc = check_rows(d_o, "d_o", T, D)) || (rc = check_rows(dx, "dx", T, D)) ||
      (rc = check_rows(dg_log, "dg_log", T, D)) || (rc = check_row_overlap(dx, "dx")) ||
      (rc = check_row_overlap(dg_log, "dg_log")))
    return rc;
  if (!scan_served(T, N, D))
    return fail(GDP_EUNSUPPORTED, "T=%lld, N=%lld, D=%lld is past the launch limits", (long long)T, (long long)N,
                (long long)D);
  const bool init = present(initial_state), points = present(checkpoints), dfin = present(d_final_state),
             dinit = present(d_initial_state);
  if (init && (rc = check_states(initial_state, "initial_state", N, D))) return rc;
  if (points && (rc = check_states(checkpoints, "checkpoints", checkpoint_rows(T), D))) return rc;
  if (dfin && (rc = check_states(d_final_state, "d_final_state", N, D))) return rc;
  if (dinit && (rc = check_states(d_initial_state, "d_initial_state", N, D))) return rc;
  const size_t need = gdp_gated_scan_backward_workspace_bytes(T, N, D);
  if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const Range ins[] = {range_of(x, "x"), range_of(g_log, "g_log"), range_of(cu_seqlens, "cu_seqlens"),
                       range_of(initial_state, "initial_state"), range_of(checkpoints, "checkpoints"),
                       range_of(d_o, "d_o"), range_of(d_final_state, "d_final_state")};
  const Range outs[] = {range_of(dx, "dx"), range_of(dg_log, "dg_log"), range_of(d_initial_state, "d_initial_state"),
                        workspace_range(workspace, need)};
  if ((rc = check_alias(ins, outs))) return rc;

  ScanArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = x->data; a.x_st = x->stride[0];
  a.g = g_log->data; a.g_st = g_log->stride[0];
  a.cu = cu_seqlens->data; a.cu_is64 = cu_seqlens->dtype == GDP_I64;
  a.T = T; a.N = N; a.D = D;
  a.complement = complement_input != 0;
  a.s0 = init ? (const float *)initial_state->data : nullptr;
  a.ws = workspace;
  const int xt = float_type(x->dtype), gt = float_type(g_log->dtype);
  hipError_t e;
  if (debug_validate()) {
    ValidateArgs va;
    std::memset(&va, 0, sizeof va);
    va.cu = a.cu; va.cu_is64 = a.cu_is64; va.N = N; va.T = T;
    if ((e = launch_validate(va, (hipStream_t)stream)) != hipSuccess)
      return fail(GDP_EHIP, "validation launch: %s", hipGetErrorString(e));
  }
  if (points) {
    a.checkpoints = (float *)checkpoints->data;
  } else {
    // the states at the checkpoints again, into the workspace behind the scan's words
    a.checkpoints = (float *)((char *)workspace + scan_state_bytes(T, D, SCAN_ROWS));
    if ((e = launch_scan(a, xt, gt, (hipStream_t)stream)) != hipSuccess)
      return fail(GDP_EHIP, "scan launch: %s", hipGetErrorString(e));
  }
  a.dout = d_o->data; a.do_st = d_o->stride[0];
  a.dfinal = dfin ? (const float *)d_final_state->data : nullptr;
  a.dx = dx->data; a.dx_st = dx->stride[0]; a.dx_f32 = dx->dtype == GDP_F32;
  a.dg = dg_log->data; a.dg_st = dg_log->stride[0]; a.dg_f32 = dg_log->dtype == GDP_F32;
  a.ds0 = dinit ? (float *)d_initial_state->data : nullptr;
  if ((e = launch_scan_backward(a, xt, gt, (hipStream_t)stream)) != hipSuccess)
    return fail(GDP_EHIP, "backward launch: %s", hipGetErrorString(e));
  return GDP_OK;
}

size_t gdp_group_norm_backward_workspace_bytes(int64_t T, int64_t G, int64_t V) {
  if (T < 0 || G < 1 || V < 1 || V > NORM_MAX_SIZE || G > NORM_MAX_GROUPS) return 0;
  return align256(norm_backward_bytes(T, G, V));
}

namespace {

// Checks the operands that both directions of the norm share and fills them in.
int norm_args(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, const gdp_tensor *gate,
              int32_t activation, int32_t subtract_mean, float eps, NormArgs *a) {
  if (x->ndim != 3) return fail(GDP_EINVAL, "x must be [T, G, V]");
  const int64_t T = x->shape[0], G = x->shape[1], V = x->shape[2];
  if (G < 1 || V < 1) return fail(GDP_EINVAL, "the group count and group size must be positive");
  if (!is_float(x->dtype)) return fail(GDP_EUNSUPPORTED, "x must be float32, bfloat16 or float16");
  if (V > NORM_MAX_SIZE || G > NORM_MAX_GROUPS)
    return fail(GDP_EUNSUPPORTED, "more than 65535 groups, or 16384 channels in a group, are not served (G=%lld, V=%lld)",
                (long long)G, (long long)V);
  if (activation != GDP_ACT_NONE && activation != GDP_ACT_SILU && activation != GDP_ACT_SIGMOID)
    return fail(GDP_EINVAL, "unknown activation %d", activation);
  // (the kernels' 1 / sqrt takes a subnormal variance for 0)
  if (!(eps >= FLT_MIN) || std::isinf(eps)) return fail(GDP_EINVAL, "eps must be at least 2^-126, and finite");
  const int64_t s3[3] = {T, G, V}, s2[2] = {G, V}, s1[1] = {V};
  int rc;
  if ((rc = check_shape(x, "x", 3, s3))) return rc;
  if (!nonneg_strides(x)) return fail(GDP_EINVAL, "x: negative strides are not supported");
  const gdp_tensor *first = nullptr;
  for (const gdp_tensor *t : {weight, bias}) {
    if (!present(t)) continue;
    const char *name = t == weight ? "weight" : "bias";
    if (t->ndim != 1 && t->ndim != 2) return fail(GDP_EINVAL, "%s must be [V] or [G, V]", name);
    if ((rc = check_shape(t, name, t->ndim, t->ndim == 1 ? s1 : s2))) return rc;
    if (!contiguous(t)) return fail(GDP_EINVAL, "%s must be contiguous", name);
    if (t->dtype != GDP_F32 && t->dtype != x->dtype)
      return fail(GDP_EUNSUPPORTED, "%s must be float32 or x's dtype", name);
    if (first && (first->ndim != t->ndim || first->dtype != t->dtype))
      return fail(GDP_EINVAL, "weight and bias must share one shape and dtype");
    first = t;
  }
  if (present(gate)) {
    if ((rc = check_shape(gate, "gate", 3, s3))) return rc;
    if (gate->dtype != x->dtype) return fail(GDP_EUNSUPPORTED, "gate must have x's dtype");
    if (!nonneg_strides(gate)) return fail(GDP_EINVAL, "gate: negative strides are not supported");
  }
  std::memset(a, 0, sizeof *a);
  a->x = x->data; a->x_st = x->stride[0]; a->x_sh = x->stride[1];
  a->w = present(weight) ? weight->data : nullptr;
  a->b = present(bias) ? bias->data : nullptr;
  a->w_type = first ? float_type(first->dtype) : EL_F32;
  a->w_sh = first && first->ndim == 2 ? V : 0;
  if (present(gate)) { a->z = gate->data; a->z_st = gate->stride[0]; a->z_sh = gate->stride[1]; }
  a->T = T; a->G = (int)G; a->V = (int)V;
  a->act = activation; a->center = subtract_mean != 0; a->eps = eps;
  return GDP_OK;
}

// An output [T, G, V] of x's dtype whose elements are distinct.
int check_norm_output(const gdp_tensor *t, const char *name, const gdp_tensor *x) {
  const int64_t s3[3] = {x->shape[0], x->shape[1], x->shape[2]};
  if (int rc = check_shape(t, name, 3, s3)) return rc;
  if (t->dtype != x->dtype) return fail(GDP_EUNSUPPORTED, "%s must have x's dtype", name);
  if (!nonneg_strides(t)) return fail(GDP_EINVAL, "%s: negative strides are not supported", name);
  const int64_t T = s3[0], G = s3[1], V = s3[2], st = t->stride[0], sh = t->stride[1];
  // distinct in either nesting: groups within tokens, or tokens within groups
  const bool within = (G == 1 || sh >= V) && (T <= 1 || st >= (G - 1) * sh + V);
  const bool across = (T <= 1 || st >= V) && (G == 1 || sh >= (T - 1) * st + V);
  if (!within && !across) return fail(GDP_EALIAS, "%s: its elements overlap", name);
  return GDP_OK;
}

}  // namespace

int gdp_group_norm(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, const gdp_tensor *gate,
                   int32_t activation, int32_t subtract_mean, float eps, const gdp_tensor *y, void *stream) {
  g_last_error.clear();
  if (!present(x) || !present(y)) return fail(GDP_EINVAL, "x and y are required");
  NormArgs a;
  int rc;
  if ((rc = norm_args(x, weight, bias, gate, activation, subtract_mean, eps, &a))) return rc;
  if ((rc = check_norm_output(y, "y", x))) return rc;
  const Range ins[] = {range_of(x, "x"), range_of(weight, "weight"), range_of(bias, "bias"), range_of(gate, "gate")};
  const Range outs[] = {range_of(y, "y")};
  if ((rc = check_alias(ins, outs))) return rc;
  a.y = y->data; a.y_st = y->stride[0]; a.y_sh = y->stride[1];
  const hipError_t e = launch_norm(a, float_type(x->dtype), (hipStream_t)stream);
  if (e != hipSuccess) return fail(GDP_EHIP, "norm launch: %s", hipGetErrorString(e));
  return GDP_OK;
}

int gdp_group_norm_backward(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias,
                            const gdp_tensor *gate, int32_t activation, int32_t subtract_mean, float eps,
                            const gdp_tensor *d_y, const gdp_tensor *dx, const gdp_tensor *dweight,
                            const gdp_tensor *dbias, const gdp_tensor *dgate, void *workspace,
                            size_t workspace_bytes, void *stream) {
  g_last_error.clear();
  if (!present(x) || !present(d_y) || !present(dx)) return fail(GDP_EINVAL, "x, d_y and dx are required");
  NormArgs a;
  int rc;
  if ((rc = norm_args(x, weight, bias, gate, activation, subtract_mean, eps, &a))) return rc;
  const int64_t T = x->shape[0], G = x->shape[1], V = x->shape[2];
  const int64_t s3[3] = {T, G, V};
  if ((rc = check_shape(d_y, "d_y", 3, s3))) return rc;
  if (d_y->dtype != x->dtype) return fail(GDP_EUNSUPPORTED, "d_y must have x's dtype");
  if (!nonneg_strides(d_y)) return fail(GDP_EINVAL, "d_y: negative strides are not supported");
  if ((rc = check_norm_output(dx, "dx", x))) return rc;
  if (present(gate) != present(dgate)) return fail(GDP_EINVAL, "gate and dgate go together");
  if (present(dgate) && (rc = check_norm_output(dgate, "dgate", x))) return rc;
  if (present(weight) != present(dweight)) return fail(GDP_EINVAL, "weight and dweight go together");
  if (present(bias) != present(dbias)) return fail(GDP_EINVAL, "bias and dbias go together");
  const gdp_tensor *params[2] = {weight, bias}, *grads[2] = {dweight, dbias};
  for (int i = 0; i < 2; ++i) {
    if (!present(params[i])) continue;
    const char *name = i == 0 ? "dweight" : "dbias";
    if ((rc = check_shape(grads[i], name, params[i]->ndim, params[i]->shape))) return rc;
    if (grads[i]->dtype != GDP_F32) return fail(GDP_EUNSUPPORTED, "%s must be float32", name);
    if (!contiguous(grads[i])) return fail(GDP_EINVAL, "%s must be contiguous", name);
  }
  const bool sums = present(weight) || present(bias);
  const size_t need = sums ? gdp_group_norm_backward_workspace_bytes(T, G, V) : 0;
  if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const Range ins[] = {range_of(x, "x"), range_of(weight, "weight"), range_of(bias, "bias"), range_of(gate, "gate"),
                       range_of(d_y, "d_y")};
  const Range outs[] = {range_of(dx, "dx"), range_of(dgate, "dgate"), range_of(dweight, "dweight"),
                        range_of(dbias, "dbias"), workspace_range(workspace, need)};
  if ((rc = check_alias(ins, outs))) return rc;
  a.dy = d_y->data; a.dy_st = d_y->stride[0]; a.dy_sh = d_y->stride[1];
  a.dx = dx->data; a.dx_st = dx->stride[0]; a.dx_sh = dx->stride[1];
  if (present(dgate)) { a.dz = dgate->data; a.dz_st = dgate->stride[0]; a.dz_sh = dgate->stride[1]; }
  a.dw = present(dweight) ? (float *)dweight->data : nullptr;
  a.db = present(dbias) ? (float *)dbias->data : nullptr;
  a.ws = (float *)workspace;
  const hipError_t e = launch_norm_backward(a, float_type(x->dtype), (hipStream_t)stream);
  if (e != hipSuccess) return fail(GDP_EHIP, "norm backward launch: %s", hipGetErrorString(e));
  return GDP_OK;
}

}  // extern "C"
