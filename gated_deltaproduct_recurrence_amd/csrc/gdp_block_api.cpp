// gdp_block_api.cpp -- C ABI of the short convolution, of the selective scan and of
// the norms around a block (declared in include/gdp.h).  As in gdp_api.cpp: host-side
// validation of shapes, dtypes, strides and pointer ranges, then launches on the
// caller's stream.

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstring>

#include "gdp.h"
#include "gdp_block.h"
#include "gdp_check.h"
#include "gdp_layer_check.h"

using namespace gdp;

namespace {

// A contiguous parameter of the shape `s`, float32 or x's dtype.
int check_param(const gdp_tensor *t, const char *name, int ndim, const int64_t *s, int32_t x_type) {
  if (int rc = check_shape(t, name, ndim, s)) return rc;
  if (!contiguous(t)) return fail(GDP_EINVAL, "%s must be contiguous", name);
  if (t->dtype != GDP_F32 && t->dtype != x_type)
    return fail(GDP_EUNSUPPORTED, "%s must be float32 or x's dtype", name);
  return GDP_OK;
}

// A contiguous tensor of the shape `s` (negative entries: any) and dtype.
int check_packed(const gdp_tensor *t, const char *name, int ndim, const int64_t *s, int32_t dtype) {
  if (int rc = check_shape(t, name, ndim, s)) return rc;
  if (t->dtype != dtype)
    return fail(GDP_EUNSUPPORTED, "%s must be %s", name, dtype == GDP_F32 ? "float32" : "of the input's dtype");
  if (!contiguous(t)) return fail(GDP_EINVAL, "%s must be contiguous", name);
  return GDP_OK;
}

// An output [R, C] of a dtype, its rows distinct.
int check_output(const gdp_tensor *t, const char *name, int64_t R, int64_t C, int32_t dtype, const char *whose) {
  if (int rc = check_rows(t, name, R, C)) return rc;
  if (t->dtype != dtype) return fail(GDP_EUNSUPPORTED, "%s must have %s dtype", name, whose);
  return check_row_overlap(t, name);
}

// (before a channel count is held in 32 bits)
int check_channels(int64_t D) {
  if (D > BLOCK_MAX_CHANNELS)
    return fail(GDP_EUNSUPPORTED, "more than %lld channels are not served (D=%lld)", (long long)BLOCK_MAX_CHANNELS,
                (long long)D);
  return GDP_OK;
}

// GDP_DEBUG_VALIDATE: the device checks of cu_seqlens and the slots
int validate(const void *cu, int cu_is64, int64_t N, int64_t T, const void *slots, int slots_is64, int64_t num_slots,
             void *stream) {
  if (!debug_validate()) return GDP_OK;
  ValidateArgs va;
  std::memset(&va, 0, sizeof va);
  va.cu = cu; va.cu_is64 = cu_is64; va.N = cu ? N : 0; va.T = T;
  va.slots = slots; va.slots_is64 = slots_is64; va.nslots_given = slots ? N : 0; va.num_slots = num_slots;
  const hipError_t e = launch_validate(va, (hipStream_t)stream);
  return e == hipSuccess ? GDP_OK : fail(GDP_EHIP, "validation launch: %s", hipGetErrorString(e));
}

int launched(hipError_t e, const char *what) {
  return e == hipSuccess ? GDP_OK : fail(GDP_EHIP, "%s launch: %s", what, hipGetErrorString(e));
}

// ------------------------------------------------------------ short convolution

// Checks and fills in what the calls over sequences and the single-token step share.
int conv_args(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, int32_t activation, ConvArgs *a) {
  if (!present(x) || !present(weight)) return fail(GDP_EINVAL, "x and weight are required");
  if (x->ndim != 2) return fail(GDP_EINVAL, "x must be [T, D]");
  if (weight->ndim != 2) return fail(GDP_EINVAL, "weight must be [D, W]");
  const int64_t T = x->shape[0], D = x->shape[1], W = weight->shape[1];
  if (D < 1) return fail(GDP_EINVAL, "x needs at least one channel");
  int rc;
  if ((rc = check_channels(D))) return rc;
  if (!is_float(x->dtype)) return fail(GDP_EUNSUPPORTED, "x must be float32, bfloat16 or float16");
  if (W < 2 || W > CONV_MAX_TAPS)
    return fail(GDP_EUNSUPPORTED, "2 to %d taps are served, got %lld", CONV_MAX_TAPS, (long long)W);
  if (activation != GDP_ACT_NONE && activation != GDP_ACT_SILU && activation != GDP_ACT_SIGMOID)
    return fail(GDP_EINVAL, "unknown activation %d", activation);
  const int64_t ws[2] = {D, W}, bs[1] = {D};
  if ((rc = check_rows(x, "x", T, D)) || (rc = check_param(weight, "weight", 2, ws, x->dtype))) return rc;
  if (present(bias)) {
    if ((rc = check_param(bias, "bias", 1, bs, x->dtype))) return rc;
    if (bias->dtype != weight->dtype) return fail(GDP_EINVAL, "weight and bias must share one dtype");
  }
  std::memset(a, 0, sizeof *a);
  a->x = x->data; a->x_st = x->stride[0];
  a->w = weight->data;
  a->b = present(bias) ? bias->data : nullptr;
  a->w_type = float_type(weight->dtype);
  a->D = (int)D; a->W = (int)W;
  a->act = activation;
  return GDP_OK;
}

int conv_sequences(const gdp_tensor *x, const gdp_tensor *cu, const gdp_tensor *initial_state, ConvArgs *a) {
  if (!present(cu)) return fail(GDP_EINVAL, "cu_seqlens is required (varlen input only)");
  int rc;
  if ((rc = check_cu(cu))) return rc;
  const int64_t T = x->shape[0], N = cu->shape[0] - 1;
  if (!conv_served(T, N, a->D))
    return fail(GDP_EUNSUPPORTED, "T=%lld, N=%lld, D=%d is past the launch limits", (long long)T, (long long)N, a->D);
  a->T = (int)T; a->N = (int)N;
  a->cu = cu->data; a->cu_is64 = cu->dtype == GDP_I64;
  if (present(initial_state)) {
    const int64_t s[3] = {N, a->W - 1, a->D};
    if ((rc = check_packed(initial_state, "initial_state", 3, s, x->dtype))) return rc;
    a->s0 = initial_state->data;
  }
  return GDP_OK;
}

int conv_slots(const gdp_tensor *x, const gdp_tensor *cache, const gdp_tensor *slots, int64_t N, ConvArgs *a) {
  const int64_t s[3] = {-1, a->W - 1, a->D};
  int rc;
  if ((rc = check_packed(cache, "state_cache", 3, s, x->dtype)) || (rc = check_indices(slots, N))) return rc;
  a->cache = cache->data;
  a->num_slots = cache->shape[0];
  a->slots = slots->data;
  a->slots_is64 = slots->dtype == GDP_I64;
  return GDP_OK;
}

}  // namespace

extern "C" {

int gdp_short_conv(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, int32_t activation,
                   const gdp_tensor *cu_seqlens, const gdp_tensor *initial_state, int32_t output_final_state,
                   const gdp_tensor *state_cache, const gdp_tensor *state_indices, const gdp_tensor *y,
                   const gdp_tensor *final_state, void *stream) {
  g_last_error.clear();
  ConvArgs a;
  int rc;
  if (!present(y)) return fail(GDP_EINVAL, "y is required");
  if ((rc = conv_args(x, weight, bias, activation, &a)) || (rc = conv_sequences(x, cu_seqlens, initial_state, &a)) ||
      (rc = check_output(y, "y", a.T, a.D, x->dtype, "x's")))
    return rc;
  const bool sink = present(state_cache);
  if (output_final_state) {
    if (!present(final_state)) return fail(GDP_EINVAL, "output_final_state needs a final_state buffer");
    const int64_t s[3] = {a.N, a.W - 1, a.D};
    if ((rc = check_packed(final_state, "final_state", 3, s, x->dtype))) return rc;
    a.final_state = final_state->data;
  }
  if (sink != present(state_indices)) return fail(GDP_EINVAL, "state_cache and state_indices go together");
  if (sink && (rc = conv_slots(x, state_cache, state_indices, a.N, &a))) return rc;
  const Range ins[] = {range_of(x, "x"), range_of(weight, "weight"), range_of(bias, "bias"),
                       range_of(cu_seqlens, "cu_seqlens"), range_of(initial_state, "initial_state"),
                       range_if(sink, state_indices, "state_indices")};
  const Range outs[] = {range_of(y, "y"), range_if(output_final_state != 0, final_state, "final_state"),
                        range_if(sink, state_cache, "state_cache")};
  if ((rc = check_alias(ins, outs))) return rc;
  a.y = y->data; a.y_st = y->stride[0];
  if ((rc = validate(a.cu, a.cu_is64, a.N, a.T, a.slots, a.slots_is64, a.num_slots, stream))) return rc;
  return launched(launch_conv(a, float_type(x->dtype), (hipStream_t)stream), "convolution");
}

int gdp_short_conv_decode(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, int32_t activation,
                          const gdp_tensor *state_cache, const gdp_tensor *state_indices, const gdp_tensor *y,
                          void *stream) {
  g_last_error.clear();
  ConvArgs a;
  int rc;
  if (!present(y)) return fail(GDP_EINVAL, "y is required");
  if (!present(state_cache) || !present(state_indices))
    return fail(GDP_EINVAL, "state_cache and state_indices are required");
  if ((rc = conv_args(x, weight, bias, activation, &a))) return rc;
  const int64_t N = x->shape[0];
  if ((rc = check_output(y, "y", N, a.D, x->dtype, "x's")) ||
      (rc = conv_slots(x, state_cache, state_indices, N, &a)))
    return rc;
  if (!conv_served(0, N, a.D))
    return fail(GDP_EUNSUPPORTED, "N=%lld, D=%d is past the launch limits", (long long)N, a.D);
  a.N = (int)N;
  const Range ins[] = {range_of(x, "x"), range_of(weight, "weight"), range_of(bias, "bias"),
                       range_of(state_indices, "state_indices")};
  const Range outs[] = {range_of(y, "y"), range_of(state_cache, "state_cache")};
  if ((rc = check_alias(ins, outs))) return rc;
  a.y = y->data; a.y_st = y->stride[0];
  if ((rc = validate(nullptr, 0, N, 0, a.slots, a.slots_is64, a.num_slots, stream))) return rc;
  return launched(launch_conv_decode(a, float_type(x->dtype), (hipStream_t)stream), "convolution step");
}

size_t gdp_short_conv_backward_workspace_bytes(int64_t T, int64_t N, int64_t D, int64_t W) {
  if (T < 0 || N < 0 || D < 1 || W < 2 || W > CONV_MAX_TAPS || !conv_served(T, N, D)) return 0;
  return align256(conv_backward_bytes(T, N, D, W));
}

int gdp_short_conv_backward(const gdp_tensor *x, const gdp_tensor *weight, const gdp_tensor *bias, int32_t activation,
                            const gdp_tensor *cu_seqlens, const gdp_tensor *initial_state, const gdp_tensor *d_y,
                            const gdp_tensor *d_final_state, const gdp_tensor *dx, const gdp_tensor *dweight,
                            const gdp_tensor *dbias, const gdp_tensor *d_initial_state, void *workspace,
                            size_t workspace_bytes, void *stream) {
  g_last_error.clear();
  ConvArgs a;
  int rc;
  if (!present(d_y) || !present(dx) || !present(dweight)) return fail(GDP_EINVAL, "d_y, dx and dweight are required");
  if ((rc = conv_args(x, weight, bias, activation, &a)) || (rc = conv_sequences(x, cu_seqlens, initial_state, &a)) ||
      (rc = check_rows(d_y, "d_y", a.T, a.D)))
    return rc;
  if (d_y->dtype != x->dtype) return fail(GDP_EUNSUPPORTED, "x and d_y must share one dtype");
  if ((rc = check_output(dx, "dx", a.T, a.D, x->dtype, "x's"))) return rc;
  if (present(bias) != present(dbias)) return fail(GDP_EINVAL, "bias and dbias go together");
  if ((rc = check_packed(dweight, "dweight", 2, weight->shape, GDP_F32))) return rc;
  if (present(dbias) && (rc = check_packed(dbias, "dbias", 1, bias->shape, GDP_F32))) return rc;
  const int64_t s[3] = {a.N, a.W - 1, a.D};
  if (present(d_final_state) && (rc = check_packed(d_final_state, "d_final_state", 3, s, GDP_F32))) return rc;
  if (present(d_initial_state) && (rc = check_packed(d_initial_state, "d_initial_state", 3, s, GDP_F32))) return rc;
  const size_t need = gdp_short_conv_backward_workspace_bytes(a.T, a.N, a.D, a.W);
  if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const Range ins[] = {range_of(x, "x"), range_of(weight, "weight"), range_of(bias, "bias"),
                       range_of(cu_seqlens, "cu_seqlens"), range_of(initial_state, "initial_state"),
                       range_of(d_y, "d_y"), range_of(d_final_state, "d_final_state")};
  const Range outs[] = {range_of(dx, "dx"), range_of(dweight, "dweight"), range_of(dbias, "dbias"),
                        range_of(d_initial_state, "d_initial_state"), workspace_range(workspace, need)};
  if ((rc = check_alias(ins, outs))) return rc;
  a.dy = d_y->data; a.dy_st = d_y->stride[0];
  a.dfinal = present(d_final_state) ? (const float *)d_final_state->data : nullptr;
  a.dx = dx->data; a.dx_st = dx->stride[0];
  a.ds0 = present(d_initial_state) ? (float *)d_initial_state->data : nullptr;
  a.dw = (float *)dweight->data;
  a.db = present(dbias) ? (float *)dbias->data : nullptr;
  a.ws = (float *)workspace;
  if ((rc = validate(a.cu, a.cu_is64, a.N, a.T, nullptr, 0, 0, stream))) return rc;
  return launched(launch_conv_backward(a, float_type(x->dtype), (hipStream_t)stream), "convolution backward");
}

}  // extern "C"

// --------------------------------------------------------------- selective scan

namespace {

int select_args(const gdp_tensor *u, const gdp_tensor *dt, const gdp_tensor *A, const gdp_tensor *B,
                const gdp_tensor *C, const gdp_tensor *skip, const gdp_tensor *gate, const gdp_tensor *dt_bias,
                int32_t dt_softplus, SelectArgs *a) {
  if (!present(u) || !present(dt) || !present(A) || !present(B) || !present(C))
    return fail(GDP_EINVAL, "u, dt, A, B and C are required");
  if (u->ndim != 2) return fail(GDP_EINVAL, "u must be [T, D]");
  if (A->ndim != 2) return fail(GDP_EINVAL, "A must be [D, S]");
  if (B->ndim != 3) return fail(GDP_EINVAL, "B must be [T, G, S]");
  const int64_t T = u->shape[0], D = u->shape[1], S = A->shape[1], G = B->shape[1];
  if (D < 1) return fail(GDP_EINVAL, "u needs at least one channel");
  int rc;
  if ((rc = check_channels(D))) return rc;
  if (!is_float(u->dtype)) return fail(GDP_EUNSUPPORTED, "u must be float32, bfloat16 or float16");
  if (dt->dtype != GDP_F32 && dt->dtype != u->dtype) return fail(GDP_EUNSUPPORTED, "dt must be float32 or u's dtype");
  if (B->dtype != u->dtype || C->dtype != u->dtype) return fail(GDP_EUNSUPPORTED, "B and C must have u's dtype");
  if (S < 1 || S > SELECT_MAX_STATES)
    return fail(GDP_EUNSUPPORTED, "1 to %d states per channel are served, got %lld", SELECT_MAX_STATES, (long long)S);
  if (G < 1 || D % G != 0)
    return fail(GDP_EINVAL, "the %lld channels must be a multiple of the %lld groups of B and C", (long long)D, (long long)G);
  const int64_t as[2] = {D, S}, bs[3] = {T, G, S}, ds[1] = {D};
  if ((rc = check_rows(u, "u", T, D)) || (rc = check_rows(dt, "dt", T, D)) ||
      (rc = check_packed(A, "A", 2, as, GDP_F32)) || (rc = check_shape(B, "B", 3, bs)) ||
      (rc = check_shape(C, "C", 3, bs)))
    return rc;
  if (!nonneg_strides(B) || !nonneg_strides(C)) return fail(GDP_EINVAL, "B, C: negative strides are not supported");
  if (present(skip) && (rc = check_packed(skip, "skip", 1, ds, GDP_F32))) return rc;
  if (present(dt_bias) && (rc = check_packed(dt_bias, "dt_bias", 1, ds, GDP_F32))) return rc;
  if (present(gate)) {
    if ((rc = check_rows(gate, "gate", T, D))) return rc;
    if (gate->dtype != u->dtype) return fail(GDP_EUNSUPPORTED, "gate must have u's dtype");
  }
  std::memset(a, 0, sizeof *a);
  a->u = u->data; a->u_st = u->stride[0];
  a->dt = dt->data; a->dt_st = dt->stride[0];
  a->A = (const float *)A->data;
  a->B = B->data; a->B_st = B->stride[0]; a->B_sg = B->stride[1];
  a->C = C->data; a->C_st = C->stride[0]; a->C_sg = C->stride[1];
  a->skip = present(skip) ? (const float *)skip->data : nullptr;
  a->bias = present(dt_bias) ? (const float *)dt_bias->data : nullptr;
  if (present(gate)) { a->z = gate->data; a->z_st = gate->stride[0]; }
  a->D = (int)D; a->G = (int)G; a->S = (int)S;
  a->softplus = dt_softplus != 0;
  return GDP_OK;
}

int select_sequences(const gdp_tensor *u, const gdp_tensor *cu, const gdp_tensor *initial_state, SelectArgs *a) {
  if (!present(cu)) return fail(GDP_EINVAL, "cu_seqlens is required (varlen input only)");
  int rc;
  if ((rc = check_cu(cu))) return rc;
  const int64_t T = u->shape[0], N = cu->shape[0] - 1;
  if (!select_served(T, N, a->D, a->G, a->S))
    return fail(GDP_EUNSUPPORTED, "T=%lld, N=%lld, D=%d is past the launch limits", (long long)T, (long long)N, a->D);
  a->T = (int)T; a->N = (int)N;
  a->cu = cu->data; a->cu_is64 = cu->dtype == GDP_I64;
  if (present(initial_state)) {
    const int64_t s[3] = {N, a->D, a->S};
    if ((rc = check_packed(initial_state, "initial_state", 3, s, GDP_F32))) return rc;
    a->s0 = (const float *)initial_state->data;
  }
  return GDP_OK;
}

int select_slots(const gdp_tensor *cache, const gdp_tensor *slots, int64_t N, SelectArgs *a) {
  const int64_t s[3] = {-1, a->D, a->S};
  int rc;
  if ((rc = check_packed(cache, "state_cache", 3, s, GDP_F32)) || (rc = check_indices(slots, N))) return rc;
  a->cache = (float *)cache->data;
  a->num_slots = cache->shape[0];
  a->slots = slots->data;
  a->slots_is64 = slots->dtype == GDP_I64;
  return GDP_OK;
}

bool select_sizes_ok(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S) {
  return T >= 0 && N >= 0 && D >= 1 && G >= 1 && D % G == 0 && S >= 1 && S <= SELECT_MAX_STATES &&
         select_served(T, N, D, G, S);
}

int check_points(const gdp_tensor *points, const SelectArgs &a) {
  const int64_t s[3] = {a.T / SELECT_ROWS + a.N, a.S, a.D};
  return check_packed(points, "checkpoints", 3, s, GDP_F32);
}

}  // namespace

extern "C" {

size_t gdp_selective_scan_workspace_bytes(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S) {
  return select_sizes_ok(T, N, D, G, S) ? select_bytes(T, N, D, G, S) : 0;
}

int gdp_selective_scan(const gdp_tensor *u, const gdp_tensor *dt, const gdp_tensor *A, const gdp_tensor *B,
                       const gdp_tensor *C, const gdp_tensor *skip, const gdp_tensor *gate, const gdp_tensor *dt_bias,
                       int32_t dt_softplus, const gdp_tensor *cu_seqlens, const gdp_tensor *initial_state,
                       int32_t output_final_state, const gdp_tensor *state_cache, const gdp_tensor *state_indices,
                       int32_t return_checkpoints, const gdp_tensor *o, const gdp_tensor *final_state,
                       const gdp_tensor *checkpoints, void *workspace, size_t workspace_bytes, void *stream) {
  g_last_error.clear();
  SelectArgs a;
  int rc;
  if (!present(o)) return fail(GDP_EINVAL, "o is required");
  if ((rc = select_args(u, dt, A, B, C, skip, gate, dt_bias, dt_softplus, &a)) ||
      (rc = select_sequences(u, cu_seqlens, initial_state, &a)) ||
      (rc = check_output(o, "o", a.T, a.D, u->dtype, "u's")))
    return rc;
  const bool sink = present(state_cache);
  if (output_final_state) {
    if (!present(final_state)) return fail(GDP_EINVAL, "output_final_state needs a final_state buffer");
    const int64_t s[3] = {a.N, a.D, a.S};
    if ((rc = check_packed(final_state, "final_state", 3, s, GDP_F32))) return rc;
    a.final_state = (float *)final_state->data;
  }
  if (sink != present(state_indices)) return fail(GDP_EINVAL, "state_cache and state_indices go together");
  if (sink && (rc = select_slots(state_cache, state_indices, a.N, &a))) return rc;
  if (return_checkpoints) {
    if (!present(checkpoints)) return fail(GDP_EINVAL, "return_checkpoints needs a checkpoints buffer");
    if ((rc = check_points(checkpoints, a))) return rc;
    a.points = (float *)checkpoints->data;
  }
  const size_t need = gdp_selective_scan_workspace_bytes(a.T, a.N, a.D, a.G, a.S);
  if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const Range ins[] = {range_of(u, "u"), range_of(dt, "dt"), range_of(A, "A"), range_of(B, "B"), range_of(C, "C"),
                       range_of(skip, "skip"), range_of(gate, "gate"), range_of(dt_bias, "dt_bias"),
                       range_of(cu_seqlens, "cu_seqlens"), range_of(initial_state, "initial_state"),
                       range_if(sink, state_indices, "state_indices")};
  const Range outs[] = {range_of(o, "o"), range_if(output_final_state != 0, final_state, "final_state"),
                        range_if(sink, state_cache, "state_cache"),
                        range_if(return_checkpoints != 0, checkpoints, "checkpoints"),
                        workspace_range(workspace, need)};
  if ((rc = check_alias(ins, outs))) return rc;
  a.o = o->data; a.o_st = o->stride[0];
  a.ws = workspace;
  if ((rc = validate(a.cu, a.cu_is64, a.N, a.T, a.slots, a.slots_is64, a.num_slots, stream))) return rc;
  return launched(launch_select(a, float_type(u->dtype), float_type(dt->dtype), (hipStream_t)stream), "selective scan");
}

int gdp_selective_scan_decode(const gdp_tensor *u, const gdp_tensor *dt, const gdp_tensor *A, const gdp_tensor *B,
                              const gdp_tensor *C, const gdp_tensor *skip, const gdp_tensor *gate,
                              const gdp_tensor *dt_bias, int32_t dt_softplus, const gdp_tensor *state_cache,
                              const gdp_tensor *state_indices, const gdp_tensor *o, void *stream) {
  g_last_error.clear();
  SelectArgs a;
  int rc;
  if (!present(o)) return fail(GDP_EINVAL, "o is required");
  if (!present(state_cache) || !present(state_indices))
    return fail(GDP_EINVAL, "state_cache and state_indices are required");
  if ((rc = select_args(u, dt, A, B, C, skip, gate, dt_bias, dt_softplus, &a))) return rc;
  const int64_t N = u->shape[0];
  if ((rc = check_output(o, "o", N, a.D, u->dtype, "u's")) || (rc = select_slots(state_cache, state_indices, N, &a)))
    return rc;
  if (!select_served(0, N, a.D, a.G, a.S))
    return fail(GDP_EUNSUPPORTED, "N=%lld, D=%d is past the launch limits", (long long)N, a.D);
  a.N = (int)N;
  const Range ins[] = {range_of(u, "u"), range_of(dt, "dt"), range_of(A, "A"), range_of(B, "B"), range_of(C, "C"),
                       range_of(skip, "skip"), range_of(gate, "gate"), range_of(dt_bias, "dt_bias"),
                       range_of(state_indices, "state_indices")};
  const Range outs[] = {range_of(o, "o"), range_of(state_cache, "state_cache")};
  if ((rc = check_alias(ins, outs))) return rc;
  a.o = o->data; a.o_st = o->stride[0];
  if ((rc = validate(nullptr, 0, N, 0, a.slots, a.slots_is64, a.num_slots, stream))) return rc;
  return launched(launch_select_decode(a, float_type(u->dtype), float_type(dt->dtype), (hipStream_t)stream),
                  "selective scan step");
}

size_t gdp_selective_scan_backward_workspace_bytes(int64_t T, int64_t N, int64_t D, int64_t G, int64_t S,
                                                   int32_t with_checkpoints) {
  return select_sizes_ok(T, N, D, G, S) ? select_backward_bytes(T, N, D, G, S, with_checkpoints != 0) : 0;
}

int gdp_selective_scan_backward(const gdp_tensor *u, const gdp_tensor *dt, const gdp_tensor *A, const gdp_tensor *B,
                                const gdp_tensor *C, const gdp_tensor *skip, const gdp_tensor *gate,
                                const gdp_tensor *dt_bias, int32_t dt_softplus, const gdp_tensor *cu_seqlens,
                                const gdp_tensor *initial_state, const gdp_tensor *checkpoints, const gdp_tensor *d_o,
                                const gdp_tensor *d_final_state, const gdp_tensor *du, const gdp_tensor *ddt,
                                const gdp_tensor *dA, const gdp_tensor *dB, const gdp_tensor *dC,
                                const gdp_tensor *dskip, const gdp_tensor *dgate, const gdp_tensor *ddt_bias,
                                const gdp_tensor *d_initial_state, void *workspace, size_t workspace_bytes,
                                void *stream) {
  g_last_error.clear();
  SelectArgs a;
  int rc;
  if (!present(d_o)) return fail(GDP_EINVAL, "d_o is required");
  if (!present(du) || !present(ddt) || !present(dA) || !present(dB) || !present(dC))
    return fail(GDP_EINVAL, "du, ddt, dA, dB and dC are required");
  if ((rc = select_args(u, dt, A, B, C, skip, gate, dt_bias, dt_softplus, &a)) ||
      (rc = select_sequences(u, cu_seqlens, initial_state, &a)) || (rc = check_rows(d_o, "d_o", a.T, a.D)))
    return rc;
  if (d_o->dtype != u->dtype) return fail(GDP_EUNSUPPORTED, "u and d_o must share one dtype");
  if (present(skip) != present(dskip)) return fail(GDP_EINVAL, "skip and dskip go together");
  if (present(gate) != present(dgate)) return fail(GDP_EINVAL, "gate and dgate go together");
  if (present(dt_bias) != present(ddt_bias)) return fail(GDP_EINVAL, "dt_bias and ddt_bias go together");
  const int64_t bs[3] = {a.T, a.G, a.S}, ds[1] = {a.D}, ss[3] = {a.N, a.D, a.S};
  if ((rc = check_output(du, "du", a.T, a.D, u->dtype, "u's")) ||
      (rc = check_output(ddt, "ddt", a.T, a.D, dt->dtype, "dt's")) ||
      (rc = check_packed(dA, "dA", 2, A->shape, GDP_F32)) || (rc = check_packed(dB, "dB", 3, bs, u->dtype)) ||
      (rc = check_packed(dC, "dC", 3, bs, u->dtype)))
    return rc;
  if (present(dskip) && (rc = check_packed(dskip, "dskip", 1, ds, GDP_F32))) return rc;
  if (present(ddt_bias) && (rc = check_packed(ddt_bias, "ddt_bias", 1, ds, GDP_F32))) return rc;
  if (present(dgate) && (rc = check_output(dgate, "dgate", a.T, a.D, u->dtype, "u's"))) return rc;
  if (present(d_final_state) && (rc = check_packed(d_final_state, "d_final_state", 3, ss, GDP_F32))) return rc;
  if (present(d_initial_state) && (rc = check_packed(d_initial_state, "d_initial_state", 3, ss, GDP_F32))) return rc;
  const bool points = present(checkpoints);
  if (points && (rc = check_points(checkpoints, a))) return rc;
  const size_t need = gdp_selective_scan_backward_workspace_bytes(a.T, a.N, a.D, a.G, a.S, points);
  if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const Range ins[] = {range_of(u, "u"), range_of(dt, "dt"), range_of(A, "A"), range_of(B, "B"), range_of(C, "C"),
                       range_of(skip, "skip"), range_of(gate, "gate"), range_of(dt_bias, "dt_bias"),
                       range_of(cu_seqlens, "cu_seqlens"), range_of(initial_state, "initial_state"),
                       range_of(checkpoints, "checkpoints"), range_of(d_o, "d_o"),
                       range_of(d_final_state, "d_final_state")};
  const Range outs[] = {range_of(du, "du"), range_of(ddt, "ddt"), range_of(dA, "dA"), range_of(dB, "dB"),
                        range_of(dC, "dC"), range_of(dskip, "dskip"), range_of(dgate, "dgate"),
                        range_of(ddt_bias, "ddt_bias"), range_of(d_initial_state, "d_initial_state"),
                        workspace_range(workspace, need)};
  if ((rc = check_alias(ins, outs))) return rc;
  a.points = points ? (float *)checkpoints->data : nullptr;
  a.d_o = d_o->data; a.do_st = d_o->stride[0];
  a.dfinal = present(d_final_state) ? (const float *)d_final_state->data : nullptr;
  a.du = du->data; a.du_st = du->stride[0];
  a.ddt = ddt->data; a.ddt_st = ddt->stride[0];
  a.dA = (float *)dA->data;
  a.dB = dB->data; a.dC = dC->data;
  a.dskip = present(dskip) ? (float *)dskip->data : nullptr;
  a.dbias = present(ddt_bias) ? (float *)ddt_bias->data : nullptr;
  if (present(dgate)) { a.dz = dgate->data; a.dz_st = dgate->stride[0]; }
  a.ds0 = present(d_initial_state) ? (float *)d_initial_state->data : nullptr;
  a.ws = workspace;
  if ((rc = validate(a.cu, a.cu_is64, a.N, a.T, nullptr, 0, 0, stream))) return rc;
  return launched(launch_select_backward(a, float_type(u->dtype), float_type(dt->dtype), (hipStream_t)stream),
                  "selective scan backward");
}

}  // extern "C"

// ---------------------------------------------------------- norms around a block

namespace {

int resnorm_args(const gdp_tensor *x, const gdp_tensor *y, const gdp_tensor *post_weight, const gdp_tensor *pre_weight,
                 const gdp_tensor *gate, int32_t gate_activation, int32_t post_norm, int32_t pre_norm,
                 float residual_scale, float eps, ResNormArgs *a) {
  if (!present(x) || !present(y)) return fail(GDP_EINVAL, "x and y are required");
  if (y->ndim != 2) return fail(GDP_EINVAL, "y must be [T, D]");
  const int64_t T = y->shape[0], D = y->shape[1];
  if (D < 1) return fail(GDP_EINVAL, "y needs at least one channel");
  if (!is_float(y->dtype)) return fail(GDP_EUNSUPPORTED, "y must be float32, bfloat16 or float16");
  if (x->dtype != GDP_F32 && x->dtype != y->dtype) return fail(GDP_EUNSUPPORTED, "x must be float32 or of y's dtype");
  if (D > RESNORM_MAX_CHANNELS)
    return fail(GDP_EUNSUPPORTED, "more than %lld channels are not served (D=%lld)", (long long)RESNORM_MAX_CHANNELS,
                (long long)D);
  if (gate_activation != GDP_ACT_NONE && gate_activation != GDP_ACT_SILU && gate_activation != GDP_ACT_SIGMOID)
    return fail(GDP_EINVAL, "unknown activation %d", gate_activation);
  if (gate_activation != GDP_ACT_NONE && !present(gate)) return fail(GDP_EINVAL, "an activation needs a gate");
  // (the kernels' 1 / sqrt takes a subnormal mean square for 0)
  if (!(eps >= FLT_MIN) || std::isinf(eps)) return fail(GDP_EINVAL, "eps must be at least 2^-126, and finite");
  if (!std::isfinite(residual_scale)) return fail(GDP_EINVAL, "residual_scale must be finite");
  int rc;
  if ((rc = check_rows(x, "x", T, D)) || (rc = check_rows(y, "y", T, D))) return rc;
  const int64_t s[1] = {D};
  const gdp_tensor *first = nullptr;
  for (const gdp_tensor *t : {post_weight, pre_weight}) {
    if (!present(t)) continue;
    const char *name = t == post_weight ? "post_weight" : "pre_weight";
    if ((rc = check_shape(t, name, 1, s))) return rc;
    if (!contiguous(t)) return fail(GDP_EINVAL, "%s must be contiguous", name);
    if (t->dtype != GDP_F32 && t->dtype != y->dtype)
      return fail(GDP_EUNSUPPORTED, "%s must be float32 or of y's dtype", name);
    if (first && first->dtype != t->dtype) return fail(GDP_EINVAL, "post_weight and pre_weight must share one dtype");
    first = t;
  }
  if (present(pre_weight) && !pre_norm) return fail(GDP_EINVAL, "pre_weight needs pre_norm");
  if (present(gate)) {
    if ((rc = check_rows(gate, "gate", T, D))) return rc;
    if (gate->dtype != y->dtype) return fail(GDP_EUNSUPPORTED, "gate must have y's dtype");
  }
  std::memset(a, 0, sizeof *a);
  a->x = x->data; a->x_st = x->stride[0];
  a->y = y->data; a->y_st = y->stride[0];
  if (present(gate)) { a->z = gate->data; a->z_st = gate->stride[0]; }
  a->w_post = present(post_weight) ? post_weight->data : nullptr;
  a->w_pre = present(pre_weight) ? pre_weight->data : nullptr;
  a->w_type = first ? float_type(first->dtype) : EL_F32;
  a->T = T; a->D = (int)D;
  a->act = gate_activation; a->post = post_norm != 0; a->pre = pre_norm != 0;
  a->scale = residual_scale; a->eps = eps;
  return GDP_OK;
}

// the same elements: what a call may write over once it has read them
bool same_view(const gdp_tensor *p, const gdp_tensor *q) {
  return p->data == q->data && p->dtype == q->dtype && (p->shape[0] <= 1 || p->stride[0] == q->stride[0]);
}

}  // namespace

extern "C" {

int gdp_residual_norm(const gdp_tensor *x, const gdp_tensor *y, const gdp_tensor *post_weight,
                      const gdp_tensor *pre_weight, const gdp_tensor *gate, int32_t gate_activation, int32_t post_norm,
                      int32_t pre_norm, float residual_scale, float eps, const gdp_tensor *r, const gdp_tensor *n,
                      void *stream) {
  g_last_error.clear();
  ResNormArgs a;
  int rc;
  if ((rc = resnorm_args(x, y, post_weight, pre_weight, gate, gate_activation, post_norm, pre_norm, residual_scale, eps,
                         &a)))
    return rc;
  if (!present(r)) return fail(GDP_EINVAL, "r is required");
  if (present(n) != (pre_norm != 0)) return fail(GDP_EINVAL, "n and pre_norm go together");
  if ((rc = check_output(r, "r", a.T, a.D, x->dtype, "x's"))) return rc;
  if (present(n) && (rc = check_output(n, "n", a.T, a.D, y->dtype, "y's"))) return rc;
  const bool in_place = same_view(r, x);
  const Range ins[] = {range_if(!in_place, x, "x"), range_of(y, "y"), range_of(post_weight, "post_weight"),
                       range_of(pre_weight, "pre_weight"), range_of(gate, "gate")};
  const Range outs[] = {range_of(r, "r"), range_of(n, "n")};
  if ((rc = check_alias(ins, outs))) return rc;
  a.r = r->data; a.r_st = r->stride[0];
  if (present(n)) { a.n = n->data; a.n_st = n->stride[0]; }
  return launched(launch_resnorm(a, float_type(y->dtype), float_type(x->dtype), (hipStream_t)stream), "residual norm");
}

size_t gdp_residual_norm_backward_workspace_bytes(int64_t T, int64_t D) {
  if (T < 0 || D < 1 || D > RESNORM_MAX_CHANNELS) return 0;
  return align256(resnorm_backward_bytes(T, D));
}

int gdp_residual_norm_backward(const gdp_tensor *x, const gdp_tensor *y, const gdp_tensor *post_weight,
                               const gdp_tensor *pre_weight, const gdp_tensor *gate, int32_t gate_activation,
                               int32_t post_norm, int32_t pre_norm, float residual_scale, float eps,
                               const gdp_tensor *d_r, const gdp_tensor *d_n, const gdp_tensor *dx,
                               const gdp_tensor *dy, const gdp_tensor *dpost_weight, const gdp_tensor *dpre_weight,
                               const gdp_tensor *dgate, void *workspace, size_t workspace_bytes, void *stream) {
  g_last_error.clear();
  ResNormArgs a;
  int rc;
  if ((rc = resnorm_args(x, y, post_weight, pre_weight, gate, gate_activation, post_norm, pre_norm, residual_scale, eps,
                         &a)))
    return rc;
  if (!present(dx) || !present(dy)) return fail(GDP_EINVAL, "dx and dy are required");
  if (present(d_n) != (pre_norm != 0)) return fail(GDP_EINVAL, "d_n and pre_norm go together");
  if (!present(d_n) && !present(d_r)) return fail(GDP_EINVAL, "d_r is required without pre_norm");
  if (present(gate) != present(dgate)) return fail(GDP_EINVAL, "gate and dgate go together");
  if (present(post_weight) != present(dpost_weight))
    return fail(GDP_EINVAL, "post_weight and dpost_weight go together");
  if (present(pre_weight) != present(dpre_weight)) return fail(GDP_EINVAL, "pre_weight and dpre_weight go together");
  if (present(d_r)) {
    if ((rc = check_rows(d_r, "d_r", a.T, a.D))) return rc;
    if (d_r->dtype != x->dtype) return fail(GDP_EUNSUPPORTED, "d_r must have x's dtype");
  }
  if (present(d_n)) {
    if ((rc = check_rows(d_n, "d_n", a.T, a.D))) return rc;
    if (d_n->dtype != y->dtype) return fail(GDP_EUNSUPPORTED, "d_n must have y's dtype");
  }
  if ((rc = check_output(dx, "dx", a.T, a.D, x->dtype, "x's")) || (rc = check_output(dy, "dy", a.T, a.D, y->dtype, "y's")))
    return rc;
  if (present(dgate) && (rc = check_output(dgate, "dgate", a.T, a.D, y->dtype, "y's"))) return rc;
  const int64_t s[1] = {a.D};
  if (present(dpost_weight) && (rc = check_packed(dpost_weight, "dpost_weight", 1, s, GDP_F32))) return rc;
  if (present(dpre_weight) && (rc = check_packed(dpre_weight, "dpre_weight", 1, s, GDP_F32))) return rc;
  const bool sums = present(post_weight) || present(pre_weight);
  const size_t need = sums ? gdp_residual_norm_backward_workspace_bytes(a.T, a.D) : 0;
  if ((rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const Range ins[] = {range_of(x, "x"), range_of(y, "y"), range_of(post_weight, "post_weight"),
                       range_of(pre_weight, "pre_weight"), range_of(gate, "gate"), range_of(d_r, "d_r"),
                       range_of(d_n, "d_n")};
  const Range outs[] = {range_of(dx, "dx"), range_of(dy, "dy"), range_of(dgate, "dgate"),
                        range_of(dpost_weight, "dpost_weight"), range_of(dpre_weight, "dpre_weight"),
                        workspace_range(workspace, need)};
  if ((rc = check_alias(ins, outs))) return rc;
  if (present(d_r)) { a.dr = d_r->data; a.dr_st = d_r->stride[0]; }
  if (present(d_n)) { a.dn = d_n->data; a.dn_st = d_n->stride[0]; }
  a.dx = dx->data; a.dx_st = dx->stride[0];
  a.dy = dy->data; a.dy_st = dy->stride[0];
  if (present(dgate)) { a.dz = dgate->data; a.dz_st = dgate->stride[0]; }
  a.dw_post = present(dpost_weight) ? (float *)dpost_weight->data : nullptr;
  a.dw_pre = present(dpre_weight) ? (float *)dpre_weight->data : nullptr;
  a.ws = (float *)workspace;
  return launched(launch_resnorm_backward(a, float_type(y->dtype), float_type(x->dtype), (hipStream_t)stream),
                  "residual norm backward");
}

}  // extern "C"
