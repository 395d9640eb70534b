// gdp_layer_check.h -- host-side argument checks shared by the C ABI of the layers
// (gdp_layer_api.cpp) and of what stands around them (gdp_block_api.cpp).  Not installed.
#pragma once

#include <cstdint>

#include "gdp.h"
#include "gdp_check.h"
#include "gdp_launch.h"

namespace gdp {

inline int float_type(int32_t dt) { return dt == GDP_F32 ? EL_F32 : (dt == GDP_BF16 ? EL_BF16 : EL_F16); }
inline bool is_float(int32_t dt) { return dt == GDP_F32 || dt == GDP_BF16 || dt == GDP_F16; }
inline bool is_index(int32_t dt) { return dt == GDP_I32 || dt == GDP_I64; }

// A [R, C] operand: exact shape, inner dimension contiguous, no negative strides.
inline int check_rows(const gdp_tensor *t, const char *name, int64_t R, int64_t C) {
  const int64_t s[2] = {R, C};
  if (int rc = check_shape(t, name, 2, s)) return rc;
  if (!nonneg_strides(t)) return fail(GDP_EINVAL, "%s: negative strides are not supported", name);
  return GDP_OK;
}

// Rows of an output must not share elements.
inline int check_row_overlap(const gdp_tensor *t, const char *name) {
  if (t->shape[0] > 1 && t->stride[0] < t->shape[1])
    return fail(GDP_EALIAS, "%s: its rows overlap (row stride %lld, %lld columns)", name, (long long)t->stride[0],
                (long long)t->shape[1]);
  return GDP_OK;
}

// A float32 contiguous [R, C] state buffer (R < 0: any).
inline int check_states(const gdp_tensor *t, const char *name, int64_t R, int64_t C) {
  const int64_t s[2] = {R, C};
  if (int rc = check_shape(t, name, 2, s)) return rc;
  if (t->dtype != GDP_F32) return fail(GDP_EUNSUPPORTED, "%s must be float32", name);
  if (!contiguous(t)) return fail(GDP_EINVAL, "%s must be contiguous", name);
  return GDP_OK;
}

inline int check_cu(const gdp_tensor *cu) {
  if (cu->ndim != 1 || cu->shape[0] < 1 || !contiguous(cu))
    return fail(GDP_EINVAL, "cu_seqlens must be a contiguous [N+1] vector");
  if (!is_index(cu->dtype)) return fail(GDP_EINVAL, "cu_seqlens must be int32 or int64");
  return GDP_OK;
}

inline int check_indices(const gdp_tensor *slots, int64_t N) {
  const int64_t s[1] = {N};
  if (!is_index(slots->dtype)) return fail(GDP_EINVAL, "state_indices must be int32 or int64");
  return check_shape(slots, "state_indices", 1, s);
}

inline int check_slots(const gdp_tensor *cache, const gdp_tensor *slots, int64_t N, int64_t D) {
  if (int rc = check_states(cache, "state_cache", -1, D)) return rc;
  return check_indices(slots, N);
}

// No output overlaps an input or another output.
template <int NI, int NO> int check_alias(const Range (&ins)[NI], const Range (&outs)[NO]) {
  for (const Range &ro : outs)
    for (const Range &ri : ins)
      if (overlap(ro, ri)) return fail(GDP_EALIAS, "%s overlaps input %s", ro.name, ri.name);
  for (int i = 0; i < NO; ++i)
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return fail(GDP_EALIAS, "%s overlaps %s", outs[i].name, outs[j].name);
  return GDP_OK;
}

inline int check_workspace(const void *ws, size_t given, size_t need) {
  if (need == 0) return GDP_OK;
  if (!ws || given < need) return fail(GDP_EWORKSPACE, "workspace of %zu bytes given, %zu needed", given, need);
  if ((uintptr_t)ws & 255) return fail(GDP_EWORKSPACE, "workspace must be 256-byte aligned");
  return GDP_OK;
}

inline Range range_if(bool use, const gdp_tensor *t, const char *name) { return use ? range_of(t, name) : Range{0, 0, name}; }

inline Range workspace_range(const void *ws, size_t bytes) {
  return Range{(uintptr_t)ws, (uintptr_t)ws + bytes, "workspace"};
}

}  // namespace gdp
