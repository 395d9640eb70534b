// gdp_check.h -- host-side argument checks shared by the C ABI's translation
// units (gdp_api.cpp, gdp_layer_api.cpp): the per-thread error message, shapes,
// strides and byte ranges.  Nothing here reads device memory.  Not installed.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <string>

#include "gdp.h"

namespace gdp {

// message of the last failed call of this thread (gdp_last_error)
inline thread_local std::string g_last_error;

inline int fail(int code, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

inline bool present(const gdp_tensor *t) { return t != nullptr && t->data != nullptr; }

// GDP_DEBUG_VALIDATE=1: launch the device checks of cu_seqlens and the state indices
inline bool debug_validate() {
  const char *s = std::getenv("GDP_DEBUG_VALIDATE");
  return s != nullptr && s[0] == '1' && s[1] == '\0';
}

inline int elem_size(int32_t dt) {
  switch (dt) {
    case GDP_F32: return 4;
    case GDP_BF16: return 2;
    case GDP_I32: return 4;
    case GDP_I64: return 8;
    case GDP_F16: return 2;
    default: return 0;
  }
}

// Checks ndim, the exact shape and that the innermost stride is 1 (of one element it
// does not matter, and torch keeps any there).
inline int check_shape(const gdp_tensor *t, const char *name, int ndim, const int64_t *shape) {
  if (t->ndim != ndim) return fail(GDP_EINVAL, "%s: expected %d dims, got %d", name, ndim, t->ndim);
  for (int d = 0; d < ndim; ++d)
    if (shape[d] >= 0 && t->shape[d] != shape[d])
      return fail(GDP_EINVAL, "%s: dim %d is %lld, expected %lld", name, d, (long long)t->shape[d],
                  (long long)shape[d]);
  if (ndim > 0 && t->shape[ndim - 1] != 1 && t->stride[ndim - 1] != 1)
    return fail(GDP_EINVAL, "%s: innermost dimension must be contiguous", name);
  return GDP_OK;
}

inline bool contiguous(const gdp_tensor *t) {
  int64_t expect = 1;
  for (int d = t->ndim - 1; d >= 0; --d) {
    if (t->shape[d] != 1 && t->stride[d] != expect) return false;
    expect *= t->shape[d];
  }
  return true;
}

// [lo, hi) byte range a tensor may touch (strides are non-negative here).
struct Range { uintptr_t lo, hi; const char *name; };

inline Range range_of(const gdp_tensor *t, const char *name) {
  Range r{0, 0, name};
  if (!present(t)) return r;
  int64_t last = 0;
  for (int d = 0; d < t->ndim; ++d) {
    if (t->shape[d] == 0) return r;
    last += (t->shape[d] - 1) * t->stride[d];
  }
  r.lo = (uintptr_t)t->data;
  r.hi = r.lo + (uintptr_t)((last + 1) * elem_size(t->dtype));
  return r;
}

inline bool overlap(const Range &a, const Range &b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline bool nonneg_strides(const gdp_tensor *t) {
  for (int d = 0; d < t->ndim; ++d)
    if (t->stride[d] < 0) return false;
  return true;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace gdp
