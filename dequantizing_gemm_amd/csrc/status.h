// status.h -- status codes and the thread-local error text behind
// int4_last_error(), shared by the files that implement the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/int4dq.h"

namespace int4dq {

inline thread_local char g_err[512] = "";

inline int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

inline int ok() {
  g_err[0] = '\0';
  return INT4DQ_OK;
}

// a * b with overflow check into *out (both non-negative).
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

inline int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(INT4DQ_EHIP, "%s: %s", what, hipGetErrorString(e));
}

}  // namespace int4dq
