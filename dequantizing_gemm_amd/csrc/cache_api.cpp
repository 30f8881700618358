// cache_api.cpp -- the C ABI declared in include/int4dq_cache.h: argument
// validation and launch on the caller's stream. As in api.cpp, no HIP call is
// made before the arguments have been validated.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/int4dq_cache.h"
#include "cache_check.h"

namespace {

using int4dq::AttentionArgs;
using int4dq::CacheView;
using int4dq::RowsView;
using int4dq::fail;
using int4dq::hip_status;
using int4dq::ok;

using int4dq::call_fits;
using int4dq::check_attention;
using int4dq::check_cache;
using int4dq::ll;
using int4dq::strides_ok;

}  // namespace

extern "C" {

int64_t int4_cache_row_bytes(int64_t head_dim) {
  if (head_dim < 1 || head_dim > int4dq::kMaxHeadDim) return -1;
  return 16 * int4dq::cache_blocks(head_dim);
}

int int4_cache_write(const int4_cache_t* cache, const int4_cache_rows_t* rows, const void* k, int64_t k_row_stride,
                     int64_t k_head_stride, const void* v, int64_t v_row_stride, int64_t v_head_stride, int dtype,
                     void* stream) {
  const char* fn = "int4_cache_write";
  CacheView c;
  RowsView r;
  const int rc = check_cache(fn, cache, rows, true, &c, &r);
  if (rc != INT4DQ_OK) return rc;
  if (dtype < INT4DQ_ROWS_F32 || dtype > INT4DQ_ROWS_BF16) return fail(INT4DQ_EINVAL, "%s: unknown dtype %d", fn, dtype);
  if (!strides_ok(k_row_stride, k_head_stride) || !strides_ok(v_row_stride, v_head_stride))
    return fail(INT4DQ_EINVAL, "%s: a stride is out of range", fn);
  if (r.rows == 0 || r.batch == 0) return ok();
  if (!k || !v) return fail(INT4DQ_EINVAL, "%s: k and v must be non-NULL", fn);
  return hip_status(int4dq::launch_cache_write(c, r, k, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride,
                                               dtype, (hipStream_t)stream),
                    "int4_cache_write launch");
}

int int4_cache_read(const int4_cache_t* cache, const int4_cache_rows_t* rows, void* k, void* v, int dtype,
                    void* stream) {
  const char* fn = "int4_cache_read";
  CacheView c;
  RowsView r;
  const int rc = check_cache(fn, cache, rows, true, &c, &r);
  if (rc != INT4DQ_OK) return rc;
  if (dtype < INT4DQ_ROWS_F32 || dtype > INT4DQ_ROWS_BF16) return fail(INT4DQ_EINVAL, "%s: unknown dtype %d", fn, dtype);
  if (r.rows == 0 || r.batch == 0) return ok();
  if (!k || !v) return fail(INT4DQ_EINVAL, "%s: k and v must be non-NULL", fn);
  return hip_status(int4dq::launch_cache_read(c, r, k, v, dtype, (hipStream_t)stream), "int4_cache_read launch");
}

int int4_cache_attention(const int4_cache_t* cache, const int4_cache_rows_t* rows, const void* q, int64_t q_row_stride,
                         int64_t q_head_stride, int dtype, int64_t q_heads, float scale, int causal, int64_t window,
                         void* out, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  AttentionArgs a;
  const int rc = check_attention("int4_cache_attention", cache, rows, q, q_row_stride, q_head_stride, dtype, q_heads, scale,
                                 causal, window, out, lse, workspace, workspace_bytes, &a);
  if (rc != INT4DQ_OK) return rc;
  if (a.r.rows == 0 || a.r.batch == 0) return ok();
  return hip_status(int4dq::launch_cache_attention(a, workspace, workspace_bytes, (hipStream_t)stream),
                    "int4_cache_attention launch");
}

int64_t int4_cache_attention_workspace_bytes(const int4_cache_t* cache, const int4_cache_rows_t* rows,
                                             int64_t q_heads) {
  const char* fn = "int4_cache_attention_workspace_bytes";
  CacheView c;
  RowsView r;
  if (check_cache(fn, cache, rows, false, &c, &r) != INT4DQ_OK) return -1;
  if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads || !call_fits(r, c, q_heads)) {
    fail(INT4DQ_EINVAL, "%s: q_heads must be a multiple of heads, rows * q_heads up to 2^27, batch * heads up to 2^22", fn);
    return -1;
  }
  if (r.rows == 0 || r.batch == 0) return 0;
  return int4dq::cache_attention_workspace(c, r, (int)(q_heads / c.heads));
}

}  // extern "C"
