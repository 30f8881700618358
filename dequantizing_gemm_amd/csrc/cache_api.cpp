// cache_api.cpp -- the C ABI declared in include/int4dq_cache.h: argument
// validation and launch on the caller's stream. As in api.cpp, no HIP call is
// made before the arguments have been validated.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "../../include/int4dq_cache.h"
#include "cache.h"
#include "status.h"

namespace {

using int4dq::AttentionArgs;
using int4dq::CacheView;
using int4dq::RowsView;
using int4dq::fail;
using int4dq::hip_status;
using int4dq::mul_ok;
using int4dq::ok;

typedef long long ll;

// Sizes of both descriptors; `pointers` also their arrays.
int check(const char* fn, const int4_cache_t* c, const int4_cache_rows_t* r, bool pointers, CacheView* cv,
          RowsView* rv) {
  if (!c || !r) return fail(INT4DQ_EINVAL, "%s: the cache and rows descriptors must be non-NULL", fn);
  if (c->head_dim < 1 || c->head_dim > int4dq::kMaxHeadDim)
    return fail(INT4DQ_EINVAL, "%s: head_dim must be 1 to %d (got %lld)", fn, int4dq::kMaxHeadDim, (ll)c->head_dim);
  if (c->group < c->head_dim && c->group != 32 && c->group != 64 && c->group != 128)
    return fail(INT4DQ_EINVAL, "%s: group must be 32, 64 or 128, or at least head_dim (got %lld with head_dim %lld)",
                fn, (ll)c->group, (ll)c->head_dim);
  if (c->heads < 1 || c->heads > 65535)
    return fail(INT4DQ_EINVAL, "%s: heads must be 1 to 65535 (got %lld)", fn, (ll)c->heads);
  if (c->page_size < 16 || c->page_size > (1 << 20) || (c->page_size & (c->page_size - 1)))
    return fail(INT4DQ_EINVAL, "%s: page_size must be a power of two from 16 to 2^20 (got %lld)", fn, (ll)c->page_size);
  if (c->pages < 1 || c->pages > INT32_MAX)
    return fail(INT4DQ_EINVAL, "%s: pages must be 1 to 2^31-1 (got %lld)", fn, (ll)c->pages);
  int64_t t;
  if (!mul_ok(c->pages, c->heads, &t) || !mul_ok(t, c->page_size, &t) || !mul_ok(t, 4 * int4dq::kMaxHeadDim, &t))
    return fail(INT4DQ_EINVAL, "%s: sizes overflow int64", fn);
  if (c->pages * c->heads * (c->page_size / 16) > INT32_MAX)     // at least 2 TiB of codes
    return fail(INT4DQ_EINVAL, "%s: the cache must hold fewer than 2^31 units of 16 tokens and one head", fn);
  // a block of 256 threads for 64 rows and two for a sequence: grids below 2^32 threads
  if (r->batch < 0 || r->batch > (1 << 22))
    return fail(INT4DQ_EINVAL, "%s: batch must be 0 to 2^22 (got %lld)", fn, (ll)r->batch);
  if (r->rows < 0 || r->rows > (1 << 26))
    return fail(INT4DQ_EINVAL, "%s: rows must be 0 to 2^26 (got %lld)", fn, (ll)r->rows);
  if (!r->starts && r->rows != r->batch)
    return fail(INT4DQ_EINVAL, "%s: without starts there is one row a sequence (got %lld rows, %lld sequences)", fn,
                (ll)r->rows, (ll)r->batch);
  if (r->max_pages < 0 || r->max_pages > INT32_MAX || r->table_stride < r->max_pages || r->table_stride > (1LL << 40))
    return fail(INT4DQ_EINVAL, "%s: max_pages must be 0 to 2^31-1 and table_stride at least that (got %lld, %lld)", fn,
                (ll)r->max_pages, (ll)r->table_stride);
  if (pointers) {
    if (!c->k_packed || !c->v_packed || !c->k_scales || !c->v_scales)
      return fail(INT4DQ_EINVAL, "%s: the cache's packed and scales arrays must be non-NULL", fn);
    if (!c->k_zeros != !c->v_zeros)
      return fail(INT4DQ_EINVAL, "%s: k_zeros and v_zeros must both be given or both be NULL", fn);
    const uintptr_t all = (uintptr_t)c->k_packed | (uintptr_t)c->v_packed | (uintptr_t)c->k_scales |
                          (uintptr_t)c->v_scales | (uintptr_t)c->k_zeros | (uintptr_t)c->v_zeros;
    if (all % 16) return fail(INT4DQ_EINVAL, "%s: the cache's arrays must be 16-byte aligned", fn);
    if (r->batch > 0 && (!r->lengths || (r->max_pages > 0 && !r->page_table)))
      return fail(INT4DQ_EINVAL, "%s: page_table and lengths must be non-NULL", fn);
  }
  int shift = 0;
  while ((1LL << shift) < c->page_size) ++shift;
  const int D = (int)c->head_dim;
  const int group = c->group < D ? (int)c->group : D;
  *cv = CacheView{c->k_packed, c->k_scales, c->k_zeros, c->v_packed, c->v_scales, c->v_zeros, c->pages, shift,
                  (int)c->heads, D, group, (D + group - 1) / group, int4dq::cache_blocks(D), c->k_zeros ? 1 : 0};
  *rv = RowsView{r->page_table, r->table_stride, r->max_pages, r->lengths, r->starts, (int)r->batch, r->rows};
  return INT4DQ_OK;
}

// Element strides of a row-wise array (any sign; 0 repeats a row or a head).
bool strides_ok(int64_t row_stride, int64_t head_stride) {
  const int64_t lim = int64_t(1) << 30;      // with rows up to 2^26 and heads below 2^16: offsets below 2^57
  return row_stride >= -lim && row_stride <= lim && head_stride >= -lim && head_stride <= lim;
}

// The attention kernel's grid, a block of 256 threads for each 16 query rows of a
// head and for each sequence and head, stays below 2^32 threads.
bool call_fits(const RowsView& r, const CacheView& c, int64_t q_heads) {
  return r.rows * q_heads <= (int64_t(1) << 27) && (int64_t)r.batch * c.heads <= (int64_t(1) << 22);
}

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
  const int rc = check(fn, cache, rows, true, &c, &r);
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
  const int rc = check(fn, cache, rows, true, &c, &r);
  if (rc != INT4DQ_OK) return rc;
  if (dtype < INT4DQ_ROWS_F32 || dtype > INT4DQ_ROWS_BF16) return fail(INT4DQ_EINVAL, "%s: unknown dtype %d", fn, dtype);
  if (r.rows == 0 || r.batch == 0) return ok();
  if (!k || !v) return fail(INT4DQ_EINVAL, "%s: k and v must be non-NULL", fn);
  return hip_status(int4dq::launch_cache_read(c, r, k, v, dtype, (hipStream_t)stream), "int4_cache_read launch");
}

int int4_cache_attention(const int4_cache_t* cache, const int4_cache_rows_t* rows, const void* q, int64_t q_row_stride,
                         int64_t q_head_stride, int dtype, int64_t q_heads, float scale, int causal, int64_t window,
                         void* out, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* fn = "int4_cache_attention";
  CacheView c;
  RowsView r;
  const int rc = check(fn, cache, rows, true, &c, &r);
  if (rc != INT4DQ_OK) return rc;
  if (dtype != INT4DQ_ROWS_F16 && dtype != INT4DQ_ROWS_BF16)
    return fail(INT4DQ_EINVAL, "%s: dtype must be binary16 or bfloat16 (got %d)", fn, dtype);
  if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads)
    return fail(INT4DQ_EINVAL, "%s: q_heads must be a multiple of heads, up to 65535 (got %lld, %d)", fn, (ll)q_heads, c.heads);
  if (!call_fits(r, c, q_heads))
    return fail(INT4DQ_EINVAL, "%s: rows * q_heads must be up to 2^27 and batch * heads up to 2^22", fn);
  if (!isfinite(scale) || !(scale > 0.0f))
    return fail(INT4DQ_EINVAL, "%s: scale must be finite and above 0 (got %g)", fn, (double)scale);
  if (window < 0 || (window > 0 && !causal))
    return fail(INT4DQ_EINVAL, "%s: window must be >= 0, and needs causal (got %lld)", fn, (ll)window);
  if (!strides_ok(q_row_stride, q_head_stride))
    return fail(INT4DQ_EINVAL, "%s: a stride is out of range", fn);
  if (workspace_bytes < 0 || (workspace_bytes > 0 && !workspace))
    return fail(INT4DQ_EINVAL, "%s: workspace_bytes must be >= 0, with a non-NULL workspace when > 0", fn);
  if ((uintptr_t)workspace % 256) return fail(INT4DQ_EINVAL, "%s: workspace must be 256-byte aligned", fn);
  if (r.rows == 0 || r.batch == 0) return ok();
  if (!q || !out) return fail(INT4DQ_EINVAL, "%s: q and out must be non-NULL", fn);
  const bool wide = (uintptr_t)q % 16 == 0 && c.D % 8 == 0 && q_row_stride % 8 == 0 && q_head_stride % 8 == 0;
  int scale_exp;
  const float scale_part = (float)frexp((double)scale * 1.44269504088896340736, &scale_exp);
  const AttentionArgs a{c, r, q, q_row_stride, q_head_stride, dtype == INT4DQ_ROWS_BF16 ? 1 : 0, wide ? 1 : 0,
                        (int)(q_heads / c.heads), scale_part, scale_exp, causal ? 1 : 0, window, out, lse};
  return hip_status(int4dq::launch_cache_attention(a, workspace, workspace_bytes, (hipStream_t)stream),
                    "int4_cache_attention launch");
}

int64_t int4_cache_attention_workspace_bytes(const int4_cache_t* cache, const int4_cache_rows_t* rows,
                                             int64_t q_heads) {
  const char* fn = "int4_cache_attention_workspace_bytes";
  CacheView c;
  RowsView r;
  if (check(fn, cache, rows, false, &c, &r) != INT4DQ_OK) return -1;
  if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads || !call_fits(r, c, q_heads)) {
    fail(INT4DQ_EINVAL, "%s: q_heads must be a multiple of heads, rows * q_heads up to 2^27, batch * heads up to 2^22", fn);
    return -1;
  }
  if (r.rows == 0 || r.batch == 0) return 0;
  return int4dq::cache_attention_workspace(c, r, (int)(q_heads / c.heads));
}

}  // extern "C"
