// cache_step_api.cpp -- the C ABI declared in include/int4dq_cache_step.h: argument
// validation and launch on the caller's stream. As in api.cpp, no HIP call is made
// before the arguments have been validated.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "../../include/int4dq_cache_step.h"
#include "cache_check.h"
#include "cache_step.h"

namespace {

using int4dq::AppendArgs;
using int4dq::AttentionArgs;
using int4dq::CacheView;
using int4dq::PagesArgs;
using int4dq::RowsView;
using int4dq::call_fits;
using int4dq::check_attention;
using int4dq::check_cache;
using int4dq::fail;
using int4dq::hip_status;
using int4dq::ll;
using int4dq::ok;
using int4dq::strides_ok;

int check_pool(const char* fn, const int4_cache_pool_t* p, const int32_t* lengths, const int32_t* count,
               int32_t* new_lengths, int32_t* new_count, PagesArgs* a) {
  if (!p) return fail(INT4DQ_EINVAL, "%s: the pool descriptor must be non-NULL", fn);
  if (p->page_size < 16 || p->page_size > (1 << 20) || (p->page_size & (p->page_size - 1)))
    return fail(INT4DQ_EINVAL, "%s: page_size must be a power of two from 16 to 2^20 (got %lld)", fn, (ll)p->page_size);
  if (p->pages < 0 || p->pages > INT32_MAX)
    return fail(INT4DQ_EINVAL, "%s: pages must be 0 to 2^31-1 (got %lld)", fn, (ll)p->pages);
  if (p->batch < 0 || p->batch > (1 << 22))
    return fail(INT4DQ_EINVAL, "%s: batch must be 0 to 2^22 (got %lld)", fn, (ll)p->batch);
  if (p->max_pages < 0 || p->max_pages > INT32_MAX || p->table_stride < p->max_pages || p->table_stride > (1LL << 40))
    return fail(INT4DQ_EINVAL, "%s: max_pages must be 0 to 2^31-1 and table_stride at least that (got %lld, %lld)", fn,
                (ll)p->max_pages, (ll)p->table_stride);
  if ((p->batch > 0 && (!lengths || !new_lengths || (p->max_pages > 0 && !p->page_table))) || (p->pages > 0 && !p->free) ||
      !count || !new_count)
    return fail(INT4DQ_EINVAL, "%s: page_table, free, lengths and count must be non-NULL", fn);
  int shift = 0;
  while ((1LL << shift) < p->page_size) ++shift;
  *a = PagesArgs{p->page_table, p->table_stride, p->max_pages, (int)p->batch, shift, lengths,
                 p->free, p->pages, count, new_lengths, new_count};
  return INT4DQ_OK;
}

}  // namespace

extern "C" {

int int4_cache_release(const int4_cache_pool_t* pool, const int32_t* lengths, const uint8_t* done, const int32_t* count,
                       const int32_t* shared, int32_t* new_lengths, int32_t* new_count, void* stream) {
  const char* fn = "int4_cache_release";
  PagesArgs a;
  const int rc = check_pool(fn, pool, lengths, count, new_lengths, new_count, &a);
  if (rc != INT4DQ_OK) return rc;
  if (a.batch > 0 && !done) return fail(INT4DQ_EINVAL, "%s: done must be non-NULL", fn);
  return hip_status(int4dq::launch_cache_release(a, done, shared, (hipStream_t)stream), "int4_cache_release launch");
}

int int4_cache_extend(const int4_cache_pool_t* pool, const int32_t* lengths, const int32_t* added, const int32_t* count,
                      int32_t* new_lengths, int32_t* starts, int64_t* slots, int64_t rows, int32_t* new_count,
                      void* stream) {
  const char* fn = "int4_cache_extend";
  PagesArgs a;
  const int rc = check_pool(fn, pool, lengths, count, new_lengths, new_count, &a);
  if (rc != INT4DQ_OK) return rc;
  if (rows < 0 || rows > (1 << 26)) return fail(INT4DQ_EINVAL, "%s: rows must be 0 to 2^26 (got %lld)", fn, (ll)rows);
  if (!starts) return fail(INT4DQ_EINVAL, "%s: starts must be non-NULL", fn);
  return hip_status(int4dq::launch_cache_extend(a, added, starts, rows > 0 ? slots : nullptr, rows, (hipStream_t)stream),
                    "int4_cache_extend launch");
}

int int4_cache_append(const int4_cache_t* cache, const int4_cache_rows_t* rows, const int4_cache_transform_t* transform,
                      const void* q, int64_t q_row_stride, int64_t q_head_stride, int64_t q_heads, const void* k,
                      int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
                      int64_t v_head_stride, int dtype, void* q_out, void* stream) {
  const char* fn = "int4_cache_append";
  CacheView c;
  RowsView r;
  const int rc = check_cache(fn, cache, rows, true, &c, &r);
  if (rc != INT4DQ_OK) return rc;
  if (!transform) return fail(INT4DQ_EINVAL, "%s: the transform descriptor must be non-NULL", fn);
  const int4_cache_transform_t& t = *transform;
  if (dtype < INT4DQ_ROWS_F32 || dtype > INT4DQ_ROWS_BF16) return fail(INT4DQ_EINVAL, "%s: unknown dtype %d", fn, dtype);
  if (q_heads < 1 || q_heads > 65535)
    return fail(INT4DQ_EINVAL, "%s: q_heads must be 1 to 65535 (got %lld)", fn, (ll)q_heads);
  // below 2^24 blocks of 256 threads: of queries at most 1/8 of these rows, of keys and
  // values 1/16 of them and four a sequence and head
  if (r.rows * (c.heads + q_heads) > (1 << 25) || (int64_t)r.batch * c.heads > (1 << 20))
    return fail(INT4DQ_EINVAL, "%s: rows * (heads + q_heads) must be up to 2^25 and batch * heads up to 2^20", fn);
  if (!strides_ok(q_row_stride, q_head_stride) || !strides_ok(k_row_stride, k_head_stride) ||
      !strides_ok(v_row_stride, v_head_stride))
    return fail(INT4DQ_EINVAL, "%s: a stride is out of range", fn);
  if (!isfinite(t.eps) || t.eps < 0.0)
    return fail(INT4DQ_EINVAL, "%s: eps must be finite and not negative (got %g)", fn, t.eps);
  if (t.rope) {
    if (t.rotary_dim < 2 || t.rotary_dim % 2 || t.rotary_dim > c.D)
      return fail(INT4DQ_EINVAL, "%s: rotary_dim must be even, 2 to head_dim (got %lld)", fn, (ll)t.rotary_dim);
    if (t.rope_positions < 1 || t.rope_positions > INT32_MAX)
      return fail(INT4DQ_EINVAL, "%s: rope_positions must be 1 to 2^31-1 (got %lld)", fn, (ll)t.rope_positions);
    if (t.rope_stride < t.rotary_dim || t.rope_stride > (1 << 30))
      return fail(INT4DQ_EINVAL, "%s: rope_stride must be at least rotary_dim, up to 2^30 (got %lld)", fn, (ll)t.rope_stride);
  }
  if (r.rows == 0 || r.batch == 0) return ok();
  if (!q || !k || !v || !q_out) return fail(INT4DQ_EINVAL, "%s: q, k, v and q_out must be non-NULL", fn);
  const AppendArgs a{c, r, q, k, v, q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride,
                     q_out, (int)q_heads, t.q_norm, t.k_norm, t.eps, t.rope, t.rope_stride, t.rope_positions,
                     t.rope ? (int)(t.rotary_dim / 2) : 0, t.interleaved ? 1 : 0};
  return hip_status(int4dq::launch_cache_append(a, dtype, (hipStream_t)stream), "int4_cache_append launch");
}

int int4_cache_attention_ex(const int4_cache_t* cache, const int4_cache_rows_t* rows, const void* q, int64_t q_row_stride,
                            int64_t q_head_stride, int dtype, int64_t q_heads, float scale, int causal, int64_t window,
                            int64_t sinks, const int32_t* shared, int64_t share_from, void* out, float* lse, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  const char* fn = "int4_cache_attention_ex";
  AttentionArgs a;
  const int rc = check_attention(fn, cache, rows, q, q_row_stride, q_head_stride, dtype, q_heads, scale, causal, window, out,
                                 lse, workspace, workspace_bytes, &a);
  if (rc != INT4DQ_OK) return rc;
  if (sinks < 0) return fail(INT4DQ_EINVAL, "%s: sinks must be >= 0 (got %lld)", fn, (ll)sinks);
  if (a.r.rows == 0 || a.r.batch == 0) return ok();
  a.sinks = sinks;
  a.shared = shared;
  return hip_status(shared ? int4dq::launch_cache_attention_shared(a, share_from, workspace, workspace_bytes, (hipStream_t)stream)
                           : int4dq::launch_cache_attention(a, workspace, workspace_bytes, (hipStream_t)stream),
                    "int4_cache_attention_ex launch");
}

int64_t int4_cache_attention_ex_workspace_bytes(const int4_cache_t* cache, const int4_cache_rows_t* rows, int64_t q_heads,
                                                int shares, int64_t share_from) {
  const char* fn = "int4_cache_attention_ex_workspace_bytes";
  CacheView c;
  RowsView r;
  if (check_cache(fn, cache, rows, false, &c, &r) != INT4DQ_OK) return -1;
  if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads || !call_fits(r, c, q_heads)) {
    fail(INT4DQ_EINVAL, "%s: q_heads must be a multiple of heads, rows * q_heads up to 2^27, batch * heads up to 2^22", fn);
    return -1;
  }
  if (r.rows == 0 || r.batch == 0) return 0;
  const int ratio = (int)(q_heads / c.heads);
  const int64_t whole = int4dq::cache_attention_workspace(c, r, ratio);
  const int64_t parts = shares ? int4dq::cache_attention_shared_workspace(c, r, ratio, share_from) : 0;
  return whole > parts ? whole : parts;
}

}  // extern "C"
