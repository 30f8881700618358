/*
 * int4dq_cache_step.h -- C ABI of a serving step around the 4-bit key/value cache
 * (int4dq_cache.h): pages for new tokens, norms and rotation on the way into the
 * cache, and attention with first tokens that stay visible or that a batch shares.
 *
 * The conventions of int4dq.h and int4dq_cache.h hold here too: device pointers
 * owned by the caller, work enqueued on `stream` without waiting, arguments
 * validated before anything is enqueued, status codes and int4_last_error(),
 * nothing allocated, no state between calls, and no contents of device arrays that
 * make a call read or write out of range.
 */
#ifndef INT4DQ_CACHE_STEP_H
#define INT4DQ_CACHE_STEP_H

#include "int4dq_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The page table of a batch and the pages that no sequence has.
 *   free   [pages]: the numbers of the free pages are its first count[0] entries;
 *          pages are taken from the end and given back there.
 * The sequence b with lengths[b] tokens holds the first ceil(lengths[b] /
 * page_size) entries of its table row, at most max_pages; what the other entries
 * hold has no meaning. A length below 0 counts as 0, a count[0] outside 0 .. pages
 * as the nearer of these.
 */
typedef struct int4_cache_pool {
  int32_t *page_table;         /* [batch, max_pages], rows table_stride elements apart */
  int64_t table_stride, max_pages, batch;
  int64_t page_size;           /* tokens, a power of two from 16 to 2^20 */
  int32_t *free;               /* [pages] */
  int64_t pages;
} int4_cache_pool_t;

/*
 * Give the pages of ended sequences back.
 *   lengths, done  in : [batch] tokens of each sequence; bytes, not 0: ended.
 *   count          in : [2], of which the first is read.
 *   shared         in : [1], or NULL: the pages that lie wholly in a sequence's
 *                  first shared[0] tokens are other sequences' too and not given back.
 *   free           out: the pages of ended sequences, in the order of the sequences
 *                  and of their table rows, from place count[0] on, as far as there
 *                  is room; entries that are no page of 0 .. pages-1 are left out.
 *   new_lengths    out: [batch] lengths, 0 for ended sequences; may be lengths.
 *   new_count      out: [2] the free pages, and 0; may be count.
 * The page table is not changed. A page that is listed twice is given back twice.
 * Errors: EINVAL for a NULL pointer (other than shared) or a size out of range:
 * batch above 2^22, max_pages or pages above 2^31-1, a table_stride below max_pages
 * (and batch = 0 is valid).
 */
int int4_cache_release(const int4_cache_pool_t *pool, const int32_t *lengths, const uint8_t *done,
                       const int32_t *count, const int32_t *shared, int32_t *new_lengths,
                       int32_t *new_count, void *stream);

/*
 * Pages for new tokens, and what a call that writes or attends to them is given.
 *   lengths    in : [batch] tokens before.
 *   added      in : [batch] new tokens (below 0 counts as 0), or NULL: one each.
 *   count      in : [2], of which the first is read.
 *   page_table out: the entries that the new tokens need beyond those held, taken
 *              from the free pages in the order of the sequences and of their table
 *              rows; -1 where these run out. Tokens past max_pages pages get none.
 *   new_lengths out: [batch] lengths + added, at most 2^31-1, which a caller keeps
 *              below: from there on the new rows have the last positions. May be lengths.
 *   starts     out: [batch + 1] exclusive sums of added: the rows of each sequence
 *              as int4dq_cache.h has them.
 *   slots      out: [rows], or NULL: for each row page * page_size + the place on
 *              the page of its position, as the other calls derive it from new_lengths
 *              and starts, -1 where it has no page and behind the last sequence's rows.
 *   new_count  out: [2] the free pages, and how many more were needed; may be count.
 * An entry of -1 counts as held, so that a token that lacks a page has none later either.
 * A caller who does not want that takes the step back where new_count[1] is above 0: the
 * call leaves free, and lengths and count where they are not its outputs, as they were;
 * with these, pages given back by int4_cache_release, and the call once more, the table's
 * entries are written anew.
 * Errors: those of int4_cache_release, and EINVAL for rows outside 0 .. 2^26.
 */
int int4_cache_extend(const int4_cache_pool_t *pool, const int32_t *lengths, const int32_t *added,
                      const int32_t *count, int32_t *new_lengths, int32_t *starts, int64_t *slots,
                      int64_t rows, int32_t *new_count, void *stream);

/*
 * Norms and rotation of queries and keys. For the channels x of a row and head at
 * position p (each step rounds to binary32, the mean and root are binary64):
 *   with a norm:  r = binary32(1 / sqrt(mean(x^2) + eps)), y = (x r) weight;
 *   with a rope:  for each pair (a, b) of the first rotary_dim channels
 *                 (y_a cos - y_b sin, y_b cos + y_a sin), cos = rope[p, i], sin =
 *                 rope[p, rotary_dim / 2 + i] for pair i: channels i and
 *                 rotary_dim / 2 + i, or interleaved 2 i and 2 i + 1.
 */
typedef struct int4_cache_transform {
  const float *q_norm, *k_norm;          /* [head_dim] weights, or NULL: no norm */
  double eps;
  const float *rope;                     /* [rope_positions, rotary_dim] binary32, or NULL */
  int64_t rope_stride, rope_positions;   /* rows rope_stride elements apart */
  int64_t rotary_dim;                    /* even */
  int interleaved;
} int4_cache_transform_t;

/*
 * One pass from a projection's output to attention: queries normalised and rotated
 * into q_out, keys normalised, rotated and quantised into the cache, values
 * quantised into the cache. Positions are the rows' in the cache.
 *   q       in : [rows, q_heads, head_dim], k, v in : [rows, heads, head_dim] of
 *           `dtype`, rows and heads ..._row_stride / ..._head_stride elements apart,
 *           channels side by side.
 *   q_out   out: dense [rows, q_heads, head_dim] of `dtype`, rounded to nearest
 *           even; may be q where q is dense. A row that no sequence owns is left as
 *           it was; one whose position is below 0, or at or above rope_positions, is
 *           0 and its key and value are not written.
 *   cache   out: as int4_cache_write of the transformed keys (as binary32, they are
 *           not rounded to `dtype` between) and of the values.
 * Preconditions not checked: q, k and v, weights, cosines and sines are finite, and
 * with eps = 0 no row that is normalised is all zeros.
 * Errors: those of int4_cache_write, and EINVAL for q_heads outside 1 .. 65535,
 * rows * (heads + q_heads) above 2^25 or batch * heads above 2^20, a rotary_dim that
 * is odd or outside 2 .. head_dim (where there is a rope), rope_positions outside
 * 1 .. 2^31-1, a rope_stride below rotary_dim or above 2^30, an eps that is negative
 * or not finite.
 */
int int4_cache_append(const int4_cache_t *cache, const int4_cache_rows_t *rows,
                      const int4_cache_transform_t *transform, const void *q, int64_t q_row_stride,
                      int64_t q_head_stride, int64_t q_heads, const void *k, int64_t k_row_stride,
                      int64_t k_head_stride, const void *v, int64_t v_row_stride, int64_t v_head_stride,
                      int dtype, void *q_out, void *stream);

/*
 * int4_cache_attention with first tokens that stay visible and first tokens that all
 * sequences share.
 *   sinks   with window > 0: a row at position p sees the keys j <= p with
 *           j > p - window or j < sinks. Without a window it has no effect.
 *   shared  in : [1], or NULL: every sequence begins with the same shared[0] tokens
 *           (below 0: none). A sequence sees of them what it sees of its own (all
 *           up to its length, its rows up to their positions). They are read through
 *           the first row of page_table, whatever lengths[0] is, once for all
 *           sequences from share_from on, and with a workspace for it. The other entries
 *           of page_table that stand for them have to name the same keys and values.
 *   share_from  the least number of shared tokens that are computed once, whatever
 *           it costs; below 0: the library chooses, by the number of sequences and of
 *           their rows: from 1536 to 6144 tokens on for 4 or more sequences of up to 8 query
 *           rows to a key head, from 16384 on for 8 or more of 65 to 640 (16384 in all),
 *           otherwise not at all. It does not go by the window: with one that reaches
 *           few of the shared tokens a call without `shared` is faster. Results may differ
 *           in rounding.
 *   The arithmetic is that of int4_cache_attention; with shared tokens the two parts
 *   of a row are joined in binary32.
 * Errors: those of int4_cache_attention, and EINVAL for sinks < 0.
 */
int int4_cache_attention_ex(const int4_cache_t *cache, const int4_cache_rows_t *rows, const void *q,
                            int64_t q_row_stride, int64_t q_head_stride, int dtype, int64_t q_heads,
                            float scale, int causal, int64_t window, int64_t sinks,
                            const int32_t *shared, int64_t share_from, void *out, float *lse,
                            void *workspace, int64_t workspace_bytes, void *stream);

/*
 * As int4_cache_attention_workspace_bytes, of int4_cache_attention_ex; shares: 0 where
 * `shared` will be NULL.
 */
int64_t int4_cache_attention_ex_workspace_bytes(const int4_cache_t *cache,
                                                const int4_cache_rows_t *rows, int64_t q_heads,
                                                int shares, int64_t share_from);

#ifdef __cplusplus
}
#endif

#endif /* INT4DQ_CACHE_STEP_H */
