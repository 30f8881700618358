/*
 * int4dq_cache.h -- C ABI of the key/value cache held in 4-bit group codes:
 * quantising new keys and values into a paged cache, reading them back, and
 * softmax attention over the cache without writing it out in full precision.
 *
 * The codes are those of int4_quantize / int4_quantize_affine (int4dq.h): the
 * head_dim channels of one token and one head are one weight row, split into
 * groups of `group` consecutive channels (32, 64 or 128; the last may be
 * partial; or any number from head_dim up: one group) with a binary16 scale
 * each, and a zero point each where the cache is affine.
 *
 * The conventions of int4dq.h hold here too: device pointers owned by the
 * caller, work enqueued on `stream` without waiting, arguments validated before
 * anything is enqueued, status codes and int4_last_error(), nothing allocated,
 * no state between calls. The two descriptor structs are read during the call
 * and not kept; they live in host memory.
 *
 * Layout of a cache. head_dim is 1 to 256; C is the smallest of 2, 3, 4, 6, 8
 * with 32 C >= head_dim, DB = 16 C the bytes of one token's codes, and
 * G = ceil(head_dim / group). A page holds page_size tokens (a power of two
 * from 16 up) of every head. The orders are those in which the matrix
 * instructions take the codes:
 *   k_packed [pages, heads, page_size, DB]: channel d = 32 i + 8 a + e (a < 4,
 *            e < 8) of a token is nibble e % 2 (0: low) of byte 4 C a + 4 i + e / 2.
 *   v_packed [pages, heads, page_size / 16, DB, 16]: channel d of token t is
 *            nibble d % 2 of byte [t / 16, d / 2, t % 16].
 *   k_scales, v_scales [pages, heads, page_size / 16, G, 16] binary16, the
 *            scale of group g of token t at [t / 16, g, t % 16] (written ones are
 *            not negative; a cache filled elsewhere may hold either sign).
 *   k_zeros, v_zeros   bytes of the same shape, or both NULL (symmetric codes).
 * k_packed, v_packed, the scales and the zeros are 16-byte aligned.
 *
 * Rows and sequences. Sequence b owns rows starts[b] .. starts[b+1]-1 of the
 * call's row-wise arrays (keys, values, queries, outputs); they are its last
 * tokens, at positions lengths[b] - (starts[b+1] - starts[b]) .. lengths[b]-1,
 * so lengths counts the call's own rows. starts = NULL: one row a sequence
 * (rows = batch). Position p of sequence b is slot p % page_size of page
 * page_table[b * table_stride + p / page_size].
 * The contents of page_table, lengths and starts are device memory and are not
 * validated, but no content makes a call read or write out of range:
 *   - a row that no sequence owns (before starts[0], from starts[batch] on) is
 *     left as it was in every output;
 *   - a position below 0, at or above max_pages * page_size, or on a page
 *     outside 0 .. pages-1 is not written, reads back as zeros, and takes no
 *     part in attention.
 * starts must not decrease. Where two rows of one write call come to lie on the
 * same slot (a page listed twice), what that slot holds afterwards is a mixture.
 */
#ifndef INT4DQ_CACHE_H
#define INT4DQ_CACHE_H

#include "int4dq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of the row-wise arrays. */
#define INT4DQ_ROWS_F32  0     /* IEEE binary32 */
#define INT4DQ_ROWS_F16  1     /* IEEE binary16 */
#define INT4DQ_ROWS_BF16 2     /* bfloat16 */

typedef struct int4_cache {
  uint8_t *k_packed;
  uint16_t *k_scales;
  uint8_t *k_zeros;            /* NULL: symmetric codes */
  uint8_t *v_packed;
  uint16_t *v_scales;
  uint8_t *v_zeros;            /* NULL with k_zeros */
  int64_t pages, page_size, heads, head_dim, group;
} int4_cache_t;

typedef struct int4_cache_rows {
  const int32_t *page_table;   /* [batch, max_pages], rows table_stride elements apart */
  int64_t table_stride, max_pages;
  const int32_t *lengths;      /* [batch] */
  const int32_t *starts;       /* [batch + 1], or NULL: one row a sequence */
  int64_t batch;
  int64_t rows;                /* rows of the row-wise arrays */
} int4_cache_rows_t;

/*
 * Bytes of one token's codes of one head (DB above) for this head_dim, for keys
 * and for values alike; -1 if head_dim is not in 1 .. 256.
 */
int64_t int4_cache_row_bytes(int64_t head_dim);

/*
 * Quantise rows of keys and values into the cache.
 *   k, v    in : [rows, heads, head_dim] of `dtype`; rows and heads lie
 *                k_row_stride / k_head_stride (v_...) elements apart, channels
 *                side by side. Widened to binary32, which is exact.
 *   cache   out: codes, scales and zero points of the rows' positions, the bits
 *                int4_quantize (int4_quantize_affine) gives for [1, head_dim]
 *                rows of the same values; every other position is left as it
 *                was. Codes of the channels that pad head_dim to 32 C are 0.
 * Errors: EINVAL for a NULL pointer, a size out of range or that overflows,
 * heads > 65535, a group below head_dim other than 32, 64, 128, a page_size
 * that is no power of two from 16 to 2^20, 2^31 or more units of 16 tokens and one
 * head in the cache, one of k_zeros / v_zeros only, a misaligned cache array, an
 * unknown dtype, a stride beyond 2^30, batch above 2^22, rows above 2^26, a
 * table_stride below max_pages, rows != batch with starts = NULL. rows = 0 or
 * batch = 0 is a valid no-op.
 */
int int4_cache_write(const int4_cache_t *cache, const int4_cache_rows_t *rows, const void *k,
                     int64_t k_row_stride, int64_t k_head_stride, const void *v,
                     int64_t v_row_stride, int64_t v_head_stride, int dtype, void *stream);

/*
 * Read rows back: k, v out: dense [rows, heads, head_dim] of `dtype`, the value
 * code * scale ((code - zero point) * scale) of each channel at the rows'
 * positions, exact in binary32 and otherwise that rounded to nearest even.
 * With starts giving each sequence lengths[b] rows, whole sequences.
 * Errors: those of int4_cache_write.
 */
int int4_cache_read(const int4_cache_t *cache, const int4_cache_rows_t *rows, void *k, void *v,
                    int dtype, void *stream);

/*
 * Softmax attention of rows of queries over the cache. Query head h attends to
 * key/value head h / (q_heads / heads). With row t of sequence b at position p
 * (its own key is in the cache: write first), over the keys j of sequence b
 * with j < lengths[b], with causal also j <= p, and with window > 0 also
 * j > p - window:
 *   a_j = scale * q . k_j,  out = sum_j exp(a_j) v_j / sum_j exp(a_j),
 *   lse = log(sum_j exp(a_j)).
 * No keys: out = 0, lse = -infinity.
 *   q       in : [rows, q_heads, head_dim] of `dtype` (INT4DQ_ROWS_F16 or
 *                INT4DQ_ROWS_BF16), rows and heads q_row_stride / q_head_stride
 *                elements apart, channels side by side.
 *   out     out: dense [rows, q_heads, head_dim] of `dtype`.
 *   lse     out: dense [rows, q_heads] binary32, or NULL.
 *   Arithmetic: codes and queries are multiplied exactly (queries below 2^-27 of
 *   their row's largest as rounded to 2^-38 of it) and summed in
 *   binary32; probabilities and their sum are binary32; the product of a
 *   probability and a value's scale is rounded to binary16 before it multiplies
 *   the value's code, summed in binary32. That rounding is at most 2^-11 of the
 *   product or, where this is more, 2^-33 P max(S, 2^-15) with P the largest
 *   probability and S the largest value scale (in magnitude) of 16 tokens of a
 *   unit that the row sees, in the unit where that is most; or 2^-25 P where the
 *   row's largest score is 2^21 or more in magnitude. Tokens that a row does not
 *   see have no part in this, whatever their codes, scales and zero points hold.
 *   workspace: device memory, 256-byte aligned, any contents, of at least
 *                int4_cache_attention_workspace_bytes, which lets long sequences
 *                be shared out over the whole GPU; or NULL with
 *                workspace_bytes = 0, and any smaller size runs without that or
 *                with less of it.
 *                Calls that share a workspace must not overlap.
 *   Speed: prompts take about twice as long with heads of more than 192 channels in
 *   groups of 32 (with zero points, of 64 too), and with heads of 129 to 192 channels
 *   and zero points in groups of 32 or 128; groups of 128 of 192 channels, and of 64 of
 *   96, cost what groups of 32 do.
 * Preconditions not checked: q is finite and below 2^100 in magnitude, and so are
 * the scores a_j below 2^96.
 * Errors: those of int4_cache_write, and EINVAL for q_heads that is no multiple
 * of heads, a scale that is not finite and above 0, window < 0 or window
 * without causal, a bad workspace, INT4DQ_ROWS_F32, rows * q_heads above 2^27 or
 * batch * heads above 2^22.
 */
int int4_cache_attention(const int4_cache_t *cache, const int4_cache_rows_t *rows, const void *q,
                         int64_t q_row_stride, int64_t q_head_stride, int dtype, int64_t q_heads,
                         float scale, int causal, int64_t window, void *out, float *lse,
                         void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Workspace bytes of int4_cache_attention for these sizes (no pointer in the
 * descriptors is read or has to be set, except that starts = NULL says one row
 * a sequence and k_zeros = NULL symmetric codes); 0: the call does not use one.
 * -1 on invalid sizes.
 */
int64_t int4_cache_attention_workspace_bytes(const int4_cache_t *cache,
                                             const int4_cache_rows_t *rows, int64_t q_heads);

#ifdef __cplusplus
}
#endif

#endif /* INT4DQ_CACHE_H */
