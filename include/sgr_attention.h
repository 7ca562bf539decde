/*
 * sgr_attention.h -- C ABI of the attention operators that run between two
 * projections of a decode step (skinny_gemm_residual.h): queries and keys
 * normalised per head and rotated, keys and values appended to a paged cache
 * of 8-bit codes, and attention over that cache.  The output of
 * sgr_kv_attention is the A operand of the projection that follows it.
 *
 *   norm + rotation   y = x / sqrt(mean_d x_d^2 + eps) * w, then for each pair
 *                     (a, b) of the first rot_dim elements
 *                     (a cos - b sin, b cos + a sin)
 *   append            code = e4m3(x / s), s = 2^e, one s for each page and
 *                     key/value head: the smallest power of two for which no
 *                     token of the page saturates
 *   attention         o = sum_t p_t v_t / sum_t p_t, p_t = exp(scale q.k_t),
 *                     over the positions t that the query's token may see
 *
 * Sums, norms and softmax statistics are held in 32 bits, and results are
 * rounded once to BF16 or E4M3.  Attention's two products run on the tensor
 * core, which sees queries and weights in fewer bits: sgr_kv_attention says how
 * many.
 *
 * Pointers are device pointers owned by the caller; structures are host
 * memory, read during the call only.  Calls enqueue work on `stream`, return
 * without synchronising and keep no state.  Kernels launch with programmatic
 * dependent launch unless SGR_FLAG_NO_PDL is given, and read and write
 * nothing of the caller's before the preceding work on the stream has
 * completed.  Calls may be captured into a CUDA graph once sgr_init() has run
 * for the device.  Lengths, tables and positions are device data, so a graph
 * replays with new ones.
 *
 * Errors are those of skinny_gemm_residual.h, found before anything is
 * enqueued.  What only the device can see -- a page number outside the cache,
 * a length beyond the block table, a position beyond the rotation table, row
 * offsets that run backwards or past `tokens` -- is never followed: the
 * kernel clamps or skips it and records code 7 in the device error word
 * (sgr_device_error).  (Code 8: a block's shared memory did not begin where the
 * kernel needs it; nothing was computed.)
 */
#ifndef SGR_ATTENTION_H
#define SGR_ATTENTION_H

#include <stdint.h>

#include "skinny_gemm_residual.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags of sgr_kv_attention and its workspace, beside SGR_FLAG_NO_PDL: the
 * kernel for few rows (row tiles of at most 32) or many (256) whatever the
 * sizes, for sweeps and tests.  Neither: the library's choice.  Both:
 * SGR_ERR_UNSUPPORTED. */
#define SGR_FLAG_KV_FEW_ROWS 0x2u
#define SGR_FLAG_KV_MANY_ROWS 0x4u

/*
 * Rows of heads, BF16: element (token, head, d) at
 * data + token * token_stride + head * head_stride + d (strides in elements,
 * multiples of 8; data 16-byte aligned).  A slice of a packed projection
 * output, [tokens, heads, head_dim] and [heads, tokens, head_dim] all fit.
 */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
  int heads;
  int reserved; /* must be zero */
} sgr_heads;

/*
 * A paged cache.  The code of position t of a sequence, head h, element d is
 * at page * page_stride + h * head_stride + (t % page_size) * token_stride + d
 * (bytes, multiples of 16) in k and in v, page = block_table[sequence][t /
 * page_size].  [pages, heads, page_size, head_dim] and
 * [pages, page_size, heads, head_dim] both fit; positions must not overlap.
 * E4M3 codes as in skinny_gemm_residual_w8; a NaN is code 0x7F or 0xFF.
 * k_scale, v_scale: [pages, heads] FP32 with scale_stride elements between
 * pages, powers of two in [2^-64, 2^64].
 */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t page_stride;
  int64_t head_stride;
  int64_t token_stride;
  int64_t scale_stride;
  int num_pages;
  int page_size; /* tokens: 16, 32, 64 or 128 */
  int heads;     /* key/value heads */
  int head_dim;  /* 64 or 128 */
} sgr_kv_cache;

/*
 * The sequences of a call.  Sequence b has the new tokens (rows of q, k, v
 * and out) q_start[b] .. q_start[b+1]-1; q_start NULL: one row each, row b.
 * They are the last of its seq_len[b] positions: its i-th of n rows is at
 * position seq_len[b] - n + i.  A row whose position is negative (a padding
 * row: seq_len 0) is not appended, its rotated query and its attention output
 * are zeros.  Rows that no sequence has (q_start[batch] below tokens) are left
 * as they are.  Entries of block_table beyond a sequence's length are not read.
 * The kernel and split of sgr_kv_attention are chosen by max_pages and max_new:
 * any upper bounds are right, close ones fast.
 */
typedef struct {
  const int* block_table; /* [batch, max_pages], row stride table_stride */
  const int* seq_len;     /* [batch] */
  const int* q_start;     /* [batch + 1] or NULL */
  int64_t table_stride;
  int batch;
  int max_pages;
  int tokens;  /* rows in all */
  int max_new; /* upper bound of the rows of one sequence */
} sgr_kv_batch;

/*
 * Norm and rotation.  q_weight, k_weight: BF16 [head_dim], NULL = no norm of
 * that operand.  table: FP32 [table_rows, rot_dim], row p = the rot_dim / 2
 * cosines, then the sines, of position p; NULL = no rotation.  rot_dim: a
 * multiple of 16, at most head_dim; pairs are (i, i + rot_dim / 2), or
 * (2 i, 2 i + 1) where `interleaved` is nonzero.
 */
typedef struct {
  const void* q_weight;
  const void* k_weight;
  const float* table;
  float eps;
  int table_rows;
  int rot_dim;
  int interleaved;
} sgr_norm_rope;

/*
 * Queries and keys of `tokens` rows normalised per head and rotated to
 * positions[row], in one pass: q_out = rope(norm(q)), k_out likewise.  In
 * place where out and in are the same (pointer and strides); any other
 * overlap is SGR_ERR_ALIAS.  k and k_out may both be NULL.  A negative
 * position gives a row of zeros.
 */
int sgr_qk_norm_rope(const sgr_heads* q, const sgr_heads* k, const sgr_heads* q_out, const sgr_heads* k_out,
                     const int* positions, int tokens, int head_dim, const sgr_norm_rope* nr, unsigned flags,
                     void* stream);

/*
 * Appends the new tokens' keys (normalised and rotated to their positions)
 * and values to the cache, and normalises and rotates their queries into
 * q_out (q and q_out may both be NULL), in one launch.
 *
 * A page to which the call writes from its first position on gets the scale
 * of its new tokens; otherwise its scale grows to theirs where it has to, and
 * the codes of its earlier positions are rounded to the new scale (exact but
 * for codes that leave E4M3's range at the lower end).  Positions behind the
 * new tokens are not touched.  Appending the same rows again changes nothing.
 * Infinities and NaN do not count for the scale; NaN stays NaN, infinities and
 * magnitudes above 448 * 2^64 saturate.  No two sequences of a call may write to one page.
 */
int sgr_kv_append(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const sgr_heads* k,
                  const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr, unsigned flags, void* stream);

/*
 * out[row, head] = attention of the row's query over the cached positions
 * t <= position (and t > position - window where window > 0) of its sequence;
 * query head h reads key/value head h / (q->heads / cache->heads).  A row
 * that sees no position gets zeros.  Masked positions have no influence,
 * whatever they hold.  `scale` multiplies the scores (1/sqrt(head_dim) as a
 * rule).  The tensor core sees a query's elements to 2^-18 of its row's largest
 * (with their 8 bits down to 2^-9 of it at least), so a score is good to some
 * 2^-16 of |q| |k| scale.  Weights, each times the value scale of its page, are
 * good to 2^-11 of themselves down to 2^-14 of the row's largest so far, and to
 * 2^-26 of the largest below: n weights far below it are off by n 2^-26 of it
 * together at most.  The sum that divides is of the weights before they are
 * rounded.  workspace: device memory of sgr_kv_attention_workspace() bytes,
 * 16-byte aligned, without initial contents; calls that may overlap on the
 * GPU need one each.
 */
int sgr_kv_attention(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const sgr_heads* out,
                     float scale, int window, void* workspace, int64_t workspace_bytes, unsigned flags, void* stream);

/* Workspace that sgr_kv_attention needs for this batch, `q_heads` query heads
 * and these flags on `device`, in bytes (a smaller one is
 * SGR_ERR_UNSUPPORTED there).  Depends on the sizes in the structures, not on
 * device data.  Host-only apart from a device-attribute query. */
int sgr_kv_attention_workspace(int device, const sgr_kv_cache* cache, const sgr_kv_batch* batch, int q_heads,
                               unsigned flags, int64_t* bytes);

/* Host-only argument checks of the three operators (their exact rules, but
 * for the size of the workspace). */
int sgr_validate_qk_norm_rope(const sgr_heads* q, const sgr_heads* k, const sgr_heads* q_out, const sgr_heads* k_out,
                              const int* positions, int tokens, int head_dim, const sgr_norm_rope* nr);
int sgr_validate_kv_append(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                           const sgr_heads* k, const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr);
int sgr_validate_kv_attention(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                              const sgr_heads* out, float scale, int window);

#ifdef __cplusplus
}
#endif

#endif /* SGR_ATTENTION_H */
