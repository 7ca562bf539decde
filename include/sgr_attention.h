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
 *                     (sgr_kv_mask: a window, sinks, a tree of drafted tokens)
 *   mass              mass_t += sum over rows and a group's heads of
 *                     p_t / sum_t p_t: the attention weight that a cached
 *                     position has got
 *   eviction          the positions with the largest mass stay, and move to
 *                     new pages
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
 * What a row sees.  Its position is its place in the sequence, p; without a
 * mask it sees the positions t <= p.
 *   window  > 0: only t > p - window of them, and
 *   sinks   the first positions of the sequence, t < sinks, all the same
 *           (t <= p as ever; without a window they make no difference).
 *   tree    rows are drafted tokens: of the n new tokens of its sequence a row
 *           sees those whose bits are set, bit j % 64 of
 *           tree[row * tree_stride + j / 64] for the j-th (itself among them
 *           only if set; a window does not count between them), and of the
 *           positions before the new ones those that a row at position
 *           max(seq_len - n, 0) + max(bits set, 1) - 1 sees: a row without any
 *           stands where the first new token does.  Bits from n on are not
 *           looked at, nor those of padding rows.  NULL: not a tree.
 *           tree_words: words of a row, at least max_new / 64 rounded up.
 * A padding row (its place negative) sees nothing, and no row sees one.  The
 * words of tree may share no memory with what a call writes (SGR_ERR_ALIAS).
 */
typedef struct {
  const uint64_t* tree; /* [tokens, tree_words], 8-byte aligned */
  int64_t tree_stride;  /* words from row to row */
  int tree_words;
  int window;
  int sinks;
  int reserved; /* must be zero */
} sgr_kv_mask;

/*
 * The attention weight that each position of a cache has got, FP32: position t
 * of a sequence, head h at data + page * page_stride + h * head_stride +
 * t % page_size (elements), page as in sgr_kv_cache.
 */
typedef struct {
  float* data;
  int64_t page_stride;
  int64_t head_stride;
} sgr_kv_masses;

/*
 * What stays of each sequence.  n = min(keep[b], seq_len[b]) positions: the
 * first min(first, n), the last min(recent, what is left of n), and of those
 * between the ones with the largest mass (of equal ones the first; a NaN
 * counts as larger than all).  table: the pages that they move to.
 */
typedef struct {
  const int* keep;  /* [batch], not negative */
  const int* table; /* [batch, max_pages], row stride table_stride */
  int* kept;        /* [batch, heads, max_pages * page_size]: the positions that stay, ascending; entries from n on are left */
  int* new_len;     /* [batch]: n */
  int64_t table_stride;
  int max_pages;
  int first;
  int recent;
  int reserved; /* must be zero */
} sgr_kv_eviction;

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
 * The same, with row r's query and key rotated to positions[r] instead of its
 * place in the cache: drafted tokens of a tree stand at their depth, and new
 * tokens of a sequence that has lost positions (sgr_kv_evict) behind all that
 * it ever had.  A negative position counts as 0 and records code 7; without a
 * rotation table positions are not looked at.  They may share no memory with
 * q_out or the cache (SGR_ERR_ALIAS).  positions NULL: as sgr_kv_append.
 */
int sgr_kv_append_at(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const sgr_heads* k,
                     const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr, const int* positions,
                     unsigned flags, void* stream);

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

/*
 * The same over the positions that `mask` says (NULL: all up to a row's own),
 * and, with lse not NULL, lse[row * q->heads + head] = log sum_t p_t, FP32
 * (-infinity for a row that sees no position; rows of no sequence are left).
 * Takes sgr_kv_attention's workspace.
 */
int sgr_kv_attention_masked(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                            const sgr_heads* out, float* lse, float scale, const sgr_kv_mask* mask, void* workspace,
                            int64_t workspace_bytes, unsigned flags, void* stream);

/*
 * Adds to every cached position's mass, for each key/value head, the attention
 * weight that the batch's rows give it with the heads of its group:
 *
 *   mass[t, h] += sum_{rows, heads of h} exp(scale q.k_t - lse[row, head])
 *
 * over the rows that see t (mask: as sgr_kv_attention_masked; lse: what that
 * call wrote for the same q, scale and mask).  The new tokens' own positions
 * are set, not added to: a page needs no clearing before it is used where this
 * call follows every append.  A position appended without it has the mass that
 * its place had, of the page's last user or of a draft (NaN or large, perhaps,
 * and then sgr_kv_evict keeps it): set it to zero at the append.  Masked
 * weights have no part, whatever the position holds; positions that no row sees
 * keep their mass.  Scores as in sgr_kv_attention for few rows (queries to
 * 2^-22 of the row's largest), sums in FP32, of a sequence in a fixed order.
 * batch->max_new has to be an upper bound (a sequence with more rows is
 * recorded, code 7, and its later rows may be missing).  Sequences may share
 * pages of older positions (a common prompt): such a position gets the weights
 * of all of them, added in any order (its last bits may differ from run to
 * run).  A page of new positions may occur once in a call's tables.
 * workspace: sgr_kv_mass_workspace() bytes, 16-byte aligned, without initial
 * contents, one for each call that may overlap; NULL where 0 bytes are needed.
 */
int sgr_kv_mass(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const float* lse,
                const sgr_kv_masses* mass, float scale, const sgr_kv_mask* mask, void* workspace,
                int64_t workspace_bytes, unsigned flags, void* stream);

/* Workspace that sgr_kv_mass needs for this batch and `q_heads` query heads, in
 * bytes: 0 where a key/value head has at most 128 rows of a sequence (max_new
 * times the group), else 4 bytes a position and key/value head for every 128 of
 * them.  Depends on the sizes in the structures alone.  SGR_ERR_UNSUPPORTED for
 * sizes that sgr_kv_mass refuses. */
int sgr_kv_mass_workspace(const sgr_kv_cache* cache, const sgr_kv_batch* batch, int q_heads, int64_t* bytes);

/*
 * Evicts positions by their mass: for each sequence (its block table and
 * seq_len; q_start and the rows do not matter) and key/value head chooses what
 * stays and moves it, in order, to the positions 0 .. n - 1 of the pages of
 * `eviction->table`: codes, rounded to new page scales (as sgr_kv_append
 * chooses them), and mass.  Heads keep positions of their own, the same number
 * each.  The old pages are read only; a new page may be none of them, nor
 * occur twice (undefined contents otherwise).  Entries of the table beyond n
 * positions do not matter; positions of a new page behind them are not written.
 * Keys stay rotated to the positions that they had: go on with
 * sgr_kv_append_at.  A bad old page's positions count as the smallest mass and
 * move as zeros; n beyond the new table's room is cut to it; both are recorded
 * (code 7).  Cached values that are NaN do not count for the scale and stay NaN.
 */
int sgr_kv_evict(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_kv_masses* mass,
                 const sgr_kv_eviction* eviction, unsigned flags, void* stream);

/* Workspace that sgr_kv_attention needs for this batch, `q_heads` query heads
 * and these flags on `device`, in bytes (a smaller one is
 * SGR_ERR_UNSUPPORTED there).  Depends on the sizes in the structures, not on
 * device data.  Host-only apart from a device-attribute query. */
int sgr_kv_attention_workspace(int device, const sgr_kv_cache* cache, const sgr_kv_batch* batch, int q_heads,
                               unsigned flags, int64_t* bytes);

/* Host-only argument checks of the operators (their exact rules, but for the
 * size of the workspace). */
int sgr_validate_qk_norm_rope(const sgr_heads* q, const sgr_heads* k, const sgr_heads* q_out, const sgr_heads* k_out,
                              const int* positions, int tokens, int head_dim, const sgr_norm_rope* nr);
int sgr_validate_kv_append(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                           const sgr_heads* k, const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr);
int sgr_validate_kv_attention(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                              const sgr_heads* out, float scale, int window);
int sgr_validate_kv_append_at(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                              const sgr_heads* k, const sgr_heads* v, const sgr_heads* q_out, const sgr_norm_rope* nr,
                              const int* positions);
int sgr_validate_kv_attention_masked(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q,
                                     const sgr_heads* out, const float* lse, float scale, const sgr_kv_mask* mask);
int sgr_validate_kv_mass(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_heads* q, const float* lse,
                         const sgr_kv_masses* mass, float scale, const sgr_kv_mask* mask);
int sgr_validate_kv_evict(const sgr_kv_cache* cache, const sgr_kv_batch* batch, const sgr_kv_masses* mass,
                          const sgr_kv_eviction* eviction);

#ifdef __cplusplus
}
#endif

#endif /* SGR_ATTENTION_H */
