/*
 * gq_kv8.h - C ABI of libgq, fourth part: a paged key/value cache held in 8 bits
 * with one scale for each block of 16 tokens and head, the attention that reads
 * it, and the choice of the pages that a query reads, for AMD MI355X (gfx950).
 *
 * A block is 16 consecutive positions of a sequence, from a multiple of 16 on, in
 * one key/value head, keys and values apart.  Its codes are integers of -127 .. 127:
 *   x^ = S q,   q = round(x / S),   S = max(S of the older tokens, max |x| / 127, 2^-40)
 * with round half to even and S in fp32 (the quotient rounded once); "older tokens"
 * are those that lie in the block before the call, and where S grows their codes
 * become round(q S_old / S).  A value below 2^-41 is stored as 0.
 *
 * The conventions of gq.h hold for every entry point: device pointers, caller owns
 * every buffer, no allocation, no synchronization, host-side validation before
 * anything is enqueued, thread-safe, gfx950 only.  All calls can be captured into
 * a graph.
 *
 * The cache
 *   One buffer of gq_kv8_cache_bytes() bytes, 16-byte aligned, holds n_pages
 *   pages of page_size tokens.  Token slot t is position t % page_size of page
 *   t / page_size; a sequence is a row of page numbers, its token at position i lives
 *   in page page_table[row][i / page_size].  The order of bytes is the library's own;
 *   gq_kv8_append and gq_kv8_read are the way in and out.  New memory needs no initial
 *   content: a slot is read as defined only after it was written.
 * Bounds
 *   [n_pages, kv_heads, 2, head_dim] in the keys' own type: the smallest and the
 *   largest of each channel over the keys of a page, as they were appended.  Optional;
 *   gq_kv8_append keeps them up to date, gq_kv8_select reads them.
 */
#ifndef GQ_KV8_H_
#define GQ_KV8_H_

#include "gq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of a cache.  head_dim 64, 96, 128 or 256 (other multiples of 32:
 * UNSUPPORTED); page_size a power of two, 16..1024; kv_heads 1..65535. */
typedef struct {
  int32_t kv_heads;
  int32_t head_dim;
  int32_t page_size; /* tokens per page */
} gq_kv8_layout;

/* Bytes of a cache of n_pages pages: per token and head 2 head_dim bytes of codes,
 * and 8 bytes of scales per block.  Host only.  Errors: INVALID_ARG (n_pages < 1 or
 * >= 2^31, 2^62 bytes or more (so in every call), the layout's limits, a NULL
 * `bytes`), UNSUPPORTED (head_dim). */
gq_status gq_kv8_cache_bytes(int64_t n_pages, gq_kv8_layout layout, size_t* bytes);

/* Quantize the next tokens of sequences into the cache.  Sequence b brings the rows
 * starts[b] .. starts[b + 1] - 1 of k and v (row b alone where starts is NULL); its
 * length with them is kv_lens[b], so the i-th of its n goes to position
 * kv_lens[b] - n + i.
 *   k, v    [tokens, kv_heads, head_dim] of dtype (GQ_BF16 or GQ_F16); *_stride are the
 *           elements from one token, and from one head, to the next (multiples of 8),
 *           head_dim contiguous, 16-byte aligned: slices of a fused projection's output
 *           are taken as they are.  Infinities count as the type's largest value,
 *           NaN as 0
 *   page_table [batch, table_pages] int32; tokens at negative positions, past the table
 *           or in a page number outside 0 .. n_pages - 1 are skipped.  Pages that a call
 *           writes to belong to one sequence
 *   kv_lens [batch] int32
 *   starts  [batch + 1] int32, ascending, or NULL for one token each (tokens >= batch
 *           then; rows behind the last sequence are ignored); values are clamped to
 *           0 .. tokens
 *   bounds  as above, 16-byte aligned, or NULL.  A page's bounds start over when its
 *           first position is written; else they are widened
 * Where a call begins inside a block, the tokens before it in the block are ones that were
 * appended (their scale is read and kept at least, whatever the memory holds), and with
 * bounds those of its page were, with bounds.  Where a sequence is cut back and appended to
 * again, the scale (and the bounds) of the block (page) it is cut in stay as wide as they
 * were.  Errors: INVALID_ARG
 * (layout, shapes, NULL), UNSUPPORTED (dtype, head_dim, device), MISALIGNED. */
typedef struct {
  const void* k;
  int64_t k_token_stride, k_head_stride;
  const void* v;
  int64_t v_token_stride, v_head_stride;
  gq_dtype dtype;
  int64_t tokens;
  uint8_t* cache;
  int64_t n_pages;
  gq_kv8_layout layout;
  const int32_t* page_table;
  int64_t batch, table_pages;
  const int32_t* kv_lens;
  const int32_t* starts;
  void* bounds;
} gq_kv8_append_args;

gq_status gq_kv8_append(const gq_kv8_append_args* args, void* stream);

/* The values that the cache stands for at the given slots.
 *   slots [tokens] int64
 *   k, v  [tokens, kv_heads, head_dim] of out_dtype, contiguous, 16-byte
 *         aligned: GQ_F32 S q rounded once, GQ_BF16 / GQ_F16 that rounded again
 *         (nearest-even; fp16 beyond its range: infinity).  A slot out of range reads
 *         as zeros.
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim, device), MISALIGNED. */
gq_status gq_kv8_read(const uint8_t* cache, int64_t n_pages, gq_kv8_layout layout,
                      const int64_t* slots, int64_t tokens, void* k, void* v, gq_dtype out_dtype,
                      void* stream);

/* Attention of query rows over a cache.  Sequence b has queries q_starts[b] ..
 * q_starts[b + 1] - 1 (row b alone where q_starts is NULL) and kv_lens[b]
 * keys; its last query sits at position kv_lens[b] - 1, so its i-th of n is at
 * p = kv_lens[b] - n + i.  Query head h reads key/value head
 * h / (q_heads / kv_heads).  A query sees the keys j < kv_lens[b], with causal
 * set only j <= p, and with window > 0 only j > p - window.  A query that sees
 * no key gives o = 0 and lse = -infinity.
 *   s_j = scale * sum_d q_d k^_jd,  p = softmax over the keys that are seen,
 *   o = sum_j p_j v^_j,  lse = log sum_j exp(s_j)
 *   q          [q_tokens, q_heads, head_dim] of dtype, finite values; strides as in
 *              gq_kv8_append
 *   page_table [batch, table_pages] int32, or [batch, kv_heads, table_pages] with
 *              head_tables set: pages of each key/value head's own (gq_kv8_select).
 *              Entries past a sequence's length are not read; the keys of a page
 *              number outside 0 .. n_pages - 1 are not seen
 *   kv_lens    [batch] int32; negative counts as 0, more than table_pages *
 *              page_size as that many
 *   q_starts   [batch + 1] int32, ascending, or NULL for one query each
 *              (q_tokens >= batch then); values are clamped to 0 .. q_tokens.
 *              Rows of `out` that belong to no sequence are not written
 *   max_q_len, max_kv_len  host-side bounds of the query counts and of kv_lens.
 *              They choose kernels and the split; results hold without them
 *              being tight, and also where a length exceeds its bound
 *   scale      factor of the scores, finite and > 0; 1 / sqrt(head_dim) by custom
 *   out        [q_tokens, q_heads, head_dim] of dtype, contiguous, 16-byte aligned
 *   lse        [q_tokens, q_heads] float, or NULL
 * Scores, softmax statistics and outputs are kept in fp32.  The matrix cores take codes
 * exactly and queries as fp16 times a power of two per row (elements below 2^-29 of a
 * row's largest have fewer bits); weights times value scales are rounded to fp16 once
 * (2^-11), those below 2^-22 of a row's largest have fewer bits, below 2^-33 none.  What that
 * leaves is carried along (2^-22 remains) for fp16 results of a sequence of at most 8 rows
 * (queries times query heads per key/value head) in a call whose max_q_len makes at most 16;
 * with a larger max_q_len it is not.  Scores have to lie within +-2^22: beyond, their own
 * rounding moves weights by more than fp16 has room for, and results may be infinite or
 * NaN.  scale times the largest |q| of a row has fewer bits below 2^-112. */
typedef struct {
  const void* q;
  int64_t q_token_stride, q_head_stride;
  int64_t q_tokens;
  int32_t q_heads;
  gq_dtype dtype; /* GQ_BF16 or GQ_F16, of q and out */
  const uint8_t* cache;
  int64_t n_pages;
  gq_kv8_layout layout;
  const int32_t* page_table;
  int64_t batch, table_pages;
  int32_t head_tables; /* 0 or 1 */
  const int32_t* kv_lens;
  const int32_t* q_starts;
  int64_t max_q_len, max_kv_len;
  int32_t causal; /* 0 or 1 */
  int32_t window; /* 0: no window; > 0 needs causal */
  float scale;
  void* out;
  float* lse;
} gq_kv8_attention_args;

/* Scratch (bytes) of gq_kv8_attention for these arguments (of which only the
 * sizes, the layout and the options are looked at): partial outputs where a
 * sequence's keys are split over workgroups.  0 where nothing is split.
 * Queries the current device's compute-unit count when a device is present
 * (256 otherwise).  Errors: INVALID_ARG, UNSUPPORTED (head_dim, dtype). */
gq_status gq_kv8_attention_workspace_size(const gq_kv8_attention_args* args, size_t* bytes);

/* The attention.  workspace: device memory of at least
 * gq_kv8_attention_workspace_size() bytes, 16-byte aligned, of any content
 * (NULL allowed when that size is 0); nothing else may use it until the call's
 * kernels complete.  The result does not depend on timing.  Errors:
 * INVALID_ARG (shapes: q_heads a multiple of kv_heads, at most 64 query heads
 * per key/value head; window without causal; NULL; a workspace that is missing
 * or small), UNSUPPORTED (dtype, head_dim, device), MISALIGNED. */
gq_status gq_kv8_attention(const gq_kv8_attention_args* args, void* workspace,
                           size_t workspace_bytes, void* stream);

/* The pages that each query reads, by bounds of its scores.  Sequences, queries and
 * their positions p are those of gq_kv8_attention (causal); a query at p has the pages
 * 0 .. p / page_size of its row of page_table.  For query t and key/value head h the
 * score of a page is the largest, over the query heads of h, of
 *   sum_d max(q_d min_d, q_d max_d)
 * which no key of the page exceeds (as it was appended), summed in binary64 and taken as
 * q_d max_d where q_d is positive, q_d min_d where it is negative (which tells them apart
 * for an infinite q_d beside a bound of 0: that product alone is NaN); sums that are NaN do not
 * count.  Of n pages min(n, keep) are taken: the first `first` and the last
 * `last`, then those with the largest scores, of equal ones the earlier.  A page number
 * outside 0 .. n_pages - 1 has the lowest score, as has a page whose sums are all NaN.
 *   q       [q_tokens, q_heads, head_dim] of dtype, the bounds' own; strides as in
 *           gq_kv8_append
 *   pages   [q_tokens, kv_heads, keep] int32, 4-byte aligned: page numbers in the order
 *           of their positions, then -1
 *   lens    [q_tokens] int32: the keys that these pages hold up to p
 * so that gq_kv8_attention with batch = q_tokens, one query each, head_tables set,
 * page_table = pages and kv_lens = lens attends over them.  A query at a negative
 * position, or that belongs to no sequence, gets lens 0 and pages of -1.  Here a length
 * beyond max_kv_len, rounded up to whole pages, counts as that many. */
typedef struct {
  const void* q;
  int64_t q_token_stride, q_head_stride;
  int64_t q_tokens;
  int32_t q_heads;
  gq_dtype dtype;
  const void* bounds;
  int64_t n_pages;
  gq_kv8_layout layout;
  const int32_t* page_table;
  int64_t batch, table_pages;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  int64_t max_kv_len;
  int32_t keep, first, last;
  int32_t* pages;
  int32_t* lens;
} gq_kv8_select_args;

/* Scratch (bytes) of gq_kv8_select: the scores.  Host only.  Errors as below. */
gq_status gq_kv8_select_workspace_size(const gq_kv8_select_args* args, size_t* bytes);

/* The choice.  workspace as for gq_kv8_attention.  Errors: INVALID_ARG (shapes: q_heads
 * as above; keep < 1 or > 65536, first < 0, last < 1, first + last > keep; q_tokens *
 * kv_heads of 2^31 or more, or that times keep of 2^40; NULL; a workspace that is missing
 * or small), UNSUPPORTED (dtype, head_dim, device), MISALIGNED. */
gq_status gq_kv8_select(const gq_kv8_select_args* args, void* workspace, size_t workspace_bytes,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_KV8_H_ */
