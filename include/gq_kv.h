/*
 * gq_kv.h - C ABI of libgq, second part: a paged key/value cache held in 4 bits
 * and the attention that reads it, for AMD MI355X (gfx950).
 *
 * Keys and values of one layer are quantized as they are written, with the
 * group quantizer of gq.h (its storage contract, bits = 4): per token and
 * key/value head the head_dim channels form groups of group_size, each with an
 * fp16 scale S and, asymmetric, an integer zero point z:
 *   q = clamp(round(x / S) + z, 0, 15),   x^ = S (q - z)       (z = 8 symmetric)
 * Attention works on the values x^ that the cache stands for and never writes
 * them to memory:
 *   s_j = scale * sum_d q_d k^_jd,  p = softmax over the keys that are seen,
 *   o = sum_j p_j v^_j,  lse = log sum_j exp(s_j).
 *
 * The conventions of gq.h hold for every entry point: device pointers, caller
 * owns every buffer, no allocation, no synchronization, host-side validation
 * before anything is enqueued, thread-safe, gfx950 only.  All calls can be
 * captured into a graph.
 *
 * The cache
 *   One buffer of gq_kv4_cache_bytes() bytes, 16-byte aligned, holds n_pages
 *   pages of page_size tokens.  Token slot t is position t % page_size of page
 *   t / page_size.  A sequence is a row of page numbers: its token at position
 *   i lives in page page_table[row][i / page_size].  The order of bytes inside
 *   a page is the library's own; gq_kv4_write and gq_kv4_read are the way in
 *   and out.  New memory needs no initial content: a slot is read as defined
 *   only after it was written.
 */
#ifndef GQ_KV_H_
#define GQ_KV_H_

#include "gq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of a cache.  head_dim 64, 96, 128 or 256 (others: UNSUPPORTED);
 * group_size a multiple of 32 that divides head_dim; page_size a power of two,
 * 16..1024; kv_heads 1..65535. */
typedef struct {
  int32_t kv_heads;
  int32_t head_dim;
  int32_t page_size;  /* tokens per page */
  int32_t group_size; /* channels per scale */
  int32_t symmetric;  /* 0: scale + zero point, 1: scale only */
} gq_kv4_layout;

/* Bytes of a cache of n_pages pages: per token and head, for keys and for
 * values, head_dim / 2 bytes of codes and 2 (symmetric) or 4 bytes per group.
 * Host only.  Errors: INVALID_ARG (n_pages < 1 or >= 2^31, 2^63 bytes or more
 * (so in every call), the layout's limits, a NULL `bytes`), UNSUPPORTED (head_dim). */
gq_status gq_kv4_cache_bytes(int64_t n_pages, gq_kv4_layout layout, size_t* bytes);

/* Quantize keys and values into the cache.
 *   k, v   [tokens, kv_heads, head_dim] of dtype (GQ_BF16 or GQ_F16), finite
 *          values; *_stride are the elements from one token, and from one head,
 *          to the next (multiples of 8), head_dim contiguous, 16-byte aligned:
 *          slices of a fused projection's output are taken as they are
 *   slots  [tokens] int64 slot numbers.  A slot outside 0 .. n_pages *
 *          page_size - 1 (-1 by custom) is skipped.  Two tokens of one call on
 *          the same slot leave one of them, or a mix of both.
 * The codes, scales and zero points are those of gq_quantize_groups bit for
 * bit, but for the scale of a group of zeros, which is kept as 0 and not 1 (it
 * stands for zeros either way).  An infinite input saturates its group's scale; NaN leaves its group
 * with unspecified but finite values.  Errors: INVALID_ARG (layout, shapes,
 * NULL), UNSUPPORTED (dtype, head_dim, device), MISALIGNED. */
gq_status gq_kv4_write(const void* k, int64_t k_token_stride, int64_t k_head_stride,
                       const void* v, int64_t v_token_stride, int64_t v_head_stride,
                       gq_dtype dtype, int64_t tokens, const int64_t* slots, uint8_t* cache,
                       int64_t n_pages, gq_kv4_layout layout, void* stream);

/* The values that the cache stands for at the given slots.
 *   k, v  [tokens, kv_heads, head_dim] of out_dtype, contiguous, 16-byte
 *         aligned: GQ_F32 exact, GQ_BF16 / GQ_F16 nearest-even (fp16 beyond its
 *         range: infinity).  A slot out of range reads as zeros.
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim, device), MISALIGNED. */
gq_status gq_kv4_read(const uint8_t* cache, int64_t n_pages, gq_kv4_layout layout,
                      const int64_t* slots, int64_t tokens, void* k, void* v, gq_dtype out_dtype,
                      void* stream);

/* Attention of query rows over a cache.  Sequence b has queries q_starts[b] ..
 * q_starts[b + 1] - 1 (row b alone where q_starts is NULL) and kv_lens[b]
 * keys; its last query sits at position kv_lens[b] - 1, so its i-th of n is at
 * p = kv_lens[b] - n + i.  Query head h reads key/value head
 * h / (q_heads / kv_heads).  A query sees the keys j < kv_lens[b], with causal
 * set only j <= p, and with window > 0 only j > p - window.  A query that sees
 * no key gives o = 0 and lse = -infinity.
 *   q          [q_tokens, q_heads, head_dim] of dtype; strides as in gq_kv4_write
 *   page_table [batch, table_pages] int32.  Entries past a sequence's length
 *              are not read; the keys of a page number outside 0 .. n_pages - 1
 *              are not seen
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
 * Scores, softmax statistics and outputs are kept in fp32.  The matrix cores
 * take keys exactly (integers, or two fp16 parts) and queries as fp16 times a power
 * of two per row (elements below 2^-29 of a row's largest have fewer bits); weights,
 * and for more than 32 rows per key/value head values too, are rounded to fp16 once
 * (2^-11), for fp16 results of at most 8 rows the weights and of more than 32 rows
 * the values not at all.  Weights below 2^-22 of a row's largest have fewer bits
 * (2^-25 for up to 32 rows, of weight times value scale), below 2^-33 (2^-36) none.
 * For more than 32 rows keys and values are also off by up to 2^-33 of the largest
 * element among the 16 tokens of a sub-block.  Scores have to lie in fp32's range. */
typedef struct {
  const void* q;
  int64_t q_token_stride, q_head_stride;
  int64_t q_tokens;
  int32_t q_heads;
  gq_dtype dtype; /* GQ_BF16 or GQ_F16, of q and out */
  const uint8_t* cache;
  int64_t n_pages;
  gq_kv4_layout layout;
  const int32_t* page_table;
  int64_t batch, table_pages;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  int64_t max_q_len, max_kv_len;
  int32_t causal; /* 0 or 1 */
  int32_t window; /* 0: no window; > 0 needs causal */
  float scale;
  void* out;
  float* lse;
} gq_kv4_attention_args;

/* Scratch (bytes) of gq_kv4_attention for these arguments (of which only the
 * sizes, the layout and the options are looked at): partial outputs where a
 * sequence's keys are split over workgroups.  0 where nothing is split.
 * Queries the current device's compute-unit count when a device is present
 * (256 otherwise).  Errors: INVALID_ARG, UNSUPPORTED (head_dim, dtype). */
gq_status gq_kv4_attention_workspace_size(const gq_kv4_attention_args* args, size_t* bytes);

/* The attention.  workspace: device memory of at least
 * gq_kv4_attention_workspace_size() bytes, 16-byte aligned, of any content
 * (NULL allowed when that size is 0); nothing else may use it until the call's
 * kernels complete.  The result does not depend on timing.  Errors:
 * INVALID_ARG (shapes: q_heads a multiple of kv_heads, at most 64 query heads
 * per key/value head; window without causal; NULL; a workspace that is missing
 * or small), UNSUPPORTED (dtype, head_dim, device), MISALIGNED. */
gq_status gq_kv4_attention(const gq_kv4_attention_args* args, void* workspace,
                           size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_KV_H_ */
