/*
 * gq_rope.h - C ABI of libgq, third part: rotary positions of queries and keys,
 * for AMD MI355X (gfx950).
 *
 * The first rot_dim channels of every head form rot_dim / 2 pairs (a_i, b_i):
 * channels i and i + rot_dim / 2, or, interleaved, 2 i and 2 i + 1.  A token at
 * position p turns pair i by the angle t = p f_i:
 *   a' = m (a cos t - b sin t),   b' = m (b cos t + a sin t)
 * with a frequency f_i per pair and one amplitude m; channels from rot_dim on
 * are passed through.  The inverse turns by -t: the transposed map, and so the
 * gradient of the operator (m included) for a gradient of its result.
 *
 * The conventions of gq.h hold: device pointers unless marked "host", the caller
 * owns every buffer, no allocation, no synchronization, host-side validation
 * before anything is enqueued, thread-safe, gfx950 only; the call can be captured
 * into a graph.
 */
#ifndef GQ_ROPE_H_
#define GQ_ROPE_H_

#include "gq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How frequencies are scaled for contexts longer than `original_length`, the one
 * a model was trained for.  With f = base^(-2 i / rot_dim), s = factor:
 *   NONE        f
 *   LINEAR      f / s
 *   WAVELENGTH  by n = original_length f / (2 pi), the turns of a pair over that
 *               length: n <= low: f / s, n >= high: f, between them
 *               (1 - t) f / s + t f with t = (n - low) / (high - low)
 *   YARN        the same mixture with t falling over the pair's index i, from 1 at
 *               floor(c(high)) to 0 at ceil(c(low)) where c(n) =
 *               rot_dim ln(original_length / (2 pi n)) / (2 ln base) is the index
 *               that makes n turns (both held in 0 .. rot_dim - 1; at least 0.001
 *               apart); the amplitude is 0.1 ln s + 1
 * All in binary64. */
typedef enum {
  GQ_ROPE_NONE = 0,
  GQ_ROPE_LINEAR = 1,
  GQ_ROPE_WAVELENGTH = 2,
  GQ_ROPE_YARN = 3
} gq_rope_scaling_kind;

typedef struct {
  int32_t kind;           /* gq_rope_scaling_kind; the fields it does not use are ignored */
  double factor;          /* >= 1 */
  double original_length; /* > 0 */
  double low, high;       /* turns, 0 < low < high */
} gq_rope_scaling;

/* Frequencies and amplitude.  Host only: freqs (host) [rot_dim / 2], amplitude
 * (host) one value.  Errors: INVALID_ARG (rot_dim odd, < 2 or > 1024, base not a
 * finite number > 1, the scaling's limits, NULL). */
gq_status gq_rope_frequencies(int64_t rot_dim, double base, gq_rope_scaling scaling, double* freqs,
                              double* amplitude);

/* The rotation.
 *   x, out     [tokens, heads, head_dim] of dtype (GQ_BF16, GQ_F16 or GQ_F32); *_stride
 *              are the elements from one token, and from one head, to the next,
 *              head_dim contiguous: slices of a fused projection's output are taken as
 *              they are.  out may be x itself, with the same strides; other overlaps
 *              are not allowed, nor are rows of out that overlap
 *   positions  [tokens] int64, of any sign
 *   freqs      [rot_dim / 2] double
 * Angles are products in binary64, reduced to a turn there (off by 2^-52 of the
 * angle); sines, products and sums are fp32, rounded once to dtype (nearest-even).
 * Errors: INVALID_ARG (tokens < 0 or > 2^30, heads < 0 or > 65536, head_dim odd or
 * outside 2 .. 1024, rot_dim odd or outside 2 .. head_dim, strides beyond 2^40,
 * amplitude not finite, x == out with other strides, rows of out that overlap each
 * other, NULL), MISALIGNED (x, out to their elements, positions and freqs to 8 bytes),
 * UNSUPPORTED (device).  Other overlaps of x and out are the caller's to avoid. */
typedef struct {
  const void* x;
  int64_t x_token_stride, x_head_stride;
  void* out;
  int64_t out_token_stride, out_head_stride;
  gq_dtype dtype;
  int64_t tokens, heads;
  int32_t head_dim, rot_dim;
  const int64_t* positions;
  const double* freqs;
  float amplitude;
  int32_t interleaved; /* 0: pairs (i, i + rot_dim / 2), 1: (2 i, 2 i + 1) */
  int32_t inverse;     /* 0 or 1 */
} gq_rope_args;

gq_status gq_rope(const gq_rope_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_ROPE_H_ */
