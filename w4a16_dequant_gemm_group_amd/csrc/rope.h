// Rotary positions: what the kernel gets.
#pragma once

#include "gq_internal.h"
#include "gq_rope.h"

namespace gq {

struct Rope {
  const uint8_t* x;
  uint8_t* out;
  int64_t x_ts, x_hs, out_ts, out_hs;   // bytes
  const int64_t* positions;
  const double* freqs;
  int64_t tokens;
  int32_t heads, d, rot;
  float amplitude, sign;                // sign: -1 for the inverse
  int32_t tail;                         // channels from rot on have to be copied
  int32_t items;                        // pieces of a head: of pairs, then of the tail
  int32_t pair_items;
  int32_t tokens_per_group;
};

hipError_t launch_rope(const gq_rope_args& a, hipStream_t s);

}  // namespace gq
