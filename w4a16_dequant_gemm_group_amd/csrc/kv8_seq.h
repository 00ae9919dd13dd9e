// Which sequence a row of q, k or v belongs to.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gq {

struct RowSeq {
  int b;             // -1: none
  int64_t first, n;  // its first row, its rows
  int kv;            // its kv_lens
};

// The sequence that row t belongs to, found by a whole wave: 64 starts a step, as
// few steps as they are 64-fold; up to 64 sequences cost one round of loads.  starts
// (ascending) null: sequence t, row t.  Where starts are not ascending a row may end up
// with a sequence that is not its own, but every index stays inside the arrays.
__device__ __forceinline__ RowSeq seq_of_row(const int32_t* starts, const int32_t* kv_lens, int64_t batch, int64_t rows,
                                             int64_t t, int lane) {
  RowSeq s{-1, 0, 0, 0};
  if (!starts) {
    if (t < batch) s = RowSeq{(int)t, t, 1, kv_lens[t]};
    return s;
  }
  if (batch < 1) return s;
  int64_t lo = 0, len = batch;
  int x, y, kv;
  for (;;) {
    const int64_t step = (len + 63) >> 6, i = lo + lane * step;
    const bool in = i < lo + len;
    const int64_t at = in ? i : batch - 1;
    x = starts[at];
    y = starts[at + 1];
    kv = kv_lens[at];
    const int c = __popcll(__ballot(in && (int64_t)x <= t));
    if (c == 0) return s;
    const int64_t next = lo + (int64_t)(c - 1) * step, end = lo + len;
    if (step == 1) {
      lo = next;
      x = __builtin_amdgcn_readlane(x, c - 1);
      y = __builtin_amdgcn_readlane(y, c - 1);
      kv = __builtin_amdgcn_readlane(kv, c - 1);
      break;
    }
    lo = next;
    len = next + step < end ? step : end - next;
  }
  const int64_t a = x < 0 ? 0 : (x > rows ? rows : (int64_t)x);
  const int64_t b = y < a ? a : (y > rows ? rows : (int64_t)y);
  if (t < a || t >= b) return s;
  s.b = (int)lo;
  s.first = a;
  s.n = b - a;
  s.kv = kv;
  return s;
}

}  // namespace gq
