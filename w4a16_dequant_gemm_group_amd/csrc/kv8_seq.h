// Which sequence a row of q, k or v belongs to.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gq {

struct RowSeq {
  int b;             // -1: none
  int64_t first, n;  // its first row, its rows
};

// The sequence that row t belongs to, found by a whole wave: 64 starts a step, as
// few steps as they are 64-fold.  starts (ascending) null: sequence t, row t.  Rows of
// an earlier sequence may end up with a later one only if starts are not ascending;
// every index stays inside the arrays in any case.
__device__ __forceinline__ RowSeq seq_of_row(const int32_t* starts, int64_t batch, int64_t rows, int64_t t, int lane) {
  RowSeq s{-1, 0, 0};
  if (!starts) {
    if (t < batch) s = RowSeq{(int)t, t, 1};
    return s;
  }
  int64_t lo = 0, len = batch;
  bool first = true;
  while (len > 1 || first) {
    first = false;
    const int64_t step = (len + 63) >> 6, i = lo + lane * step;
    const bool le = i < lo + len && (int64_t)starts[i < batch ? i : batch - 1] <= t;
    const int c = __popcll(__ballot(le));
    if (c == 0) return s;
    const int64_t at = lo + (int64_t)(c - 1) * step, end = lo + len;
    lo = at;
    len = at + step < end ? step : end - at;
  }
  int64_t x = starts[lo], y = starts[lo + 1];
  x = x < 0 ? 0 : (x > rows ? rows : x);
  y = y < x ? x : (y > rows ? rows : y);
  if (t < x || t >= y) return s;
  s.b = (int)lo;
  s.first = x;
  s.n = y - x;
  return s;
}

}  // namespace gq
