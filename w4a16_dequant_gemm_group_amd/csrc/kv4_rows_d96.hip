// Few-row attention over the 4-bit cache, head_dim 96.
#include "kv4_rows.h"

namespace gq {

hipError_t launch_kv4_rows_96(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s) {
  if (a.c.ng == 3) return kv4::launch_rows_any<96, 3>(a, p, s);
  if (a.c.ng == 1) return kv4::launch_rows_any<96, 1>(a, p, s);
  return hipErrorInvalidValue;
}

}  // namespace gq
