// Many-row attention over the 4-bit cache, head_dim 256.
#include "kv4_tile.h"

namespace gq {

hipError_t launch_kv4_tile_256(const Kv4Attn& a, const Kv4Plan& p, hipStream_t s) {
  if (a.c.ng == 8) return kv4::launch_tile<256, 8>(a, p, s);
  if (a.c.ng == 4) return kv4::launch_tile<256, 4>(a, p, s);
  if (a.c.ng == 2) return kv4::launch_tile<256, 2>(a, p, s);
  if (a.c.ng == 1) return kv4::launch_tile<256, 1>(a, p, s);
  return hipErrorInvalidValue;
}

}  // namespace gq
