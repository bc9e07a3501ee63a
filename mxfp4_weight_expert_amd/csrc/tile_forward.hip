// Forward products of 16-bit matrices in tiles, plain and gated.
#include "tile_launch.h"

namespace moe {

hipError_t launch_tile_forward(const TileArgs& a, bool gated, hipStream_t st) {
  const int64_t nr = (a.R + (gated ? kTile / 2 : kTile) - 1) / (gated ? kTile / 2 : kTile);
  const int64_t tiles = (a.M + kTile - 1) / kTile + (a.offsets != nullptr ? a.E : 0);
  if (a.dtype == MOE_DTYPE_BF16)
    return gated ? tile_go<kForward, true, MOE_DTYPE_BF16>(a, tiles * nr, st)
                 : tile_go<kForward, false, MOE_DTYPE_BF16>(a, tiles * nr, st);
  return gated ? tile_go<kForward, true, MOE_DTYPE_FP16>(a, tiles * nr, st)
               : tile_go<kForward, false, MOE_DTYPE_FP16>(a, tiles * nr, st);
}

}  // namespace moe
