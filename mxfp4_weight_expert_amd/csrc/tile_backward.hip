// Gradients of the 16-bit products in tiles.
#include "tile_launch.h"

namespace moe {

hipError_t launch_tile_row_grad(const TileArgs& a, hipStream_t st) {
  const int64_t nr = (a.R + kTile - 1) / kTile;
  const int64_t tiles = (a.M + kTile - 1) / kTile + (a.offsets != nullptr ? a.E : 0);
  return a.dtype == MOE_DTYPE_BF16 ? tile_go<kRowGrad, false, MOE_DTYPE_BF16>(a, tiles * nr, st)
                                   : tile_go<kRowGrad, false, MOE_DTYPE_FP16>(a, tiles * nr, st);
}

hipError_t launch_tile_mat_grad(const TileArgs& a, hipStream_t st) {
  const int64_t nr = (a.R + kTile - 1) / kTile, nc = (a.C + kTile - 1) / kTile;
  return a.dtype == MOE_DTYPE_BF16 ? tile_go<kMatGrad, false, MOE_DTYPE_BF16>(a, a.E * nc * nr, st)
                                   : tile_go<kMatGrad, false, MOE_DTYPE_FP16>(a, a.E * nc * nr, st);
}

}  // namespace moe
