// Gradients of the 16-bit products in tiles.
#include "tile_launch.h"

namespace moe {

hipError_t launch_tile_row_grad(const TileArgs& a, hipStream_t st) {
  return a.dtype == MOE_DTYPE_BF16 ? tile_size<kRowGrad, false, MOE_DTYPE_BF16>(a, st)
                                   : tile_size<kRowGrad, false, MOE_DTYPE_FP16>(a, st);
}

hipError_t launch_tile_mat_grad(const TileArgs& a, hipStream_t st) {
  return a.dtype == MOE_DTYPE_BF16 ? tile_size<kMatGrad, false, MOE_DTYPE_BF16>(a, st)
                                   : tile_size<kMatGrad, false, MOE_DTYPE_FP16>(a, st);
}

}  // namespace moe
