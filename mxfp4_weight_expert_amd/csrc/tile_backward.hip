// Gradients of the 16-bit products in tiles.
#include "tile_launch.h"

namespace moe {

namespace {

// One launch for both where the matrices' tiles are the longer ones or make two rounds of
// the card: the rows' tiles then fill up what these leave (8192 rows of 7168, I 2048: 861
// us, 906 in two launches; half of 896 experts, 146 rows each, K 3584, I 384: 1030, 1110;
// 1538 rows, K 264, I 200: 16 and 21). Long tiles behind few short ones only wait for them
// (4 experts of 443 rows, K 1072, N 1720: 44 us, 33). Tiles of 128 and 256, whose sums go up
// i alike, may stand for each other (19 experts of 300 rows, K 5152, I 184, where the
// matrices alone would take 128: 100 us, 112), but not where only the rows' are small, which
// says few rows (56 of 14 rows, K 344, I 1608: 85 and 70). So a gradient asked for alone has
// the same bits.
template <int DT>
hipError_t gradients(const TileArgs& mat, const TileArgs& row, hipStream_t st) {
  const TileKind km = tile_kind<kMatGrad, false>(mat), kr = tile_kind<kRowGrad, false>(row);
  const TileKind kind = km == kTile128 ? kr : km;
  const bool fit = km == kr || (km > kTile64 && kr > kTile128);
  const int64_t items = kind == kTile64    ? tile_items<64, kMatGrad, false>(mat)
                        : kind == kTile128 ? tile_items<128, kMatGrad, false>(mat) / 2
                                           : tile_items<256, kMatGrad, false>(mat);
  if (!fit || (tile_ratio(mat, row) < 0.75 && items < 2 * tile_blocks<256>())) {
    const hipError_t err = tile_run<kRowGrad, false, DT>(row, st);
    return err != hipSuccess ? err : tile_run<kMatGrad, false, DT>(mat, st);
  }
  switch (kind) {
    case kTile64: return tile_gradients_go<64, 32, DT>(mat, row, st);
    case kTile128: return tile_gradients_go<128, 32, DT>(mat, row, st);
    case kTile256: return tile_gradients_go<256, 32, DT>(mat, row, st);
    default: return tile_gradients_go<256, 64, DT>(mat, row, st);
  }
}

}  // namespace

hipError_t launch_tile_row_grad(const TileArgs& a, hipStream_t st) {
  return a.dtype == MOE_DTYPE_BF16 ? tile_run<kRowGrad, false, MOE_DTYPE_BF16>(a, st)
                                   : tile_run<kRowGrad, false, MOE_DTYPE_FP16>(a, st);
}

hipError_t launch_tile_mat_grad(const TileArgs& a, hipStream_t st) {
  return a.dtype == MOE_DTYPE_BF16 ? tile_run<kMatGrad, false, MOE_DTYPE_BF16>(a, st)
                                   : tile_run<kMatGrad, false, MOE_DTYPE_FP16>(a, st);
}

hipError_t launch_tile_gradients(const TileArgs& mat, const TileArgs& row, hipStream_t st) {
  return mat.dtype == MOE_DTYPE_BF16 ? gradients<MOE_DTYPE_BF16>(mat, row, st) : gradients<MOE_DTYPE_FP16>(mat, row, st);
}

}  // namespace moe
