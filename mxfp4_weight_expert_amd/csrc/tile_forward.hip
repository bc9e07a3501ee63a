// Forward products of 16-bit matrices in tiles, plain and gated.
#include "tile_launch.h"

namespace moe {

hipError_t launch_tile_forward(const TileArgs& a, bool gated, hipStream_t st) {
  // Few rows of a matrix: tiles of 16 rows that read it straight into registers (64
  // experts, K 7168 x 2 N 4096 gated: 2 rows each 563 us, 638 with tiles of 128; 8 rows
  // 660 and 680, 16 rows 969 and 697; one matrix, 1 row 13 and 23 with tiles of 64, 16
  // rows 17 and 26, 32 rows 29 and 30).
  if (a.offsets == nullptr ? a.M <= 16 : a.M <= int64_t{8} * a.E) return launch_few_rows(a, gated, st);
  if (a.dtype == MOE_DTYPE_BF16)
    return gated ? tile_run<kForward, true, MOE_DTYPE_BF16>(a, st) : tile_run<kForward, false, MOE_DTYPE_BF16>(a, st);
  return gated ? tile_run<kForward, true, MOE_DTYPE_FP16>(a, st) : tile_run<kForward, false, MOE_DTYPE_FP16>(a, st);
}

}  // namespace moe
