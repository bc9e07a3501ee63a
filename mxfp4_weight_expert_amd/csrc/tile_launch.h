// Launch of the tiled 16-bit products.
#pragma once

#include "tile_product.h"

#include <algorithm>
#include <atomic>

namespace moe {

// CUs of the current GPU, asked once for each.
inline int gpu_cus() {
  constexpr int kGpus = 16;
  static std::atomic<int> kept[kGpus];
  int gpu = 0, cus = 0;
  if (hipGetDevice(&gpu) == hipSuccess) {
    if (gpu < kGpus && (cus = kept[gpu].load(std::memory_order_relaxed)) > 0) return cus;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, gpu) == hipSuccess && cus > 0) {
      if (gpu < kGpus) kept[gpu].store(cus, std::memory_order_relaxed);
      return cus;
    }
  }
  (void)hipGetLastError();  // a query's error is not the launch's
  return 256;
}

// One block a CU, a multiple of the eight XCDs, each with tiles in turn; `items`
// bounds the tiles.
template <int MODE, bool GATED, int DT>
hipError_t tile_go(const TileArgs& a, int64_t items, hipStream_t st) {
  const int64_t most = std::max(gpu_cus() / 8 * 8, 8);
  const int64_t blocks = std::min((items + 7) / 8 * 8, most);
  const int lds = kSlots * kStage + (MODE != kMatGrad && a.offsets != nullptr ? (a.E + 1) * 4 : 0);
  hipLaunchKernelGGL((tile_product_kernel<MODE, GATED, DT>), dim3(static_cast<unsigned>(blocks)),
                     dim3(kTileThreads), lds, st, a);
  return hipGetLastError();
}

}  // namespace moe
