// Launch of the tiled 16-bit products.
#pragma once

#include "tile_product.h"

#include <algorithm>
#include <atomic>
#include <cmath>

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

// Resident blocks (128: two a CU), a multiple of the eight XCDs, each with tiles in
// turn; `items` bounds the tiles.
template <int T>
int64_t tile_blocks() {
  return std::max(gpu_cus() / 8 * 8, 8) * (T == 128 ? 2 : 1);
}
template <int T, int MODE, bool GATED>
int64_t tile_items(const TileArgs& a) {
  const int64_t wide = GATED ? T / 2 : T, nr = (a.R + wide - 1) / wide;
  return nr * (MODE == kMatGrad ? static_cast<int64_t>(a.E) * ((a.C + T - 1) / T)
                                : (a.M + T - 1) / T + (a.offsets != nullptr ? std::min(a.E, a.M) : 0));
}
template <int T, int STEP>
int tile_room(const TileArgs& a) {  // LDS: stages, and the experts' first tiles
  return tile_lds(T, STEP) + (a.offsets != nullptr ? (a.E + 1) * 4 : 0);
}
template <int T, int STEP, int MODE, bool GATED, int DT>
hipError_t tile_go(const TileArgs& a, hipStream_t st) {
  const int64_t blocks = std::min((tile_items<T, MODE, GATED>(a) + 7) / 8 * 8, tile_blocks<T>());
  const int lds = tile_room<T, STEP>(a);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(tile_threads(T)), lds, st, a);
  };
  if constexpr (MODE == kForward) go(tile_product_kernel<T, STEP, MODE, GATED, DT, 1>);
  else if (a.terms == 1) go(tile_product_kernel<T, STEP, MODE, GATED, DT, 1>);
  else go(tile_product_kernel<T, STEP, MODE, GATED, DT, 2>);
  return hipGetLastError();
}
// How many tiles of the rows' gradient take as long as one of the matrices'.
inline double tile_ratio(const TileArgs& mat, const TileArgs& row) {
  return static_cast<double>(mat.M) / mat.E / row.I;
}
template <int T, int STEP, int DT>
hipError_t tile_gradients_go(const TileArgs& mat, const TileArgs& row, hipStream_t st) {
  const int64_t first = tile_items<T, kMatGrad, false>(mat), all = first + tile_items<T, kRowGrad, false>(row);
  const int64_t blocks = std::min((all + 7) / 8 * 8, tile_blocks<T>());
  const TileShare share = {static_cast<int>(first), static_cast<int>(std::clamp(tile_ratio(mat, row) + 0.5, 0.0, 1024.0))};
  const int lds = tile_room<T, STEP>(mat);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(tile_threads(T)), lds, st, mat, row, share);
  };
  if (mat.terms == 1) go(tile_gradients_kernel<T, STEP, DT, 1>);
  else go(tile_gradients_kernel<T, STEP, DT, 2>);
  return hipGetLastError();
}

// Estimated time (us) with tiles of side T: rounds of the resident blocks, each some time
// for its start and end and some for each 32 of i. Large tiles do more for a byte that
// they load, small ones fill the card: M = 256, K 7168 x 2 N 4096 gated 33 us with tiles of
// 64, 67 with 128, 160 with 256; 8192 rows 1240, 916 and, of 64, 2400 for the backward pass.
// A CU with one block of 128 runs it faster than two. The rows of an expert are taken as
// M / E; where many live elsewhere they are fewer. No tile splits its i over blocks, so many
// rows of few small matrices leave CUs without one in the matrices' gradient (8192 rows of
// one of 512 x 512, 64 tiles: 36 us, its rows' gradient 11).
template <int T, int MODE, bool GATED>
double tile_time(const TileArgs& a) {
  const double rows = std::max(1.0, static_cast<double>(a.M) / a.E);
  const int64_t wide = GATED ? T / 2 : T, nr = (a.R + wide - 1) / wide;
  const double across = MODE == kMatGrad ? a.C : rows;
  const double tiles = std::ceil(across / T) * nr * (MODE == kMatGrad ? a.E : std::min<double>(a.E, a.M));
  const double steps = std::ceil((MODE == kMatGrad ? rows : a.I) / 32) * a.terms, fill = std::min(1.0, across / T);
  const double rounds = std::ceil(tiles / static_cast<double>(tile_blocks<T>()));
  if (T == 64) return rounds * (2.2 + steps * (tiles <= 128 ? 0.12 : 0.2));
  if (T == 256) return rounds * (7 + steps * (0.45 + 0.4 * fill));
  return tiles <= gpu_cus() ? 2.5 + steps * 0.27 : rounds * (5 + steps * (0.5 + 0.2 * fill));
}

// Whether tiles of 256 take stages of 64 (tile_stage): where many rows make the matrix
// cores and not memory the bound. 64 of 256 experts' 8192 x 8 rows forward 1338 us so, 1437
// with stages of 32; half of 896 experts, 146 rows by this count, rows' gradient 27 us more.
template <int MODE>
bool long_stages(const TileArgs& a) {
  return a.M >= (MODE == kMatGrad ? 2048 : 192) * static_cast<int64_t>(a.E);
}

// The kernel of a shape: tiles of 64, 128 or 256, these with stages of 32 or 64.
enum TileKind { kTile64, kTile128, kTile256, kTile256Long };
template <int MODE, bool GATED>
TileKind tile_kind(const TileArgs& a) {
  const double t64 = tile_time<64, MODE, GATED>(a), t128 = tile_time<128, MODE, GATED>(a);
  const double t256 = tile_time<256, MODE, GATED>(a);
  if (t64 <= std::min(t128, t256)) return kTile64;
  if (t128 <= t256) return kTile128;
  return long_stages<MODE>(a) ? kTile256Long : kTile256;
}

template <int MODE, bool GATED, int DT>
hipError_t tile_run(const TileArgs& a, hipStream_t st) {
  switch (tile_kind<MODE, GATED>(a)) {
    case kTile64: return tile_go<64, 32, MODE, GATED, DT>(a, st);
    case kTile128: return tile_go<128, 32, MODE, GATED, DT>(a, st);
    case kTile256: return tile_go<256, 32, MODE, GATED, DT>(a, st);
    default: return tile_go<256, 64, MODE, GATED, DT>(a, st);
  }
}

}  // namespace moe
