// Argument checks that the operators' entry points share (host).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "moe_ops.h"

namespace moe {

constexpr int64_t kMaxSlots = int64_t{1} << 23;

inline bool known_dtype(int d) {
  return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_FP16 || d == MOE_DTYPE_FP32;
}
inline int64_t size_of(int dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 2; }
inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) &&
         y < x + static_cast<uintptr_t>(na);
}

// Rows of two matrices, `rows` of each, na and nb bytes long and sa and sb apart. With
// the same stride the rows of the one may lie between those of the other; with
// different ones the ranges decide.
inline bool rows_overlap(const void* a, int64_t na, int64_t sa, const void* b, int64_t nb, int64_t sb,
                  int64_t rows) {
  if (!overlap(a, (rows - 1) * sa + na, b, (rows - 1) * sb + nb)) return false;
  if (sa != sb) return true;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const int64_t at = (d % sa + sa) % sa;  // from a row of a to the next row of b
  return at < na || at + nb > sa;
}

// Workspace of the maps of `slots` slots: range counts at 0, then the experts' counts.
struct MapsWs {
  uint64_t counts, bytes;
};
inline MapsWs maps_ws(uint64_t slots, uint64_t E) {
  if (slots <= static_cast<uint64_t>(kFusedSlots)) return {0, 256};
  const uint64_t len = map_range_slots(static_cast<int64_t>(slots));
  const uint64_t ranges = (slots + len - 1) / len;
  const uint64_t counts = (ranges * E * 4 + 255) / 256 * 256;
  return {counts, counts + (E * 4 + 255) / 256 * 256};
}

inline int status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe
