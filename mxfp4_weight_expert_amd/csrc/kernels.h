// Host-side launchers of the layer's kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace moe {

struct RouteArgs {
  const float* logits;       // [T, Eg] or null (ids mode)
  const int32_t* topk_ids;   // [T, topk] (ids mode)
  const float* topk_w;       // [T, topk] (ids mode)
  const uint16_t* shared_logits;  // [T, S] bf16
  int T, Eg, topk, S, E, expert_offset;
  float shared_scale;
  int32_t* route_ids;    // [T, topk]
  int32_t* slot_expert;  // [T, K']
  float* slot_w;         // [T, K']
};
hipError_t launch_route(const RouteArgs& a, hipStream_t st);

struct SortArgs {
  const int32_t* slot_expert;
  int nslots, Ep, B, n_ranges, force_path;
  int32_t* range_counts;  // [n_ranges, Ep]
  int32_t* counts;        // [Ep]
  int32_t* offsets;       // [Ep + 1]
  int32_t* sorted_slot;   // [nslots]
  int32_t* expanded_idx;  // [nslots]
  int32_t* vinfo;         // [kmax_v, 4]
  int32_t* units16;       // [max_units16, 4]: 16-row units
  int32_t* dense_tiles;   // [max_dense_tiles, 4]
  int32_t* counters;      // [kCounterWords]
};
// Histogram -> scan (+ chunk table) -> scatter -> GEMM2 gate.
hipError_t launch_sort_and_gate(const SortArgs& a, hipStream_t st);

struct GemmArgs {
  const uint16_t* x;         // [T, H] bf16
  const uint8_t* w13;        // [Ep, 2I, H/2]
  const uint8_t* s13;        // [Ep, 2I, H/32]
  const uint8_t* w2;         // [Ep, H, I/2]
  const uint8_t* s2;         // [Ep, H, I/32]
  const int32_t* vinfo;
  const int32_t* units16;
  const int32_t* dense_tiles;
  const int32_t* counters;
  const int32_t* counts;  // [Ep] rows per local expert
  const int32_t* sorted_slot;
  int T, H, I, Kp, B, kmax_v, max_dense_tiles, max_units16, rows_pad;
  int Ep;  // local experts including the shared ones
  int dense_grid_tiles;  // tiles the dense GEMM2 grid is sized for (the kernels loop past it)
  ActArgs act_fn;  // GEMM1 epilogue activation
  uint16_t* act;  // [rows_pad, I] bf16 (W4A16), E4M3 codes (W4A8) or E2M1 code pairs [rows_pad, I/2] (W4A4)
  uint16_t* y;    // [rows_pad, H] bf16
  // MX activations (a8 != 0: W4A8 MXFP8, or W4A4 MXFP4 when a4 is also set):
  // quantised x and act scales
  int a8;
  int a4;
  const uint8_t* xq;    // [T, H] E4M3 (W4A8) or [T, H/2] E2M1 pairs (W4A4)
  const uint8_t* xs;    // [T, H/32] E8M0
  uint8_t* act_scales;  // [rows_pad, I/32] E8M0
};
hipError_t launch_gemm1(const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm2(const GemmArgs& a, hipStream_t st);  // split + dense, gated on device
// LDS-tiled kernels for many rows per expert (gemm_tiled.hip): GEMM1 over the
// chunk table (B >= 64); GEMM2 of both paths in one gated launch (bf16 act
// with I <= kResidentMaxI, or MX act); the generic dense GEMM2 over the dense
// tiles for bf16 act with larger I.
hipError_t launch_gemm1_tiled(const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm2_gated(const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm2_gated_mx(const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm2_dense_tiled(const GemmArgs& a, hipStream_t st);

// x -> MXFP8 (W4A8 path: xq [T, H] E4M3 codes) or MXFP4 (a4, W4A4 path:
// xq [T, H/2] E2M1 code pairs), xs [T, H/32] E8M0 scales.
hipError_t launch_quant_x(const uint16_t* x, int T, int H, uint8_t* xq, uint8_t* xs, bool a4,
                          hipStream_t st);
// MX-activation GEMM1 kernels, W4A8 or W4A4 by a4 (launch_gemm1 dispatches to
// them when a8 is set).
hipError_t launch_gemm1_a8(const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm1_tiled_a8(const GemmArgs& a, hipStream_t st);

struct FinalizeArgs {
  const uint16_t* y;
  const int32_t* expanded_idx;
  const float* slot_w;
  int T, Kp, H;
  uint16_t* out;
};
hipError_t launch_finalize(const FinalizeArgs& a, hipStream_t st);

// Maps of the dispatch operator from global ids, for many slots (sort.hip).
struct SortMapsArgs {
  const int32_t* ids;  // [nslots] global ids
  int nslots, E, expert_offset;
  int32_t* range_counts;  // [ranges of map_range_slots(nslots) slots, E]
  int32_t* counts;        // [E]
  int32_t* offsets;       // [E + 1]
  int32_t* row_slot;      // [nslots]
  int32_t* slot_row;      // [nslots]
};
int map_range_slots(int64_t nslots);
hipError_t launch_sort_maps(const SortMapsArgs& a, hipStream_t st);

// Slots up to which dispatch is one launch (dispatch.hip). H = 0: the maps alone, x
// and rows are not touched.
constexpr int kFusedSlots = 4096;
struct DispatchArgs {
  const uint8_t* x;    // [T, H]
  const int32_t* ids;  // [T, topk]
  int T, E, topk, H, expert_offset;
  int elem;  // bytes of an element
  uint8_t* rows;
  int32_t* offsets;
  int32_t* row_slot;
  int32_t* slot_row;
  int32_t* range_counts;  // workspace of the many-slot path, as in SortMapsArgs
  int32_t* counts;
};
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t st);

struct CombineArgs {
  const uint8_t* dout;  // [T, H] (backward)
  const uint8_t* rows;  // [T * topk, H]
  const int32_t* slot_row;
  const float* topk_w;  // null: 1 (forward only)
  int T, topk, H, dtype;
  uint8_t* out;    // [T, H], backward: drows [T * topk, H]
  float* dtopk_w;  // backward
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t st);
hipError_t launch_combine_backward(const CombineArgs& a, hipStream_t st);

// Tasks (row tiles x weight sets) a 4-bit product may have.
constexpr int64_t kW4MaxItems = int64_t{1} << 30;
struct W4Args {
  const void* x;           // [M, K], rows ldx apart
  const int32_t* offsets;  // [E + 1] (grouped) or null
  const uint8_t* w;        // [E, Np, K / 2] packed
  const void* scales;      // [E, N, K / group]
  const uint8_t* zeros;    // [E, N, K / group] or null
  const void* bias;        // [E, N] or null
  void* out;               // [M, N], rows ldo apart
  int M, N, K, E, format, group, dtype, out_dtype;
  int64_t ldx, ldo;
  int kw;  // waves of a block that split K (set by the launcher)
};
hipError_t launch_w4(const W4Args& a, hipStream_t st);
hipError_t launch_w4_bf16(const W4Args& a, hipStream_t st);  // launch_w4's

// Tiles a 16-bit product may have.
constexpr int64_t kMaxTileItems = int64_t{1} << 30;
// out[c, r] = sum over i of P[r, i] Q[c, i] (tile_product.h).
struct TileArgs {
  const void* p;
  const void* q;
  void* out;               // rows ldo apart
  void* gu;                // gated forward: [M, 2 R] pre-activations, or null
  const int32_t* offsets;  // [E + 1] or null
  int M, E;                // rows of all experts; matrices
  int R;                   // r: elements of a row of out (gated: features)
  int C;                   // gradient of the matrices: rows of one
  int I;                   // i to sum over, where it is not the expert's rows
  int64_t pstride;         // elements from one matrix of P to the next
  int64_t ldp, ldq, ldo;   // elements from row to row
  int dtype, out_dtype;
  int terms;               // gradients: arrays whose sum Q is, 1 or 2
  int64_t qterm;           // elements from one of them to the next
  ActArgs act;             // gated
};
hipError_t launch_tile_forward(const TileArgs& a, bool gated, hipStream_t st);
hipError_t launch_few_rows(const TileArgs& a, bool gated, hipStream_t st);  // forward (few_rows.hip)
hipError_t launch_tile_row_grad(const TileArgs& a, hipStream_t st);
hipError_t launch_tile_mat_grad(const TileArgs& a, hipStream_t st);
hipError_t launch_tile_gradients(const TileArgs& mat, const TileArgs& row, hipStream_t st);

// Gradient of the activation: dgu [M, 2 I] from dh [M, I] and the pre-activations.
struct ActGradArgs {
  const void* dh;
  const void* gu;
  void* dgu;
  void* rest;              // [M, 2 I], what dgu's rounding left, or null
  const int32_t* offsets;  // or null
  int M, I, E, dtype;
  ActArgs act;
};
hipError_t launch_act_grad(const ActGradArgs& a, hipStream_t st);

// Low-rank adapters (adapter.hip): out = base + scale[a] (x A_a^T) B_a^T for the rows
// that the maps sort by adapter.
struct AdapterArgs {
  const void* x;             // [M, K], rows ldx apart
  const int32_t* offsets;    // [A + 1]
  const int32_t* row_slot;   // sorted row -> row
  const int32_t* slot_row;   // row -> sorted row, or -1
  const void* a;             // [A, R, K]
  const void* b;             // [A, N, R]
  const float* scale;        // [A] or null: 1
  const void* base;          // [M, N], rows ldb apart, or null
  void* out;                 // [M, N], rows ldo apart; may be base
  float* part;               // workspace: [splits, M, R], x A^T by part of K
  int M, N, K, R, A, splits, dtype, out_dtype;
  int64_t ldx, ldb, ldo;
};
// Parts of K that the first product is split into.
int adapter_splits(int64_t M, int64_t A, int64_t K, int64_t R);
hipError_t launch_adapter(const AdapterArgs& a, hipStream_t st);

hipError_t launch_prepack(const uint8_t* src, uint8_t* dst, int64_t rows, int64_t row_bytes,
                          hipStream_t st);

}  // namespace moe
