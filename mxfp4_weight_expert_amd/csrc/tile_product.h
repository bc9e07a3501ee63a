// Products of 16-bit matrices in square tiles on the matrix cores, one
// kernel for the forward pass and both gradients of rows times their expert's
// matrix (offsets given) or one matrix for all rows (offsets null):
//
//   kForward  out[m, n] = sum over k of x[m, k] w[e, n, k]
//   kRowGrad  dx[m, k]  = sum over n of dout[m, n] w[e, n, k]
//   kMatGrad  dw[e, n, k] = sum over the rows m of e of dout[m, n] x[m, k]
//
// Each is out[c, r] = sum over i of P[r, i] Q[c, i], r the side whose elements
// follow each other in out. P is the A operand of the 32x32x16 MFMA and Q its B
// operand, so a lane has four neighbours of a row of out at a time:
//
//              r  c  i    P             Q
//   kForward   n  m  k    w, i inner    x, i inner
//   kRowGrad   k  m  n    w, r inner    dout, i inner
//   kMatGrad   k  n  m    x, r inner    dout, c inner
//
// In the gradients Q may be the sum of two arrays (TERMS): the i are walked once for each,
// over the same P (8192 rows, K 7168, 2 N 4096, both gradients: 1656 us, 883 with one; half
// of 896 experts, 146 rows each, K 3584, 2 N 768: 1558, 1038).
//
// Operands whose inner index is i go to LDS as rows of 64 bytes (32 i) and are
// read 16 bytes a lane. The others go as 32 rows of the tile's width, and the transposing
// LDS read (ds_read_b64_tr_b16: within 16 lanes, lane 4 a + b gives four columns
// 4 b of row a, and lane j receives column j of the four rows) makes the operand.
#pragma once

#include "rows.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace moe {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

enum { kForward, kRowGrad, kMatGrad };

constexpr int PB = 2;          // 32-blocks of r of a wave
// Tiles of T x T. T = 256, 128: T / 32 waves, each with 64 r and every second 32 c, share
// the stages. T = 64: four waves take every fourth stage each, with stages of their own
// and no barrier between them, and join their sums at the end.
constexpr int tile_split(int T) { return T == 64 ? 4 : 1; }
constexpr int tile_threads(int T) { return T == 64 ? 256 : T * 2; }
// Stages of STEP i: both operands' bytes of one, and how many are in LDS, one read and the
// others in flight. Of 32 there are four, of 64 (tiles of 256 alone) two, with half the
// barriers and whole 128-byte lines: 8192 x 8192 x 8192 878 us (forward), 843 and 893
// (gradients) against 921, 903 and 915; but where memory bounds the tile the fewer bytes
// in flight cost more (64 experts of 32 rows, K 7168 x 2 N 4096 765 us, 725).
constexpr int tile_stage(int T, int STEP) { return 2 * T * STEP * 2; }
constexpr int tile_slots(int STEP) { return STEP == 64 ? 2 : 4; }
constexpr int tile_lds(int T, int STEP) { return tile_slots(STEP) * tile_stage(T, STEP) * tile_split(T); }

template <int DT>
__device__ __forceinline__ f32x16_t mfma32(uint4 a, uint4 b, f32x16_t c) {
  if constexpr (DT == MOE_DTYPE_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                  c, 0, 0, 0);
}

// Sixteen bytes a lane from global memory to LDS at `lds` (wave-uniform) + 16 *
// lane, zeros for lanes at offset kNoRow. Written in assembly so that the compiler
// does not wait for every load in flight before each LDS read; it has no output
// registers, and the caller waits (vmcnt) before the barrier that publishes it.
__device__ __forceinline__ void load_to_lds(uint64_t base, uint32_t off, uint32_t lds) {
  // the address as scalar instructions' results: one that a vector instruction wrote would
  // need wait states before the load
  uint32_t lo, hi;
  asm("s_mov_b32 %0, %1" : "=s"(lo) : "s"(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(base))));
  asm("s_and_b32 %0, %1, 0xffff" : "=s"(hi) : "s"(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(base >> 32))) : "scc");
  const i32x4_t rsrc = {static_cast<int>(lo), static_cast<int>(hi), static_cast<int>(kNoRow), 0x00020000};
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(rsrc)
               : "memory");  // compiled code sets m0 right before each of its own uses
}

// Rows of STEP i (64 or 128 bytes): 16-byte chunk c of row r lies at chunk c ^
// chunk_swz(r). LDS serves a 16-byte read sixteen lanes at a time, in groups of four
// neighbours: 0, 12, 20 and 24 on, then 4, 8, 16 and 28 on; the chunks of these rows fall
// on different banks (no conflicts; counted).
template <int STEP>
__device__ __forceinline__ uint32_t chunk_swz(uint32_t r) { return STEP == 32 ? r >> 2 & 3 : r >> 1 & 7; }
// Rows of 512, 256 or 128 bytes: 64-byte piece g of row r lies at piece g ^ piece_swz(r): the
// four rows of a transposing read, and those of its other half eight further on, fall on
// different banks.
template <int T>
__device__ __forceinline__ uint32_t piece_swz(uint32_t r) {
  return T == 256 ? (r & 3) | (r >> 3 & 1) << 2 : T == 128 ? (r & 3) ^ (r >> 3 & 1) : r >> 1 & 1;
}

// Gated: a wave's first 32-block of r are gate rows, the second the up rows of the same
// features, which so meet in a lane.
__device__ __forceinline__ uint32_t gated_feature(uint32_t rho) { return (rho >> 6) * 32 + (rho & 31); }
__device__ __forceinline__ bool gated_up(uint32_t rho) { return (rho >> 5 & 1) != 0; }

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == MOE_DTYPE_BF16) return pack_bf16x2(lo, hi);
  else return Row<MOE_DTYPE_FP16>::pack2(lo, hi);
}
// One tile of out.
struct TileItem {
  int e;      // matrix
  int r0;     // first r (gated: feature)
  int c0;     // first c: row of Q (kMatGrad: column of dout)
  int cols;   // c that the tile has
  int first;  // kMatGrad: first of the expert's rows
  int len;    // i to sum over
};

// How a second list of tiles follows a first in one launch: blocks with one tile fewer of
// the first take `more` of the second before the others take any.
struct TileShare {
  int items;  // of the first list; 0: none
  int more;
};

template <int T, int kStep, int MODE, bool GATED, int DT, int TERMS>
__device__ __forceinline__ void tile_product(const TileArgs& a, const TileShare first_list) {
  static_assert(!GATED || MODE == kForward, "the activation follows the forward product");
  constexpr bool kPInner = MODE == kForward;   // i is P's inner index
  constexpr bool kQInner = MODE != kMatGrad;
  constexpr int kWide = GATED ? T / 2 : T;      // r of a tile
  constexpr int KW = tile_split(T), WC = KW > 1 ? 1 : 2;  // waves along i, along c
  constexpr int NQ = T / (32 * WC);               // 32-blocks of c of a wave: every WC-th
  constexpr int kSlots = tile_slots(kStep), kHalves = kStep / 16;  // 16 i an MFMA
  constexpr int kThreads = tile_threads(T), kWaves = kThreads / 64, kStage = tile_stage(T, kStep), kSide = kStage / 2;
  constexpr int kLoads = kSide / 1024 / (KW > 1 ? 1 : kWaves);  // a wave's loads of 1 KB of an operand's stage
  constexpr int kRow = 2 * T;                     // bytes of a row whose inner index is not i
  extern __shared__ __attribute__((aligned(1024))) uint8_t s_dyn[];
  __shared__ int32_t s_wave[kWaves];
  int32_t* const s_first = reinterpret_cast<int32_t*>(s_dyn + tile_lds(T, kStep));  // grouped: tiles before each expert
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)s_dyn));
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_index();
  constexpr int kAlong = T / (32 * PB);  // waves along r
  const int wr = wv % kAlong, wc = KW > 1 ? 0 : wv / kAlong;
  const int part = KW > 1 ? wv : 0, lw = KW > 1 ? 0 : wv;      // of the stages; of a stage's loads
  const uint32_t of_wave = KW > 1 ? wv * kSlots * kStage : 0;
  uint8_t* const ring = s_dyn + of_wave;
  const uint32_t ring0 = lds0 + of_wave;
  const int nr = (a.R + kWide - 1) / kWide;

  // The tiles of the experts' rows.
  int tiles = (a.M + T - 1) / T;
  if (MODE != kMatGrad && a.offsets != nullptr) {
    constexpr int kPer = kMaxExperts / kThreads;
    int n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      n[i] = 0;
      if (e < a.E) {
        const int lo = min(max(a.offsets[e], 0), a.M), hi = min(a.offsets[e + 1], a.M);
        n[i] = hi > lo ? (hi - lo + T - 1) / T : 0;
      }
      sum += n[i];
    }
    const int incl = wave_incl_scan(sum);
    if (lane == kWave - 1) s_wave[wv] = incl;
    __syncthreads();
    int at = incl - sum;
    tiles = 0;
    for (int i = 0; i < kWaves; ++i) {
      if (i < wv) at += s_wave[i];
      tiles += s_wave[i];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      if (e <= a.E) s_first[e] = at;
      at += n[i];
    }
    if (a.E == kMaxExperts && tid == kThreads - 1) s_first[kMaxExperts] = at;
    __syncthreads();
    tiles = __builtin_amdgcn_readfirstlane(tiles);
  }
  const int nc = (a.C + T - 1) / T;  // kMatGrad: tiles along dout's columns
  const int items = static_cast<int>(min(
      MODE == kMatGrad ? static_cast<int64_t>(a.E) * nc * nr : static_cast<int64_t>(tiles) * nr, kMaxTileItems));

  // The item of a block's round k. In a round the blocks of an XCD (block ids go round
  // over the eight) take neighbours, which share operands and meet in its L2. One matrix:
  // each XCD has a range of its own, so that it meets them in the next round too. Experts,
  // whose tiles cost differently: the XCDs take turns (64 experts of 256 rows 1382 us,
  // 1512 with ranges; one matrix the other way 950 and 912).
  const int walkers = static_cast<int>(gridDim.x) >> 3, xcd = blockIdx.x & 7;
  const bool ranges = a.offsets == nullptr;
  const int width = ranges ? walkers : static_cast<int>(gridDim.x);  // blocks that share a run of items
  const int place = ranges ? blockIdx.x >> 3 : xcd * walkers + (blockIdx.x >> 3);
  const int per = ranges ? (items + 7) >> 3 : items, base = ranges ? xcd * per : 0;
  const int busy = first_list.items == 0 ? 0 : (ranges ? (first_list.items + 7) >> 3 : first_list.items) % width;
  const int idle = busy > 0 ? width - busy : 0, more = idle > 0 ? min(first_list.more, per / idle) : 0;
  auto item_of = [&](int k) {
    int at = k * width + place;
    if (more > 0) {
      if (place < busy) at = idle * more + k * width + idle + place;
      else at = k < more ? k * idle + place - busy : idle * more + (k - more) * width + place - busy;
    }
    return at < per ? base + at : items;
  };

  auto decode = [&](int item) {
    TileItem t;
    if constexpr (MODE == kMatGrad) {
      const int re = item / nr, e = re / nc;
      t.e = e;
      t.r0 = (item - re * nr) * kWide;
      t.c0 = (re - e * nc) * T;
      t.cols = min(T, a.C - t.c0);
      int lo = 0, hi = a.M;
      if (a.offsets != nullptr) {
        lo = min(max(a.offsets[e], 0), a.M);
        hi = min(a.offsets[e + 1], a.M);
      }
      t.first = __builtin_amdgcn_readfirstlane(lo);
      t.len = __builtin_amdgcn_readfirstlane(max(hi - lo, 0));
    } else {
      // four row tiles take one span of r after the other
      const int g = item / (4 * nr), rem = item - g * 4 * nr, size = min(4, tiles - 4 * g);
      const int r = rem / size, tile = 4 * g + rem - r * size;
      int lo = 0, hi = a.M, e = 0, local = tile;
      if (a.offsets != nullptr) {
        int below = 0, above = a.E - 1;  // the last expert whose first tile is at or before this one
        while (below < above) {
          const int mid = (below + above + 1) >> 1;
          if (s_first[mid] <= tile) below = mid;
          else above = mid - 1;
        }
        e = __builtin_amdgcn_readfirstlane(below);
        local = tile - __builtin_amdgcn_readfirstlane(s_first[e]);
        lo = __builtin_amdgcn_readfirstlane(min(max(a.offsets[e], 0), a.M));
        hi = __builtin_amdgcn_readfirstlane(min(a.offsets[e + 1], a.M));
      }
      t.e = e;
      t.r0 = r * kWide;
      // the expert's tiles of one size, a multiple of 32: full tiles with a short last one
      // cost more, and unequal shares (64 experts of 256 rows on average 1395 us, 1497)
      const int n = (hi - lo + T - 1) / T, width = ((hi - lo + n - 1) / n + 31) & ~31;
      t.c0 = lo + local * width;
      t.cols = min(width, hi - t.c0);
      t.first = 0;
      t.len = a.I;
    }
    return t;
  };

  // ---- loads
  int l_round = 0, l_left = 0;     // the item that loads come from: its round, its i left
  int l_term = 0;                  // and its term
  uint64_t pbase = 0, qbase = 0;   // where the next stage begins
  uint32_t poff[kLoads], qoff[kLoads];
  uint32_t pi[kLoads], qi[kLoads];           // the lane's i in a stage
  auto start = [&]() {
    const TileItem t = decode(item_of(l_round));
    l_left = t.len - part * kStep;
    pbase = reinterpret_cast<uint64_t>(a.p);
    qbase = reinterpret_cast<uint64_t>(a.q);
    if constexpr (MODE == kMatGrad)
      pbase += (static_cast<uint64_t>(t.first) * a.ldp + t.r0) * 2;
    else if constexpr (kPInner)
      pbase += (static_cast<uint64_t>(t.e) * a.pstride + static_cast<uint64_t>(t.r0) * a.ldp) * 2;
    else
      pbase += (static_cast<uint64_t>(t.e) * a.pstride + t.r0) * 2;
    pbase += static_cast<uint64_t>(part) * (kPInner ? kStep * 2 : a.ldp * (kStep * 2));
    qbase += static_cast<uint64_t>(part) * (kQInner ? kStep * 2 : a.ldq * (kStep * 2));
    qbase += (MODE == kMatGrad ? static_cast<uint64_t>(t.first) * a.ldq + t.c0
                               : static_cast<uint64_t>(t.c0) * a.ldq) * 2;
    if constexpr (TERMS > 1) qbase += static_cast<uint64_t>(l_term) * a.qterm * 2;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      // a load of rows whose inner index is not i: two rows of 512 bytes, four of 256, eight of 128
      const uint32_t row = (lw * kLoads + j) * (1024 / kRow) + lane / (kRow / 16);
      const uint32_t across = ((lane / 4 % (kRow / 64)) ^ piece_swz<T>(row)) * 4 + (lane & 3);  // 16-byte chunk
      if constexpr (kPInner) {
        const uint32_t rho = (lw * kLoads + j) * (512 / kStep) + lane / (kStep / 8);
        const uint32_t chunk = (lane % (kStep / 8)) ^ chunk_swz<kStep>(rho);
        const uint32_t r = GATED ? gated_feature(rho) : rho;
        const bool in = t.r0 + r < static_cast<uint32_t>(a.R);
        poff[j] = in ? (r + (GATED && gated_up(rho) ? a.R : 0)) * static_cast<uint32_t>(a.ldp) * 2 + chunk * 16 : kNoRow;
        pi[j] = chunk * 8;
      } else {
        const bool in = t.r0 + across * 8 < static_cast<uint32_t>(a.R);
        poff[j] = in ? row * static_cast<uint32_t>(a.ldp) * 2 + across * 16 : kNoRow;
        pi[j] = row;
      }
      if constexpr (kQInner) {
        const uint32_t c = (lw * kLoads + j) * (512 / kStep) + lane / (kStep / 8);
        const uint32_t chunk = (lane % (kStep / 8)) ^ chunk_swz<kStep>(c);
        qoff[j] = c < static_cast<uint32_t>(t.cols) ? c * static_cast<uint32_t>(a.ldq) * 2 + chunk * 16 : kNoRow;
        qi[j] = chunk * 8;
      } else {
        qoff[j] = across * 8 < static_cast<uint32_t>(t.cols) ? row * static_cast<uint32_t>(a.ldq) * 2 + across * 16 : kNoRow;
        qi[j] = row;
      }
    }
  };
  // The next stage into slot `slot`; past the last item loads that touch no memory, so
  // that the waits count the same everywhere.
  auto issue = [&](int slot) {
    while (l_left <= 0 && item_of(l_round) < items) {
      if (TERMS == 1 || ++l_term == TERMS) {
        l_term = 0;
        ++l_round;
      }
      if (item_of(l_round) < items) start();
    }
    const uint32_t left = max(l_left, 0), at = ring0 + slot * kStage + lw * kLoads * 1024;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      load_to_lds(pbase, pi[j] < left ? poff[j] : kNoRow, at + j * 1024);
      load_to_lds(qbase, qi[j] < left ? qoff[j] : kNoRow, at + kSide + j * 1024);
    }
    pbase += kPInner ? KW * kStep * 2 : static_cast<uint64_t>(a.ldp) * (KW * kStep * 2);
    qbase += kQInner ? KW * kStep * 2 : static_cast<uint64_t>(a.ldq) * (KW * kStep * 2);
    l_left -= KW * kStep;
  };

  if (item_of(0) >= items) return;
  start();
#pragma unroll
  for (int s = 0; s < kSlots - 1; ++s) issue(s);

  // ---- operands from LDS
  const int l32 = lane & 31, half = lane >> 5;
  uint32_t pat[kPInner ? kHalves : PB], qat[kQInner ? kHalves : NQ];
  if constexpr (kPInner) {
#pragma unroll
    for (int s = 0; s < kHalves; ++s)
      pat[s] = (wr * PB * 32 + l32) * 2 * kStep + (((2 * s + half) ^ chunk_swz<kStep>(l32)) << 4);
  } else {
    const uint32_t row = half * 8 + (lane >> 2 & 3), gg = lane >> 4 & 1, q = lane & 3;
#pragma unroll
    for (int p = 0; p < PB; ++p) pat[p] = row * kRow + (((wr * PB + p) ^ piece_swz<T>(row)) << 6) + (4 * gg + q) * 8;
  }
  if constexpr (kQInner) {
#pragma unroll
    for (int s = 0; s < kHalves; ++s)
      qat[s] = kSide + (wc * 32 + l32) * 2 * kStep + (((2 * s + half) ^ chunk_swz<kStep>(l32)) << 4);
  } else {
    const uint32_t row = half * 8 + (lane >> 2 & 3), gg = lane >> 4 & 1, q = lane & 3;
#pragma unroll
    for (int n = 0; n < NQ; ++n) qat[n] = kSide + row * kRow + (((WC * n + wc) ^ piece_swz<T>(row)) << 6) + (4 * gg + q) * 8;
  }
  auto transposed = [&](const uint8_t* at) {  // eight i of 32 rows or columns
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * kRow));
    const uint2 u = __builtin_bit_cast(uint2, lo), v = __builtin_bit_cast(uint2, hi);
    return uint4{u.x, u.y, v.x, v.y};
  };
  auto read_p = [&](const uint8_t* stage, int s, int b) {
    if constexpr (kPInner) return ld16(stage + pat[s] + b * 32 * 2 * kStep);
    else return transposed(stage + pat[b] + s * 16 * kRow);
  };
  auto read_q = [&](const uint8_t* stage, int s, int n) {
    if constexpr (kQInner) return ld16(stage + qat[s] + n * WC * 32 * 2 * kStep);
    else return transposed(stage + qat[n] + s * 16 * kRow);
  };

  // Waits until a stage's loads are done: those of the stages after it, and
  // `stores` stores behind them, may be under way.
  auto wait_stage = [&](int stores) {
    constexpr int kAhead = (kSlots - 2) * 2 * kLoads;
    if (stores >= 32) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAhead + 32) : "memory");
    else if (stores >= 16) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAhead + 16) : "memory");
    else if (stores >= 8) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAhead + 8) : "memory");
    else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAhead) : "memory");
  };

  f32x16_t acc[PB][NQ];
  uint4 p0[PB], q0[NQ], p1[PB], q1[NQ];
  int slot = 0, stores = 0;
  for (int round = 0; item_of(round) < items; ++round) {
    const TileItem t = decode(item_of(round));
    const int stages = TERMS * max(0, (t.len - part * kStep + KW * kStep - 1) / (KW * kStep));  // this wave's
    // 32-blocks of c that hold anything, for this wave
    const int blocks = min(NQ, max(0, (t.cols - 32 * wc + 32 * WC - 1) / (32 * WC)));
#pragma unroll
    for (int b = 0; b < PB; ++b)
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[b][n][v] = 0.0f;

    // A stage's last 16 i are multiplied after the next stage's barrier, while
    // that stage's first operands are read.
    auto walk = [&](auto nqc) {
      constexpr int N = decltype(nqc)::value;
      // Products of 16 i from operands in registers, with the LDS reads of the next 16,
      // written before them, between the first.
      auto mul = [&](const uint4 (&p)[PB], const uint4 (&q)[NQ]) {
        constexpr int kMuls = PB * N, kReads = (kPInner ? PB : 2 * PB) + (kQInner ? N : 2 * N);
#pragma unroll
        for (int i = 0; i < kMuls; ++i)
          acc[i % PB][i / PB] = mfma32<DT>(p[i % PB], q[i / PB], acc[i % PB][i / PB]);
#pragma unroll
        for (int i = 0; i < kReads; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one LDS read
          if (i < kMuls) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
        }
        __builtin_amdgcn_sched_barrier(0);
      };
#pragma unroll
      for (int b = 0; b < PB; ++b) p1[b] = uint4{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < N; ++n) q1[n] = uint4{0, 0, 0, 0};
      for (int k = 0; k < stages; ++k) {
        // this stage has come, and no wave still reads the slot
        // that the next loads go to
        // (the stores of the last item's results, younger than its loads, go on)
        if (k >= kSlots - 1) stores = 0;
        wait_stage(stores);
        if constexpr (KW == 1) __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(slot == 0 ? kSlots - 1 : slot - 1);
        const uint8_t* const stage = ring + slot * kStage;
        if constexpr (N > 0) {
#pragma unroll
          for (int s = 0; s < kHalves; s += 2) {
#pragma unroll
            for (int b = 0; b < PB; ++b) p0[b] = read_p(stage, s, b);
#pragma unroll
            for (int n = 0; n < N; ++n) q0[n] = read_q(stage, s, n);
            mul(p1, q1);
#pragma unroll
            for (int b = 0; b < PB; ++b) p1[b] = read_p(stage, s + 1, b);
#pragma unroll
            for (int n = 0; n < N; ++n) q1[n] = read_q(stage, s + 1, n);
            mul(p0, q0);
          }
        }
        slot = slot == kSlots - 1 ? 0 : slot + 1;
      }
      mul(p1, q1);
    };
    switch (blocks) {
      case 4: walk(std::integral_constant<int, NQ>{}); break;
      case 3: walk(std::integral_constant<int, std::min(NQ, 3)>{}); break;
      case 2: walk(std::integral_constant<int, 2>{}); break;
      case 1: walk(std::integral_constant<int, 1>{}); break;
      default: walk(std::integral_constant<int, 0>{}); break;
    }

    // ---- results: register 4 b + i of lane (l, h) is c = l, r = 8 b + 4 h + i of a
    // block. They pass through LDS, in the slot of the stage read last, 32 rows of up to
    // 128 bytes at a time, so that the stores write whole rows of 128 bytes (their 16-byte
    // pieces, straight from the registers, lie in 64 places: 2102 us where these take 1626
    // for 64 experts' gradients of 2048 x 7168 in 32 bits).
    auto meet = [&]() {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    if constexpr (KW == 1) meet();  // no wave still reads that slot
    uint8_t* const mine = ring + (slot == 0 ? kSlots - 1 : slot - 1) * kStage + lw * 4096;
    const int64_t row0 = (MODE == kMatGrad ? static_cast<int64_t>(t.e) * a.C : 0) + t.c0;
    // put(b): eight or sixteen bytes of four neighbours in row l32 of the piece; 16-byte
    // chunks are swapped so that neither side meets bank conflicts
    int ln = lane;
    asm volatile("" : "+v"(ln));  // addresses made from it are not kept in registers throughout
    const int l32 = ln & 31, half = ln >> 5;
    auto place = [&](int row, int chunk) { return mine + row * 128 + ((chunk ^ (row >> 1 & 7)) << 4); };
    auto put16 = [&](int col, float x, float y, float z, float w) {
      *reinterpret_cast<uint2*>(place(l32, col >> 3) + (col & 4) * 2) = uint2{pack2<DT>(x, y), pack2<DT>(z, w)};
    };
    auto put32 = [&](int col, float x, float y, float z, float w) {
      *reinterpret_cast<uint4*>(place(l32, col >> 2)) =
          uint4{__float_as_uint(x), __float_as_uint(y), __float_as_uint(z), __float_as_uint(w)};
    };
    // Rows of BYTES from `mine` to columns [at, ...) of rows [c0, c0 + 32) of the tile; n
    // elements of `size` bytes of them are columns of out.
    auto flush = [&](void* to, int64_t ld, int at, int c0, int n, auto bytesc, auto sizec) {
      constexpr int bytes = decltype(bytesc)::value, size = decltype(sizec)::value, lanes = bytes / 16;
      uint32_t stride = static_cast<uint32_t>(ld) * size;
      asm volatile("" : "+s"(stride));
      const __amdgpu_buffer_rsrc_t rs =
          make_rsrc(static_cast<uint8_t*>(to) + (row0 * ld + at) * size, static_cast<uint32_t>(t.cols) * stride);
      __builtin_amdgcn_wave_barrier();
      const int chunk = ln % lanes;
#pragma unroll
      for (int i = 0; i < 32 * lanes / 64; ++i) {
        const int row = i * (64 / lanes) + ln / lanes;
        const uint32_t off = chunk * (16 / size) < n ? (c0 + row) * stride + chunk * 16 : kNoRow;
        bst16(rs, c0 + row < t.cols ? off : kNoRow, ld16(place(row, chunk)));
      }
      __builtin_amdgcn_wave_barrier();
    };
    constexpr std::integral_constant<int, 128> whole{};
    constexpr std::integral_constant<int, 64> half_row{};
    constexpr std::integral_constant<int, 32> quarter_row{};
    constexpr std::integral_constant<int, 2> two{};
    constexpr std::integral_constant<int, 4> four{};
    if constexpr (KW > 1) {
      // Each wave's sums of one c block to its own slot; wave w adds up block w % 2,
      // registers 8 (w / 2) on of both r blocks: 16 r each.
      f32x4_t sum[2][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int b = 0; b < PB; ++b)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            reinterpret_cast<f32x4_t*>(mine)[(b * 4 + g) * kWave + ln] =
                f32x4_t{acc[b][n][4 * g], acc[b][n][4 * g + 1], acc[b][n][4 * g + 2], acc[b][n][4 * g + 3]};
        s_wave[wv] = static_cast<int>(mine - s_dyn);
        meet();
        if ((wv & 1) == n) {
#pragma unroll
          for (int b = 0; b < PB; ++b)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              sum[b][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int w = 0; w < KW; ++w)
                sum[b][g] += reinterpret_cast<const f32x4_t*>(s_dyn + s_wave[w])[(b * 4 + (wv >> 1) * 2 + g) * kWave + ln];
            }
        }
        meet();
      }
      const int c0 = (wv & 1) * 32, first = t.r0 + (wv >> 1) * 16;
      if constexpr (GATED) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = act_apply(sum[0][g][i], sum[1][g][i], a.act);
          put16(g * 8 + half * 4, h[0], h[1], h[2], h[3]);
        }
        flush(a.out, a.ldo, first, c0, a.R - first, quarter_row, two);
      }
#pragma unroll
      for (int b = 0; b < PB; ++b) {
        if (GATED && a.gu == nullptr) break;
        const int r0 = GATED ? first : first + b * 32;
        const bool wide = !GATED && a.out_dtype == MOE_DTYPE_FP32;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (wide) put32(g * 8 + half * 4, sum[b][g][0], sum[b][g][1], sum[b][g][2], sum[b][g][3]);
          else put16(g * 8 + half * 4, sum[b][g][0], sum[b][g][1], sum[b][g][2], sum[b][g][3]);
        }
        if (GATED) flush(a.gu, 2 * a.R, r0 + b * a.R, c0, a.R - r0, quarter_row, two);
        else if (wide) flush(a.out, a.ldo, r0, c0, a.R - r0, half_row, four);
        else flush(a.out, a.ldo, r0, c0, a.R - r0, quarter_row, two);
      }
      continue;
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int c0 = (WC * n + wc) * 32;
      if constexpr (GATED) {
        const int f0 = wr * 32, left = a.R - t.r0 - f0;
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
          float h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = act_apply(acc[0][n][v + i], acc[1][n][v + i], a.act);
          put16(v * 2 + half * 4, h[0], h[1], h[2], h[3]);
        }
        flush(a.out, a.ldo, t.r0 + f0, c0, left, half_row, two);
        if (a.gu != nullptr) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int v = 0; v < 16; v += 4)
              put16(v * 2 + half * 4, acc[b][n][v], acc[b][n][v + 1], acc[b][n][v + 2], acc[b][n][v + 3]);
            flush(a.gu, 2 * a.R, t.r0 + f0 + b * a.R, c0, left, half_row, two);
          }
        }
      } else if (a.out_dtype == MOE_DTYPE_FP32) {
#pragma unroll
        for (int b = 0; b < PB; ++b) {
          const int r0 = t.r0 + (wr * PB + b) * 32;
#pragma unroll
          for (int v = 0; v < 16; v += 4)
            put32(v * 2 + half * 4, acc[b][n][v], acc[b][n][v + 1], acc[b][n][v + 2], acc[b][n][v + 3]);
          flush(a.out, a.ldo, r0, c0, a.R - r0, whole, four);
        }
      } else {
        const int r0 = t.r0 + wr * PB * 32;
#pragma unroll
        for (int b = 0; b < PB; ++b)
#pragma unroll
          for (int v = 0; v < 16; v += 4)
            put16(b * 32 + v * 2 + half * 4, acc[b][n][v], acc[b][n][v + 1], acc[b][n][v + 2], acc[b][n][v + 3]);
        flush(a.out, a.ldo, r0, c0, a.R - r0, whole, two);
      }
    }
    stores = GATED ? (a.gu != nullptr ? 6 : 2) * NQ : (a.out_dtype == MOE_DTYPE_FP32 ? 8 : 4) * NQ;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads write this block's LDS
}

template <int T, int STEP, int MODE, bool GATED, int DT, int TERMS>
__global__ __launch_bounds__(tile_threads(T), T == 64 ? 1 : 2) void tile_product_kernel(TileArgs a) {
  tile_product<T, STEP, MODE, GATED, DT, TERMS>(a, TileShare{0, 0});
}

// Both gradients: the matrices' tiles, then the rows', which fill up what the first leave
// of the card.
template <int T, int STEP, int DT, int TERMS>
__global__ __launch_bounds__(tile_threads(T), T == 64 ? 1 : 2) void tile_gradients_kernel(TileArgs mat, TileArgs row,
                                                                                          TileShare share) {
  tile_product<T, STEP, kMatGrad, false, DT, TERMS>(mat, TileShare{0, 0});
  __syncthreads();  // both use the same LDS
  tile_product<T, STEP, kRowGrad, false, DT, TERMS>(row, share);
}

}  // namespace moe
