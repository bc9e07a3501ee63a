// Products of 16-bit matrices in tiles of 256 x 256 on the matrix cores, one
// kernel for the forward pass and both gradients of rows times their expert's
// matrix (offsets given) or one matrix for all rows (offsets null):
//
//   kForward  out[m, n] = sum over k of x[m, k] w[e, n, k]
//   kRowGrad  dx[m, k]  = sum over n of dout[m, n] w[e, n, k]
//   kMatGrad  dw[e, n, k] = sum over the rows m of e of dout[m, n] x[m, k]
//
// Each is out[c, r] = sum over i of P[r, i] Q[c, i], r the side whose elements
// follow each other in out. P is the A operand of the 32x32x16 MFMA and Q its B
// operand, so a lane has 16 consecutive elements of out:
//
//              r  c  i    P             Q
//   kForward   n  m  k    w, i inner    x, i inner
//   kRowGrad   k  m  n    w, r inner    dout, i inner
//   kMatGrad   k  n  m    x, r inner    dout, c inner
//
// Operands whose inner index is i go to LDS as rows of 64 bytes (32 i) and are
// read 16 bytes a lane. The others go as 32 rows of 512 bytes, and the transposing
// LDS read (ds_read_b64_tr_b16: within 16 lanes, lane 4 a + b gives four columns
// 4 b of row a, and lane j receives column j of the four rows) makes the operand.
#pragma once

#include "rows.h"
#include "kernels.h"

namespace moe {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

enum { kForward, kRowGrad, kMatGrad };

constexpr int kTile = 256;              // both sides of a tile
constexpr int kStep = 32;               // i of a stage
constexpr int kSide = kTile * kStep * 2;  // bytes of one operand's stage (16 KB)
constexpr int kStage = 2 * kSide;
constexpr int kSlots = 4;               // stages in LDS: one read, up to three in flight
constexpr int kTileThreads = 512;
constexpr int kStageLoads = kStage / 1024 / (kTileThreads / 64);  // a wave's, of 1 KB

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
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(base));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(base >> 32));
  const i32x4_t rsrc = {static_cast<int>(lo), static_cast<int>(hi & 0xffffu), static_cast<int>(kNoRow), 0x00020000};
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(rsrc)
               : "memory", "m0");
}

// Rows of 64 bytes: 16-byte chunk c of row r lies at chunk c ^ chunk_swz(r), so
// that 16 rows of a multiple of 16, and 32 of a multiple of 32, read at one chunk
// fall on different banks.
__device__ __forceinline__ uint32_t chunk_swz(uint32_t r) { return (r >> 3 & 1) * 2 + ((r >> 2 ^ r >> 4) & 1); }
// Rows of 512 bytes: 64-byte piece g of row r lies at piece g ^ piece_swz(r): the four
// rows of a transposing read, and those of its other half eight further on, fall on
// different banks.
__device__ __forceinline__ uint32_t piece_swz(uint32_t r) { return (r & 3) | (r >> 3 & 1) << 2; }

// The r of tile row rho of P (0..255), from the tile's first. In a 32-row block the
// MFMA gives a lane rows 8 b + 4 h + i (h its half, registers 4 b + i): they stand
// for r = 16 h + 4 b + i, the lane's registers in order. Gated: registers 0..7 are
// gate rows and 8..15 up rows of the same eight features.
__device__ __forceinline__ uint32_t plain_row(uint32_t rho) {
  const uint32_t b = rho >> 3 & 3, h = rho >> 2 & 1, i = rho & 3;
  return (rho & ~31u) + 16 * h + 4 * b + i;
}
__device__ __forceinline__ uint32_t gated_feature(uint32_t rho) {
  const uint32_t b = rho >> 3 & 1, h = rho >> 2 & 1, i = rho & 3;
  return (rho >> 5) * 16 + 8 * h + 4 * b + i;
}
__device__ __forceinline__ bool gated_up(uint32_t rho) { return (rho >> 4 & 1) != 0; }

// One tile of out.
struct TileItem {
  int e;      // matrix
  int r0;     // first r (gated: feature)
  int c0;     // first c: row of Q (kMatGrad: column of dout)
  int cols;   // c that the tile has
  int first;  // kMatGrad: first of the expert's rows
  int len;    // i to sum over
};

template <int MODE, bool GATED, int DT>
__global__ __launch_bounds__(kTileThreads, 2) void tile_product_kernel(TileArgs a) {
  static_assert(!GATED || MODE == kForward, "the activation follows the forward product");
  constexpr bool kPInner = MODE == kForward;   // i is P's inner index
  constexpr bool kQInner = MODE != kMatGrad;
  constexpr int kWide = GATED ? kTile / 2 : kTile;  // r of a tile
  constexpr int PB = 2, NQ = 4;                     // 32-blocks of a wave: r, c
  extern __shared__ __attribute__((aligned(1024))) uint8_t s_dyn[];
  __shared__ int32_t s_wave[kTileThreads / 64];
  int32_t* const s_first = reinterpret_cast<int32_t*>(s_dyn + kSlots * kStage);  // grouped: tiles before each expert
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint8_t*)s_dyn));
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_index();
  const int wr = wv & 3, wc = wv >> 2;  // wave: 64 r, and every second 32 c
  const int nr = (a.R + kWide - 1) / kWide;

  // The tiles of the experts' rows.
  int tiles = (a.M + kTile - 1) / kTile;
  if (MODE != kMatGrad && a.offsets != nullptr) {
    constexpr int kPer = kMaxExperts / kTileThreads;
    int n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      n[i] = 0;
      if (e < a.E) {
        const int lo = min(max(a.offsets[e], 0), a.M), hi = min(a.offsets[e + 1], a.M);
        n[i] = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
      }
      sum += n[i];
    }
    const int incl = wave_incl_scan(sum);
    if (lane == kWave - 1) s_wave[wv] = incl;
    __syncthreads();
    int at = incl - sum;
    tiles = 0;
    for (int i = 0; i < kTileThreads / 64; ++i) {
      if (i < wv) at += s_wave[i];
      tiles += s_wave[i];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      if (e <= a.E) s_first[e] = at;
      at += n[i];
    }
    if (a.E == kMaxExperts && tid == kTileThreads - 1) s_first[kMaxExperts] = at;
    __syncthreads();
    tiles = __builtin_amdgcn_readfirstlane(tiles);
  }
  const int nc = (a.C + kTile - 1) / kTile;  // kMatGrad: tiles along dout's columns
  const int items = static_cast<int>(min(
      MODE == kMatGrad ? static_cast<int64_t>(a.E) * nc * nr : static_cast<int64_t>(tiles) * nr, kMaxTileItems));

  // The blocks of an XCD (block ids go round over the eight) walk a range of the
  // items together, so that neighbours, which share operands, meet in its L2.
  const int per = (items + 7) >> 3, walkers = static_cast<int>(gridDim.x) >> 3;
  const int xcd = blockIdx.x & 7, last = min(items, (xcd + 1) * per);
  const int item0 = xcd * per + (blockIdx.x >> 3);

  auto decode = [&](int item) {
    TileItem t;
    if constexpr (MODE == kMatGrad) {
      const int re = item / nr, e = re / nc;
      t.e = e;
      t.r0 = (item - re * nr) * kWide;
      t.c0 = (re - e * nc) * kTile;
      t.cols = min(kTile, a.C - t.c0);
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
      t.c0 = lo + local * kTile;
      t.cols = min(kTile, hi - t.c0);
      t.first = 0;
      t.len = a.I;
    }
    return t;
  };

  // ---- loads. A wave brings 2 KB of each operand: 32 rows of 64 bytes, or 4 of 512.
  int l_item = item0, l_left = 0;  // i left of the item that loads come from
  uint64_t pbase = 0, qbase = 0;   // where the next stage begins
  uint32_t poff[2], qoff[2];
  uint32_t pi[2], qi[2];           // the lane's i in a stage
  auto start = [&]() {
    const TileItem t = decode(l_item);
    l_left = t.len;
    pbase = reinterpret_cast<uint64_t>(a.p);
    qbase = reinterpret_cast<uint64_t>(a.q);
    if constexpr (MODE == kMatGrad)
      pbase += (static_cast<uint64_t>(t.first) * a.ldp + t.r0) * 2;
    else if constexpr (kPInner)
      pbase += (static_cast<uint64_t>(t.e) * a.pstride + static_cast<uint64_t>(t.r0) * a.ldp) * 2;
    else
      pbase += (static_cast<uint64_t>(t.e) * a.pstride + t.r0) * 2;
    qbase += (MODE == kMatGrad ? static_cast<uint64_t>(t.first) * a.ldq + t.c0
                               : static_cast<uint64_t>(t.c0) * a.ldq) * 2;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (kPInner) {
        const uint32_t rho = wv * 32 + j * 16 + (lane >> 2), chunk = (lane & 3) ^ chunk_swz(rho);
        const uint32_t r = GATED ? gated_feature(rho) : plain_row(rho);
        const bool in = t.r0 + r < static_cast<uint32_t>(a.R);
        poff[j] = in ? (r + (GATED && gated_up(rho) ? a.R : 0)) * static_cast<uint32_t>(a.ldp) * 2 + chunk * 16 : kNoRow;
        pi[j] = chunk * 8;
      } else {
        const uint32_t row = wv * 4 + j * 2 + (lane >> 5);
        const uint32_t chunk = ((lane >> 2 & 7) ^ piece_swz(row)) * 4 + (lane & 3);
        const bool in = t.r0 + chunk * 8 < static_cast<uint32_t>(a.R);
        poff[j] = in ? row * static_cast<uint32_t>(a.ldp) * 2 + chunk * 16 : kNoRow;
        pi[j] = row;
      }
      if constexpr (kQInner) {
        const uint32_t c = wv * 32 + j * 16 + (lane >> 2), chunk = (lane & 3) ^ chunk_swz(c);
        qoff[j] = c < static_cast<uint32_t>(t.cols) ? c * static_cast<uint32_t>(a.ldq) * 2 + chunk * 16 : kNoRow;
        qi[j] = chunk * 8;
      } else {
        const uint32_t row = wv * 4 + j * 2 + (lane >> 5);
        const uint32_t chunk = ((lane >> 2 & 7) ^ piece_swz(row)) * 4 + (lane & 3);
        qoff[j] = chunk * 8 < static_cast<uint32_t>(t.cols) ? row * static_cast<uint32_t>(a.ldq) * 2 + chunk * 16 : kNoRow;
        qi[j] = row;
      }
    }
  };
  // The next stage into slot `slot`; past the last item loads that touch no memory, so
  // that the waits count the same everywhere.
  auto issue = [&](int slot) {
    while (l_left <= 0 && l_item < last) {
      l_item += walkers;
      if (l_item < last) start();
    }
    const uint32_t at = lds0 + slot * kStage + wv * 2048;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      load_to_lds(pbase, pi[j] < static_cast<uint32_t>(max(l_left, 0)) ? poff[j] : kNoRow, at + j * 1024);
      load_to_lds(qbase, qi[j] < static_cast<uint32_t>(max(l_left, 0)) ? qoff[j] : kNoRow, at + kSide + j * 1024);
    }
    pbase += kPInner ? kStep * 2 : static_cast<uint64_t>(a.ldp) * (kStep * 2);
    qbase += kQInner ? kStep * 2 : static_cast<uint64_t>(a.ldq) * (kStep * 2);
    l_left -= kStep;
  };

  if (item0 >= last) return;
  start();
#pragma unroll
  for (int s = 0; s < kSlots - 1; ++s) issue(s);

  // ---- operands from LDS
  const int l32 = lane & 31, half = lane >> 5;
  uint32_t pat[2], qat[4];
  if constexpr (kPInner) {
#pragma unroll
    for (int s = 0; s < 2; ++s) pat[s] = (wr * 64 + l32) * 64 + (((2 * s + half) ^ chunk_swz(l32)) << 4);
  } else {
    const uint32_t row = half * 8 + (lane >> 2 & 3), gg = lane >> 4 & 1, q = lane & 3;
    // columns 4 q of a 16-lane group stand for the rows 16 gg + 4 q of the MFMA
    const uint32_t b = 2 * gg + (q >> 1), h = q & 1;
#pragma unroll
    for (int p = 0; p < 2; ++p) pat[p] = row * 512 + (((wr * 2 + p) ^ piece_swz(row)) << 6) + (4 * h + b) * 8;
  }
  if constexpr (kQInner) {
#pragma unroll
    for (int s = 0; s < 2; ++s) qat[s] = kSide + (wc * 32 + l32) * 64 + (((2 * s + half) ^ chunk_swz(l32)) << 4);
    qat[2] = qat[3] = 0;
  } else {
    const uint32_t row = half * 8 + (lane >> 2 & 3), gg = lane >> 4 & 1, q = lane & 3;
#pragma unroll
    for (int n = 0; n < 4; ++n) qat[n] = kSide + row * 512 + (((2 * n + wc) ^ piece_swz(row)) << 6) + (4 * gg + q) * 8;
  }
  auto transposed = [&](const uint8_t* at) {  // eight i of 32 rows or columns
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * 512));
    const uint2 u = __builtin_bit_cast(uint2, lo), v = __builtin_bit_cast(uint2, hi);
    return uint4{u.x, u.y, v.x, v.y};
  };
  auto read_p = [&](const uint8_t* stage, int s, int b) {
    if constexpr (kPInner) return ld16(stage + pat[s] + b * 32 * 64);
    else return transposed(stage + pat[b] + s * 16 * 512);
  };
  auto read_q = [&](const uint8_t* stage, int s, int n) {
    if constexpr (kQInner) return ld16(stage + qat[s] + n * 64 * 64);
    else return transposed(stage + qat[n] + s * 16 * 512);
  };

  f32x16_t acc[PB][NQ];
  uint4 p0[PB], q0[NQ], p1[PB], q1[NQ];
  int slot = 0;
  for (int item = item0; item < last; item += walkers) {
    const TileItem t = decode(item);
    const int stages = (t.len + kStep - 1) / kStep;
    // 32-blocks of c that hold anything, for this wave
    const int blocks = min(NQ, max(0, (t.cols - 32 * wc + 63) >> 6));
#pragma unroll
    for (int b = 0; b < PB; ++b)
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[b][n][v] = 0.0f;

    // A stage's second half is multiplied after the next stage's barrier, while
    // that stage's first operands are read.
    auto walk = [&](auto nqc) {
      constexpr int N = decltype(nqc)::value;
      auto mul = [&](const uint4 (&p)[PB], const uint4 (&q)[NQ]) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int b = 0; b < PB; ++b) acc[b][n] = mfma32<DT>(p[b], q[n], acc[b][n]);
      };
#pragma unroll
      for (int b = 0; b < PB; ++b) p1[b] = uint4{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < N; ++n) q1[n] = uint4{0, 0, 0, 0};
      for (int k = 0; k < stages; ++k) {
        // this stage has come (three are in flight), and no wave still reads the slot
        // that the next loads go to
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kSlots - 2) * kStageLoads) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(slot == 0 ? kSlots - 1 : slot - 1);
        const uint8_t* const stage = s_dyn + slot * kStage;
        if constexpr (N > 0) {
#pragma unroll
          for (int b = 0; b < PB; ++b) p0[b] = read_p(stage, 0, b);
#pragma unroll
          for (int n = 0; n < N; ++n) q0[n] = read_q(stage, 0, n);
          mul(p1, q1);
#pragma unroll
          for (int b = 0; b < PB; ++b) p1[b] = read_p(stage, 1, b);
#pragma unroll
          for (int n = 0; n < N; ++n) q1[n] = read_q(stage, 1, n);
          mul(p0, q0);
        }
        slot = slot == kSlots - 1 ? 0 : slot + 1;
      }
      mul(p1, q1);
    };
    switch (blocks) {
      case 4: walk(std::integral_constant<int, 4>{}); break;
      case 3: walk(std::integral_constant<int, 3>{}); break;
      case 2: walk(std::integral_constant<int, 2>{}); break;
      case 1: walk(std::integral_constant<int, 1>{}); break;
      default: walk(std::integral_constant<int, 0>{}); break;
    }

    // ---- results: lane (c, h) has 16 r of each 32-block
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int c = (2 * n + wc) * 32 + l32;
      if (c >= t.cols) continue;
      const int64_t row = (MODE == kMatGrad ? static_cast<int64_t>(t.e) * a.C : 0) + t.c0 + c;
#pragma unroll
      for (int b = 0; b < PB; ++b) {
        if constexpr (GATED) {
          const int f = t.r0 + (wr * PB + b) * 16 + half * 8;
          if (f >= a.R) continue;
          float h[8];
          float g[8], u[8];
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            g[v] = acc[b][n][v];
            u[v] = acc[b][n][v + 8];
            h[v] = act_apply(g[v], u[v], a.act);
          }
          uint16_t* const o = static_cast<uint16_t*>(a.out) + row * a.ldo + f;
          *reinterpret_cast<uint4*>(o) = Row<DT>::pack(h);
          if (a.gu != nullptr) {
            uint16_t* const p = static_cast<uint16_t*>(a.gu) + row * 2 * a.R + f;
            *reinterpret_cast<uint4*>(p) = Row<DT>::pack(g);
            *reinterpret_cast<uint4*>(p + a.R) = Row<DT>::pack(u);
          }
        } else {
          const int r = t.r0 + (wr * PB + b) * 32 + half * 16;
          float f[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) f[v] = acc[b][n][v];
          if (a.out_dtype == MOE_DTYPE_FP32) {
            float* const o = static_cast<float*>(a.out) + row * a.ldo + r;
#pragma unroll
            for (int v = 0; v < 16; v += 4)
              if (r + v < a.R) *reinterpret_cast<uint4*>(o + v) = Row<MOE_DTYPE_FP32>::pack(f + v);
          } else {
            uint16_t* const o = static_cast<uint16_t*>(a.out) + row * a.ldo + r;
#pragma unroll
            for (int v = 0; v < 16; v += 8)
              if (r + v < a.R) *reinterpret_cast<uint4*>(o + v) = Row<DT>::pack(f + v);
          }
        }
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads write this block's LDS
}

}  // namespace moe
