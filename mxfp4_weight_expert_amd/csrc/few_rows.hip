// Forward products of 16-bit matrices for few rows (decode): out[m, n] = sum over k of
// x[m, k] w[e, n, k], or the gated product. The matrices bound it, read once: 64 tokens
// of 16 of 896 experts, K 3584 x 2 N 384 gated 563 us, 6.0 TB/s, K 384 x N 3584 295, 5.7 (a
// large copy reaches 4.9); one token, K 7168 x 2 N 2048 12.9, 4.6, as few blocks hold little
// in flight. Tokens of an expert share its matrix through L2, so the reads are cached
// (non-temporal ones 679 us where these take 584).
//
// Weights go from global memory straight into the 16x16x32 MFMA as its rows, 16 rows x 64
// bytes a load, tokens as its columns (from the caches: a few rows of x). A task is a
// tile of up to 16 rows of one expert times RB (kw = W) or W RB (kw = 1) groups of 16
// weight rows; with kw = W the block's waves split K. Sums meet in LDS, from where the
// activation and the stores take them. Gated groups are eight gate rows and the eight up
// rows of the same features. A wave keeps D steps of K in flight; loads past its last
// step are out of their buffer's range and touch no memory, so every step issues the same
// loads and the waits cover the step being used alone.
#include "rows.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

#include "tile_launch.h"

namespace moe {

namespace {

constexpr int W = 4;  // waves of a block

template <int DT>
__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
  if constexpr (DT == MOE_DTYPE_BF16)
    return mfma16x16x32(as_bf16x8(a), as_bf16x8(b), c);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                  0, 0, 0);
}

template <int DT, bool GATED, int RB>
__global__ __launch_bounds__(64 * W, 4) void few_rows_kernel(TileArgs a, int kw) {
  constexpr int D = RB == 4 ? 1 : RB == 2 ? 2 : 4;
  constexpr int kOut = GATED ? 8 : 16;  // columns of out of a group
  __shared__ f32x4_t s_part[W][RB][kWave];
  __shared__ int32_t s_first[kMaxExperts + 1];  // grouped: row tiles before each expert
  __shared__ int32_t s_wave[W];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_index(), c = lane & 15, q = lane >> 4;
  const int sets = W / kw, kpart = wv % kw, set = wv / kw;
  const int nk = (a.I + 63) >> 6, k0 = nk * kpart / kw, nsteps = nk * (kpart + 1) / kw - k0;
  const int groups = (a.R + kOut - 1) / kOut, ntn = (groups + RB * sets - 1) / (RB * sets);

  int tiles = (a.M + 15) >> 4;
  if (a.offsets != nullptr) {
    constexpr int kPer = kMaxExperts / (64 * W);
    int n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      n[i] = 0;
      if (e < a.E) {
        const int lo = min(max(a.offsets[e], 0), a.M), hi = min(a.offsets[e + 1], a.M);
        n[i] = hi > lo ? (hi - lo + 15) >> 4 : 0;
      }
      sum += n[i];
    }
    const int incl = wave_incl_scan(sum);
    if (lane == kWave - 1) s_wave[wv] = incl;
    __syncthreads();
    int at = incl - sum;
    tiles = 0;
    for (int i = 0; i < W; ++i) {
      if (i < wv) at += s_wave[i];
      tiles += s_wave[i];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s_first[tid * kPer + i] = at;
      at += n[i];
    }
    if (tid == 64 * W - 1) s_first[kMaxExperts] = at;
    __syncthreads();
    tiles = __builtin_amdgcn_readfirstlane(tiles);
  }
  const int items = static_cast<int>(min(static_cast<int64_t>(tiles) * ntn, kMaxTileItems));
  const uint32_t xrow = static_cast<uint32_t>(a.ldq) * 2, wrow = static_cast<uint32_t>(a.ldp) * 2;

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    int e = 0, tn, row0, rows;
    if (a.offsets == nullptr) {
      tn = item / tiles;
      row0 = (item - tn * tiles) * 16;
      rows = min(16, a.M - row0);
    } else {
      int lo = 0, hi = a.E - 1;
      const int tile = item / ntn;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_first[mid] <= tile) lo = mid;
        else hi = mid - 1;
      }
      e = __builtin_amdgcn_readfirstlane(lo);
      const int first = s_first[e], te = __builtin_amdgcn_readfirstlane(s_first[e + 1] - first);
      const int local = item - first * ntn;
      tn = local / te;  // row tiles of the same weights are neighbours
      const int r0 = min(max(a.offsets[e], 0), a.M), r1 = min(a.offsets[e + 1], a.M);
      row0 = r0 + (local - tn * te) * 16;
      rows = min(16, r1 - row0);
    }
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);
    const int bg0 = __builtin_amdgcn_readfirstlane(tn) * RB * sets, rg0 = bg0 + set * RB;

    const __amdgpu_buffer_rsrc_t xb = make_rsrc(
        static_cast<const uint8_t*>(a.q) + static_cast<size_t>(row0) * xrow, kNoRow);
    const __amdgpu_buffer_rsrc_t wb = make_rsrc(
        static_cast<const uint8_t*>(a.p) + static_cast<size_t>(e) * a.pstride * 2, kNoRow);
    f32x4_t acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // lanes of rows that are not there read the tile's first: no column of the result
    // meets another
    const uint32_t xoff = (c < rows ? c : 0) * xrow + q * 16;
    uint32_t woff[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int g = rg0 + b, r = g * kOut + (GATED ? c & 7 : c);
      woff[b] = r < a.R ? static_cast<uint32_t>(r + (GATED && c >= 8 ? a.R : 0)) * wrow + q * 16 : kNoRow;
    }
    uint4 x[D][2], w[D][RB][2];
    auto load = [&](int d, int step) {  // both halves of a row's 128 bytes together
      const int k = (k0 + step) * 64;
      bool in[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        in[j] = step < nsteps && k + j * 32 + q * 8 < a.I;
        x[d][j] = bld16(xb, in[j] ? xoff + k * 2 + j * 64 : kNoRow);
      }
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) w[d][b][j] = bld16(wb, in[j] ? woff[b] + k * 2 + j * 64 : kNoRow);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    for (int s0 = 0; s0 < nsteps; s0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int b = 0; b < RB; ++b) acc[b] = mfma16<DT>(w[d][b][j], x[d][j], acc[b]);
        __builtin_amdgcn_sched_barrier(0);
        load(d, s0 + d + D);
        __builtin_amdgcn_sched_barrier(0);
      }
    }

    // value (row i of group b, token m) is register i % 4 of lane (m, i / 4)
    __syncthreads();  // the last task's sums have been read
#pragma unroll
    for (int b = 0; b < RB; ++b) s_part[wv][b][lane] = acc[b];
    __syncthreads();
    auto sum = [&](int s, int b, int i, int m) {
      float v = 0.0f;
      for (int p = 0; p < kw; ++p) v += reinterpret_cast<const float*>(&s_part[s * kw + p][b][(i >> 2) * 16 + m])[i & 3];
      return v;
    };
    constexpr int kEach = GATED ? 4 : 8;  // pairs of columns of a group
    for (int at = tid; at < sets * RB * kEach * rows; at += 64 * W) {
      const int pair = at % (sets * RB * kEach), m = at / (sets * RB * kEach);
      const int g = pair / kEach, i = pair % kEach * 2, s = g / RB, b = g % RB;
      const int n = (bg0 + g) * kOut + i;
      if (n >= a.R) continue;
      float v[2] = {sum(s, b, i, m), sum(s, b, i + 1, m)};
      const int64_t row = row0 + m;
      if constexpr (GATED) {
        const float u[2] = {sum(s, b, i + 8, m), sum(s, b, i + 9, m)};
        if (a.gu != nullptr) {
          uint16_t* const gu = static_cast<uint16_t*>(a.gu) + row * 2 * a.R + n;
          *reinterpret_cast<uint32_t*>(gu) = pack2<DT>(v[0], v[1]);
          *reinterpret_cast<uint32_t*>(gu + a.R) = pack2<DT>(u[0], u[1]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) v[j] = act_apply(v[j], u[j], a.act);
      }
      if (!GATED && a.out_dtype == MOE_DTYPE_FP32)
        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + row * a.ldo + n) = float2{v[0], v[1]};
      else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * a.ldo + n) = pack2<DT>(v[0], v[1]);
    }
  }
}

template <int DT, bool GATED, int RB>
void few_go(const TileArgs& a, int kw, hipStream_t st) {
  const int64_t groups = (a.R + (GATED ? 7 : 15)) / (GATED ? 8 : 16), sets = W / kw;
  const int64_t tiles = (a.M + 15) / 16 + (a.offsets != nullptr ? std::min(a.E, a.M) : 0);
  const int64_t items = tiles * ((groups + RB * sets - 1) / (RB * sets));
  const int64_t most = int64_t{gpu_cus()} * 4;
  hipLaunchKernelGGL((few_rows_kernel<DT, GATED, RB>), dim3(static_cast<unsigned>(std::min(items, most))),
                     dim3(64 * W), 0, st, a, kw);
}

// Where the weight groups would not fill the card four times over, one group a task, and the
// waves split K if each then has three steps or more; else tasks of two groups (K of 768 on,
// split) or four a wave, which read x less often.
template <int DT, bool GATED>
void few_size(const TileArgs& a, hipStream_t st) {
  const int64_t groups = (a.R + (GATED ? 7 : 15)) / (GATED ? 8 : 16);
  const int64_t U = groups * (a.offsets != nullptr ? std::min(a.E, a.M) : 1);
  const bool deep = a.I >= 768;
  if (U < 2048) few_go<DT, GATED, 1>(a, deep ? W : 1, st);
  else if (deep) few_go<DT, GATED, 2>(a, W, st);
  else few_go<DT, GATED, 4>(a, 1, st);
}

}  // namespace

hipError_t launch_few_rows(const TileArgs& a, bool gated, hipStream_t st) {
  if (a.dtype == MOE_DTYPE_BF16) gated ? few_size<MOE_DTYPE_BF16, true>(a, st) : few_size<MOE_DTYPE_BF16, false>(a, st);
  else gated ? few_size<MOE_DTYPE_FP16, true>(a, st) : few_size<MOE_DTYPE_FP16, false>(a, st);
  return hipGetLastError();
}

}  // namespace moe
