#pragma once

// Products of a few rows with 4-bit weights in the packed layout, for one
// matrix or one per expert:
//   out[m, n] = bias[n] + sum over groups g of s[n, g] *
//               sum over k in g of (c[n, k] - z[n, g]) x[m, k].
// The weights bound it: N * K / 2 bytes and the scales, read once.
//
// Tokens are the M side of the 16x16x32 MFMA, weights the N side: lane
// (r = lane % 16, q = lane / 16) loads 16 bytes = 32 codes of weight row r, so
// a wave's load is one contiguous 1 KB block of the packed layout (a K step of
// 128), and a group's scale is one value per lane for its four results.
// A lane's 32 codes are a 32-group of their own, so MFMA j on dword j of every
// lane would mix four groups. Two ways out:
//   - bfloat16 tokens with MXFP4: the scale is applied by the hardware convert
//     (exact: a code times a power of two is a bfloat16), and the groups may mix;
//   - else a 4x4 dword transpose across the quads (two lane swaps each of 32 and
//     of 16 lanes) gives MFMA j group j of the step, whose sum meets its scale in
//     32 bits.
// INT4 codes 0..15 are read as E4M3: its codes 0..15 are k * 2^-9 (subnormals
// and the first binade), so the convert with scale 2^9 gives the code exactly.
// The zero points are taken off as sum over g of (s z)[n, g] X[m, g], X the sum
// of x over the group, by one 16x16x4 float MFMA a step: exact codes and one
// correction in 32 bits.
#include "rows.h"
#include "kernels.h"

#include <atomic>

namespace moe {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

typedef uint32_t u32x4_byte __attribute__((ext_vector_type(4), aligned(1)));

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
// d[j] of quad q <- d[q] of quad j, for the 16 lanes of each quad.
__device__ __forceinline__ void transpose_quads(uint32_t (&d)[4]) {
  swap32(d[0], d[2]);
  swap32(d[1], d[3]);
  swap16(d[0], d[1]);
  swap16(d[2], d[3]);
}

template <int DT>
__device__ __forceinline__ f32x4_t mfma_rows(uint4 a, uint4 b, f32x4_t c) {
  if constexpr (DT == MOE_DTYPE_BF16)
    return mfma16x16x32(as_bf16x8(a), as_bf16x8(b), c);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// Eight E2M1 codes (low nibble first) -> eight halves, exact.
__device__ __forceinline__ uint4 decode_fp4x8_f16(uint32_t d) {
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 3));
  return r;
}
// Eight codes 0..15 -> tokens' type, exact, in the order 0 2 4 6 1 3 5 7.
template <int DT, bool HI>
__device__ __forceinline__ uint32_t code_pair(uint32_t bytes) {
  if constexpr (DT == MOE_DTYPE_BF16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, 512.0f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 512.0f, HI));
}
template <int DT>
__device__ __forceinline__ uint4 decode_int4x8(uint32_t d) {
  const uint32_t lo = d & 0x0f0f0f0fu, hi = (d >> 4) & 0x0f0f0f0fu;
  return uint4{code_pair<DT, false>(lo), code_pair<DT, true>(lo), code_pair<DT, false>(hi),
               code_pair<DT, true>(hi)};
}
// Tokens in that order.
__device__ __forceinline__ uint4 even_odd(const uint4& v) {
  return uint4{__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
               __builtin_amdgcn_perm(v.y, v.x, 0x07060302u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u)};
}

// E8M0 byte as a float: 2^(e - 127), 255 NaN, 0 the subnormal 2^-127.
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  const uint32_t bits = e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : e << 23;
  return __uint_as_float(bits);
}
template <int DT>
__device__ __forceinline__ float scale16(uint32_t bits) {
  if constexpr (DT == MOE_DTYPE_BF16)
    return __uint_as_float(bits << 16);
  else
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

// How a lane's 32 codes of a K step meet the MFMAs (dword j feeds MFMA j).
// kMix: dword j as loaded, MFMA j mixing the four 32-groups of the step (one
// scale for all of them: G = 128, or scales inside the codes); kHalf: two lane
// swaps, MFMAs 0, 1 on the first 64 and 2, 3 on the second (G = 64); kOne: four
// swaps, MFMA j on 32-group j.
enum { kMix, kHalf, kOne };
__device__ __forceinline__ constexpr int w4_layout(int fmt, int g, int dt) {
  return fmt == MOE_W4_MXFP4 ? (dt == MOE_DTYPE_BF16 ? kMix : kOne)
                             : (g == 32 ? kOne : g == 64 ? kHalf : kMix);
}
// Byte offset in a step's 256 bytes of a token row: quad q's 16 bytes for MFMA j.
template <int L>
__device__ __forceinline__ constexpr uint32_t token_quad(uint32_t q) {
  return L == kMix ? q * 64 : L == kHalf ? (q & 1) * 64 + (q >> 1) * 32 : q * 16;
}
template <int L>
__device__ __forceinline__ constexpr uint32_t token_mfma(uint32_t j) {
  return L == kMix ? j * 16 : L == kHalf ? (j & 1) * 16 + (j >> 1) * 128 : j * 64;
}

constexpr int kW4Waves = 4;
// K steps in flight per wave: three where a step is 8 KB of tokens and weights,
// two where the tokens alone are 8 or 16 KB.
constexpr int w4_depth(int mt, int rb) { return mt == 1 ? (rb == 4 ? 3 : 4) : 2; }

// One wave copies `bytes` (a multiple of ALIGN) of global memory to LDS with its
// block: 16-byte pieces, then the last bytes one ALIGN unit a thread.
template <int ALIGN>
__device__ __forceinline__ void block_to_lds(uint8_t* lds, const uint8_t* src, int bytes) {
  const int n = bytes >> 4, tid = threadIdx.x;
  for (int c = tid; c < n; c += 256)
    *reinterpret_cast<uint4*>(lds + 16 * c) = __builtin_bit_cast(
        uint4, static_cast<u32x4_t>(*reinterpret_cast<const u32x4_byte*>(src + 16 * c)));
  const int at = 16 * n + ALIGN * tid;
  if (at < bytes) {
    if constexpr (ALIGN == 1) lds[at] = src[at];
    else if constexpr (ALIGN == 2)
      *reinterpret_cast<uint16_t*>(lds + at) = *reinterpret_cast<const uint16_t*>(src + at);
    else *reinterpret_cast<uint32_t*>(lds + at) = *reinterpret_cast<const uint32_t*>(src + at);
  }
}

// LDS: the waves' parts, then the scale rows and the zero points of the block's
// weight rows.
template <int MT, int RB>
__host__ __device__ constexpr int w4_part_bytes(int kw) { return kw == 1 ? 0 : kW4Waves * RB * MT * 1024; }

// FMT, G: weight format and group; DT: tokens' type; MT: 16-row tiles of x a
// task takes; RB: 16-row weight groups a wave takes.
//
// A task is a row tile times RB (kw = 4) or 4 RB (kw = 1) weight groups. With
// kw = 4 the four waves split K and join in LDS at the end; with kw = 1 (short
// K) each has weight groups of its own. A wave walks its K steps with a ring
// of w4_depth steps in flight, tokens and weights; loads past its last step are
// out of their buffer's range and touch no memory, so every step issues the
// same loads and the waits cover the step being used alone. The scales of the
// block's weight rows lie one after another and come to LDS in one copy.
template <int FMT, int G, int DT, int MT, int RB>
__global__ __launch_bounds__(256) void w4_kernel(W4Args a) {
  constexpr int L = w4_layout(FMT, G, DT);
  constexpr bool kInt = FMT == MOE_W4_INT4;
  constexpr bool kFold = FMT == MOE_W4_MXFP4 && DT == MOE_DTYPE_BF16;  // scale in the convert
  constexpr int D = w4_depth(MT, RB);
  constexpr int kTile = 16 * MT;
  constexpr int kGroups = 128 / G;                   // groups of a step
  constexpr int kScale = kInt ? 2 : 1;               // bytes of a scale
  extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];
  __shared__ int32_t s_first[kMaxExperts + 1];  // grouped: row tiles before each expert
  __shared__ int32_t s_wave[kW4Waves];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_index();
  const int r = lane & 15, q = lane >> 4;
  const int nk = a.K >> 7, ng = (a.N + 15) >> 4;
  const int sets = kW4Waves / a.kw;  // sets of weight groups in the block
  const int kpart = wv % a.kw, set = wv / a.kw;
  const int k0 = nk * kpart / a.kw, nsteps = nk * (kpart + 1) / a.kw - k0;
  const int ntn = (ng + RB * sets - 1) / (RB * sets);
  const int srow = nk * kGroups * kScale, zrow = nk * kGroups;  // bytes of a weight row's
  uint8_t* const s_scale = s_dyn + w4_part_bytes<MT, RB>(a.kw);
  uint8_t* const s_zero = s_scale + ((RB * sets * 16 * srow + 15) & ~15);

  int tiles = (a.M + kTile - 1) / kTile;
  if (a.offsets != nullptr) {
    constexpr int kPer = kMaxExperts / 256;
    int c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      c[i] = 0;
      if (e < a.E) {
        const int lo = min(max(a.offsets[e], 0), a.M), hi = min(a.offsets[e + 1], a.M);
        c[i] = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
      }
      sum += c[i];
    }
    const int incl = wave_incl_scan(sum);
    if (lane == kWave - 1) s_wave[wv] = incl;
    __syncthreads();
    int at = incl - sum;
    tiles = 0;
    for (int i = 0; i < kW4Waves; ++i) {
      if (i < wv) at += s_wave[i];
      tiles += s_wave[i];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s_first[tid * kPer + i] = at;
      at += c[i];
    }
    if (tid == 255) s_first[kMaxExperts] = at;
    __syncthreads();
    tiles = __builtin_amdgcn_readfirstlane(tiles);
  }
  const int items = tiles * ntn;

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    int e = 0, tn, row0, rows;
    if (a.offsets == nullptr) {
      // row tiles of the same weights are neighbours: the second's come from L2
      tn = item / tiles;
      row0 = (item - tn * tiles) * kTile;
      rows = min(kTile, a.M - row0);
    } else {
      int lo = 0, hi = a.E - 1;  // the last expert whose first tile is at or before the item's
      const int tile = item / ntn;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_first[mid] <= tile) lo = mid;
        else hi = mid - 1;
      }
      e = __builtin_amdgcn_readfirstlane(lo);
      const int first = s_first[e], te = s_first[e + 1] - first;
      const int local = item - first * ntn;
      tn = local / te;
      const int m = local - tn * te;
      const int r0 = min(max(a.offsets[e], 0), a.M), r1 = min(a.offsets[e + 1], a.M);
      row0 = r0 + m * kTile;
      rows = min(kTile, r1 - row0);
    }
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);
    tn = __builtin_amdgcn_readfirstlane(tn);
    const int bg0 = tn * RB * sets;       // the block's first weight group
    const int rg0 = bg0 + set * RB;       // the wave's
    const int live = min(RB, ng - rg0);   // groups of it that exist; may be <= 0

    // the block's scale rows; a task's first barrier is passed by a wave only
    // after it has read the last one's
    {
      const size_t row = static_cast<size_t>(e) * a.N + bg0 * 16;
      const int nrow = min(RB * sets * 16, a.N - bg0 * 16);
      block_to_lds<kInt ? 2 : 4>(s_scale, static_cast<const uint8_t*>(a.scales) + row * srow, nrow * srow);
      if (kInt && a.zeros != nullptr) block_to_lds<1>(s_zero, a.zeros + row * zrow, nrow * zrow);
    }

    // tokens: rows past the tile's are out of the buffer's range and read as 0
    const uint32_t xrow = static_cast<uint32_t>(a.ldx) * 2;
    const __amdgpu_buffer_rsrc_t xb = make_rsrc(
        static_cast<const uint8_t*>(a.x) + static_cast<size_t>(row0) * xrow,
        static_cast<uint32_t>(rows - 1) * xrow + static_cast<uint32_t>(a.K) * 2);
    uint32_t xoff[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
      xoff[t] = t * 16 + r < rows ? (t * 16 + r) * xrow + token_quad<L>(q) + k0 * 256 : kNoRow;
    const uint32_t gbytes = static_cast<uint32_t>(nk) * kPkBlock;  // a weight group's
    const __amdgpu_buffer_rsrc_t wb = make_rsrc(
        a.w + (static_cast<size_t>(e) * ng + rg0) * gbytes, live > 0 ? live * gbytes : 0);
    const uint32_t woff = k0 * kPkBlock + r * 64 + q * 16;

    uint4 xf[D][MT][4], w[D][RB];
    auto load = [&](int d, int step) {  // step: wave-uniform
      const bool in = step < nsteps;
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xf[d][t][j] = bld16(xb, in ? xoff[t] + step * 256 + token_mfma<L>(j) : kNoRow);
#pragma unroll
      for (int b = 0; b < RB; ++b)
        w[d][b] = bld16nt(wb, in ? woff + b * gbytes + step * kPkBlock : kNoRow);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    __syncthreads();  // scales are in LDS

    f32x4_t acc[RB][MT];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[b][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    auto compute = [&](int d, int ks) {
      float xs[MT];  // lane (m, q): sum of row m's tokens of MFMA q
      if constexpr (kInt) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t one = r == 4 * j ? (DT == MOE_DTYPE_BF16 ? 0x3f803f80u : 0x3c003c00u) : 0u;
            sum = mfma_rows<DT>(uint4{one, one, one, one}, xf[d][t][j], sum);
            xf[d][t][j] = even_odd(xf[d][t][j]);
          }
          xs[t] = sum[0];
        }
      }
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int wr = (set * RB + b) * 16 + r;  // weight row in the block's
        uint32_t dw[4] = {w[d][b].x, w[d][b].y, w[d][b].z, w[d][b].w};
        if constexpr (kFold) {
          const float s = e8m0_scale_operand(s_scale[wr * srow + ks * 4 + q]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 f = __builtin_bit_cast(uint4, decode_fp4x8(dw[j], s));
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[b][t] = mfma_rows<DT>(xf[d][t][j], f, acc[b][t]);
          }
        } else {
          constexpr int kPer = 4 / kGroups;  // MFMAs a group's sum takes
          float s[kGroups];
          const uint8_t* sp = s_scale + wr * srow + ks * kGroups * kScale;
          if constexpr (!kInt) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(sp);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) s[g] = e8m0_value((v >> (8 * g)) & 0xffu);
          } else {
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
              s[g] = scale16<DT>(reinterpret_cast<const uint16_t*>(sp)[g]);
          }
          if constexpr (L == kOne) {
            transpose_quads(dw);
          } else if constexpr (L == kHalf) {
            swap32(dw[0], dw[2]);
            swap32(dw[1], dw[3]);
          }
          f32x4_t part[MT];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 f;
            if constexpr (kInt) f = decode_int4x8<DT>(dw[j]);
            else f = decode_fp4x8_f16(dw[j]);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              if (j % kPer == 0) part[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
              part[t] = mfma_rows<DT>(xf[d][t][j], f, part[t]);
              if (j % kPer == kPer - 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[b][t][i] += s[j / kPer] * part[t][i];
              }
            }
          }
          if constexpr (kInt) {
            const int gq = q / kPer;
            float z = 8.0f, sq = s[0];
            if (a.zeros != nullptr) z = static_cast<float>(s_zero[wr * zrow + ks * kGroups + gq]);
#pragma unroll
            for (int g = 1; g < kGroups; ++g) sq = gq == g ? s[g] : sq;
#pragma unroll
            for (int t = 0; t < MT; ++t)
              acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(xs[t], -sq * z, acc[b][t], 0, 0, 0);
          }
        }
      }
    };
    for (int s0 = 0; s0 < nsteps; s0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (s0 + d < nsteps) compute(d, k0 + s0 + d);
        load(d, s0 + d + D);
      }
    }

    // Join the waves that share weight rows, and store: value (m, n) of a tile
    // is register m % 4 of lane (n, m / 4).
    auto store = [&](int m, int n, float v) {
      if (m >= rows || n >= a.N) return;
      if (a.bias != nullptr)
        v += Row<DT>::get(static_cast<const uint8_t*>(a.bias) + (static_cast<size_t>(e) * a.N + n) * 2);
      const size_t at = static_cast<size_t>(row0 + m) * a.ldo + n;
      if (a.out_dtype == MOE_DTYPE_FP32) static_cast<float*>(a.out)[at] = v;
      else if (a.out_dtype == MOE_DTYPE_BF16) static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(v);
      else static_cast<_Float16*>(a.out)[at] = static_cast<_Float16>(v);
    };
    if (a.kw == 1) {
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) store(t * 16 + q * 4 + i, (rg0 + b) * 16 + r, acc[b][t][i]);
      __syncthreads();  // before the next task's scales
    } else {
      f32x4_t* part = reinterpret_cast<f32x4_t*>(s_dyn);  // [wave][RB * MT][lane]
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) part[(wv * RB * MT + b * MT + t) * kWave + lane] = acc[b][t];
      __syncthreads();
      const int m = tid >> 4, nn = tid & 15;
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          float v = 0.0f;
#pragma unroll
          for (int u = 0; u < kW4Waves; ++u)
            v += reinterpret_cast<const float*>(
                part + (u * RB * MT + b * MT + t) * kWave + (m >> 2) * 16 + nn)[m & 3];
          store(t * 16 + m, (rg0 + b) * 16 + nn, v);
        }
    }
  }
}

// Blocks of a kernel that a CU holds, by its LDS (kept per size and instance).
template <class F>
int w4_resident(F kernel, int lds) {
  static std::atomic<int> kept[161];
  std::atomic<int>& k = kept[lds >> 10];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, reinterpret_cast<const void*>(kernel), 256,
                                                     (lds | 1023) + 1) != hipSuccess || n < 1)
      n = 1;
    k.store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int FMT, int G, int DT, int MT, int RB>
void w4_go(const W4Args& a, hipStream_t st) {
  constexpr bool kInt = FMT == MOE_W4_INT4;
  const int64_t sets = kW4Waves / a.kw;
  const int64_t ntn = ((a.N + 15) / 16 + RB * sets - 1) / (RB * sets);
  const int64_t tiles = (a.M + 16 * MT - 1) / (16 * MT) + (a.offsets != nullptr ? a.E : 0);
  const int64_t items = ntn * tiles;
  const int groups = (a.K >> 7) * (128 / G), nrow = RB * static_cast<int>(sets) * 16;
  const int lds = w4_part_bytes<MT, RB>(a.kw) + ((nrow * groups * (kInt ? 2 : 1) + 15) & ~15) +
                  (kInt && a.zeros != nullptr ? (nrow * groups + 15) & ~15 : 0);
  auto kernel = w4_kernel<FMT, G, DT, MT, RB>;
  const int64_t most = int64_t{256} * w4_resident(kernel, lds);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(items < most ? items : most)), dim3(256), lds,
                     st, a);
}

template <int FMT, int G, int DT>
void w4_rows(const W4Args& a, hipStream_t st) {
  // tiles of x rows: by the rows an expert has on average
  const int per = a.offsets != nullptr ? (a.M + a.E - 1) / a.E : a.M;
  // weight groups a wave takes: as many as leave two tasks for every CU
  const int64_t groups = static_cast<int64_t>((a.N + 15) / 16) * (a.offsets != nullptr ? a.E : 1);
  const int64_t tasks = groups * a.kw / kW4Waves;
  if (per <= 16) {
    if (tasks >= 4 * 512) w4_go<FMT, G, DT, 1, 4>(a, st);
    else if (tasks >= 2 * 256) w4_go<FMT, G, DT, 1, 2>(a, st);
    else w4_go<FMT, G, DT, 1, 1>(a, st);
  } else if (per <= 32) {
    if (tasks >= 4 * 256) w4_go<FMT, G, DT, 2, 4>(a, st);
    else w4_go<FMT, G, DT, 2, 1>(a, st);
  } else {
    if (tasks >= 2 * 256) w4_go<FMT, G, DT, 4, 2>(a, st);
    else w4_go<FMT, G, DT, 4, 1>(a, st);
  }
}

// All formats of one token type (one translation unit each).
template <int DT>
hipError_t w4_formats(const W4Args& a, hipStream_t st) {
  if (a.format == MOE_W4_MXFP4) w4_rows<MOE_W4_MXFP4, 32, DT>(a, st);
  else if (a.group == 32) w4_rows<MOE_W4_INT4, 32, DT>(a, st);
  else if (a.group == 64) w4_rows<MOE_W4_INT4, 64, DT>(a, st);
  else w4_rows<MOE_W4_INT4, 128, DT>(a, st);
  return hipGetLastError();
}

}  // namespace moe
