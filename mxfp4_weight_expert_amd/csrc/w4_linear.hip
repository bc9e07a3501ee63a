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

#include <type_traits>

namespace moe {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr int kW4Steps = 4;    // K steps of 128 that a wave holds of x at once (one row tile)
constexpr int kW4Waves = 4;

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

template <int DT>
__device__ __forceinline__ float sum8(const uint4& v) {
  float f[8];
  Row<DT>::unpack(v, f);
  return ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
}

}  // namespace

// Raw scales (and zero points) of one weight row's K step.
struct StepScales {
  uint32_t s[2], z;
};

// FMT, G: weight format and group; DT: tokens' type; MT: 16-row tiles of x at
// once; RB: 16-row weight groups that share a wave's tokens.
template <int FMT, int G, int DT, int MT, int RB>
__global__ __launch_bounds__(256) void w4_kernel(W4Args a) {
  constexpr bool kFold = FMT == MOE_W4_MXFP4 && DT == MOE_DTYPE_BF16;  // scale in the convert
  constexpr bool kInt = FMT == MOE_W4_INT4;
  constexpr int C = kW4Steps / MT;  // K steps of x held at once
  constexpr int kTile = 16 * MT;    // rows of x a task takes
  __shared__ f32x4_t s_part[kW4Waves][RB * MT][kWave];
  __shared__ int32_t s_first[kMaxExperts + 1];  // grouped: row tiles before each expert
  __shared__ int32_t s_wave[kW4Waves];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_index();
  const int r = lane & 15, q = lane >> 4;
  const int nk = a.K >> 7, ng = (a.N + 15) >> 4;
  const int sets = kW4Waves / a.kw;                 // weight-group sets of the block
  const int kpart = wv % a.kw, set = wv / a.kw;
  const int k0 = nk * kpart / a.kw, k1 = nk * (kpart + 1) / a.kw;
  const int ntn = (ng + RB * sets - 1) / (RB * sets);

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
  }
  const int items = tiles * ntn;

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    int e = 0, tn, row0, rows;
    if (a.offsets == nullptr) {
      // row tiles of one weight set are neighbours: the weights of the second come from L2
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
    const int rg0 = (tn * sets + set) * RB;

    // tokens: rows past the tile's are out of the buffer's range and read as 0
    const uint32_t xrow = static_cast<uint32_t>(a.ldx) * 2;
    const __amdgpu_buffer_rsrc_t xb = make_rsrc(
        static_cast<const uint8_t*>(a.x) + static_cast<size_t>(row0) * xrow,
        static_cast<uint32_t>(rows - 1) * xrow + static_cast<uint32_t>(a.K) * 2);
    uint32_t xoff[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
      xoff[t] = t * 16 + r < rows ? (t * 16 + r) * xrow + (kFold ? q * 64 : q * 16) : kNoRow;
    constexpr uint32_t xj = kFold ? 16 : 64;  // bytes from MFMA j's tokens to j + 1's

    const uint8_t* we = a.w + static_cast<size_t>(e) * ng * nk * kPkBlock + r * 64 + q * 16;
    const size_t gk = static_cast<size_t>(a.K) / G;  // groups of a row

    f32x4_t acc[RB][MT];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[b][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    for (int ks0 = k0; ks0 < k1; ks0 += C) {
      uint4 xf[C][MT][4];
      float xs[C][MT];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            xf[c][t][j] = bld16(xb, xoff[t] + min(ks0 + c, k1 - 1) * 256 + j * xj);
      if constexpr (kInt) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            uint32_t p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              p[j] = __float_as_uint(sum8<DT>(xf[c][t][j]));
              xf[c][t][j] = even_odd(xf[c][t][j]);
            }
            transpose_quads(p);
            xs[c][t] = (__uint_as_float(p[0]) + __uint_as_float(p[1])) +
                       (__uint_as_float(p[2]) + __uint_as_float(p[3]));
          }
      }
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int rg = min(rg0 + b, ng - 1);
        const int n = min(rg * 16 + r, a.N - 1);
        const uint8_t* wp = we + static_cast<size_t>(rg) * nk * kPkBlock;
        const size_t srow = (static_cast<size_t>(e) * a.N + n) * gk;
        uint4 w[C];
        StepScales sc[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int ks = min(ks0 + c, k1 - 1);
          w[c] = ldw16<true>(wp + static_cast<size_t>(ks) * kPkBlock);
          const size_t g0 = srow + static_cast<size_t>(ks) * (128 / G);
          if constexpr (FMT == MOE_W4_MXFP4) {
            sc[c].s[0] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.scales) + g0);
          } else {
            const uint8_t* sp = static_cast<const uint8_t*>(a.scales) + g0 * 2;
            if constexpr (G == 32) {
              sc[c].s[0] = reinterpret_cast<const uint32_t*>(sp)[0];
              sc[c].s[1] = reinterpret_cast<const uint32_t*>(sp)[1];
            } else if constexpr (G == 64) {
              sc[c].s[0] = *reinterpret_cast<const uint32_t*>(sp);
            } else {
              sc[c].s[0] = *reinterpret_cast<const uint16_t*>(sp);
            }
            sc[c].z = 0x08080808u;
            if (a.zeros != nullptr) {
              const uint8_t* zp = a.zeros + g0;
              if constexpr (G == 32) sc[c].z = *reinterpret_cast<const uint32_t*>(zp);
              else if constexpr (G == 64) sc[c].z = *reinterpret_cast<const uint16_t*>(zp);
              else sc[c].z = *zp;
            }
          }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (ks0 + c >= k1) break;
          uint32_t d[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
          if constexpr (kFold) {
            const float s = e8m0_scale_operand((sc[c].s[0] >> (8 * q)) & 0xffu);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 f = __builtin_bit_cast(uint4, decode_fp4x8(d[j], s));
#pragma unroll
              for (int t = 0; t < MT; ++t) acc[b][t] = mfma_rows<DT>(xf[c][t][j], f, acc[b][t]);
            }
          } else {
            constexpr int kPerGroup = G / 32;  // MFMAs a group's sum takes
            float s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int g = j / kPerGroup;
              if constexpr (FMT == MOE_W4_MXFP4) s[j] = e8m0_value((sc[c].s[0] >> (8 * j)) & 0xffu);
              else s[j] = scale16<DT>((sc[c].s[g >> 1] >> (16 * (g & 1))) & 0xffffu);
            }
            transpose_quads(d);
            f32x4_t part[MT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint4 f;
              if constexpr (kInt) f = decode_int4x8<DT>(d[j]);
              else f = decode_fp4x8_f16(d[j]);
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                if (j % kPerGroup == 0) part[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                part[t] = mfma_rows<DT>(xf[c][t][j], f, part[t]);
                if (j % kPerGroup == kPerGroup - 1) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) acc[b][t][i] += s[j] * part[t][i];
                }
              }
            }
            if constexpr (kInt) {
              const float sq = q == 0 ? s[0] : q == 1 ? s[1] : q == 2 ? s[2] : s[3];
              const uint32_t zq = (sc[c].z >> (8 * (q / kPerGroup))) & 0xffu;
              const float sz = -sq * static_cast<float>(zq);
#pragma unroll
              for (int t = 0; t < MT; ++t)
                acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(xs[c][t], sz, acc[b][t], 0, 0, 0);
            }
          }
        }
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
    } else {
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) s_part[wv][b * MT + t][lane] = acc[b][t];
      __syncthreads();
      const int m = tid >> 4, nn = tid & 15;
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          float v = 0.0f;
#pragma unroll
          for (int u = 0; u < kW4Waves; ++u) v += s_part[u][b * MT + t][(m >> 2) * 16 + nn][m & 3];
          store(t * 16 + m, (rg0 + b) * 16 + nn, v);
        }
      __syncthreads();  // before the next item's parts
    }
  }
}

namespace {
template <int FMT, int G, int DT>
hipError_t launch_rows(const W4Args& a, hipStream_t st) {
  // tiles of x rows: by the rows an expert has on average
  const int per = a.offsets != nullptr ? (a.M + a.E - 1) / a.E : a.M;
  const int mt = per <= 16 ? 1 : per <= 32 ? 2 : 4;
  auto go = [&](auto mtc) {
    constexpr int MT = decltype(mtc)::value, RB = MT == 4 ? 2 : 4;
    const int64_t sets = kW4Waves / a.kw;
    const int64_t ntn = ((a.N + 15) / 16 + RB * sets - 1) / (RB * sets);
    const int64_t tiles = (a.M + 16 * MT - 1) / (16 * MT) + (a.offsets != nullptr ? a.E : 0);
    const int64_t items = ntn * tiles;
    const int grid = static_cast<int>(items < 2048 ? items : 2048);
    hipLaunchKernelGGL((w4_kernel<FMT, G, DT, MT, RB>), dim3(grid), dim3(256), 0, st, a);
  };
  if (mt == 1) go(std::integral_constant<int, 1>{});
  else if (mt == 2) go(std::integral_constant<int, 2>{});
  else go(std::integral_constant<int, 4>{});
  return hipGetLastError();
}
template <int DT>
hipError_t launch_format(const W4Args& a, hipStream_t st) {
  if (a.format == MOE_W4_MXFP4) return launch_rows<MOE_W4_MXFP4, 32, DT>(a, st);
  if (a.group == 32) return launch_rows<MOE_W4_INT4, 32, DT>(a, st);
  if (a.group == 64) return launch_rows<MOE_W4_INT4, 64, DT>(a, st);
  return launch_rows<MOE_W4_INT4, 128, DT>(a, st);
}
}  // namespace

hipError_t launch_w4(const W4Args& a0, hipStream_t st) {
  W4Args a = a0;
  // split K over the four waves from 8 steps on; below, each wave has weight rows of its own
  a.kw = a.K >= 8 * 128 ? kW4Waves : 1;
  return a.dtype == MOE_DTYPE_BF16 ? launch_format<MOE_DTYPE_BF16>(a, st)
                                   : launch_format<MOE_DTYPE_FP16>(a, st);
}

}  // namespace moe
