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
// of x over the group, by 16x16x4 float MFMAs: exact codes and one correction in
// 32 bits.
#pragma once

#include "rows.h"
#include "kernels.h"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace moe {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_byte __attribute__((ext_vector_type(4), aligned(1)));

// 16-byte buffer load of weights, non-temporal (cache-policy operand 2) where
// they are read once: 64-token decode of 896 experts 143 us against 164 with
// plain loads. Where several row tiles read them (64 experts of 32 rows) plain
// loads take 121 us, these 131; a branch around the two kinds of load costs the
// first case 6 % (its waits then cover both), so the walk is an instance of each.
template <bool ONCE>
__device__ __forceinline__ uint4 bld16_once(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, ONCE ? 2 : 0));
}

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
// The 16-byte piece (0..15) of a step's 256 bytes of a token row that quad q
// feeds to MFMA j.
template <int L>
__device__ __forceinline__ constexpr uint32_t token_piece(uint32_t q, uint32_t j) {
  return L == kMix ? q * 4 + j
                   : L == kHalf ? (q & 1) * 4 + (q >> 1) * 2 + (j & 1) + (j >> 1) * 8 : q + j * 4;
}

// K steps that a wave has in flight: 1 KB for each weight group and each four
// rows of x. Three instead of two cost registers and gained nothing (64-token
// decode of 896 experts: 145 against 143 us).
constexpr int w4_depth(int mt) { return mt == 4 ? 1 : 2; }

// The block copies `bytes` (a multiple of ALIGN) of global memory to LDS:
// 16-byte pieces, then the last bytes one ALIGN unit a thread.
template <int ALIGN, int W>
__device__ __forceinline__ void block_to_lds(uint8_t* lds, const uint8_t* src, int bytes) {
  const int n = bytes >> 4, tid = threadIdx.x;
  for (int c = tid; c < n; c += 64 * W)
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

// LDS: for each wave the token tile of a step (its parts of the sums at the
// end), then the scale rows and the zero points of the block's weight rows.
template <int MT, int W>
__host__ __device__ constexpr int w4_token_bytes() { return W * MT * 4096; }

// The same value, but not known to be: addresses made from it are worked out
// where they are used. Hoisted out of the task loop, those of every unrolled
// step, LDS read and store would hold some 70 registers a lane throughout.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// FMT, G: weight format and group; DT: tokens' type; MT: 16-row tiles of x a
// task takes; RB: 16-row weight groups a wave takes.
//
// A task is a row tile times RB (kw = W) or W RB (kw = 1) weight groups. With
// kw = W the block's waves split K and join in LDS at the end; with kw = 1 each
// has weight groups of its own. A wave walks its K steps with a ring of
// w4_depth steps in flight, tokens and weights; loads past its last step are
// out of their buffer's range and touch no memory, so every step issues the
// same loads and the waits cover the step being used alone. The scales of the
// block's weight rows lie one after another and come to LDS in one copy.
//
// What it costs beside the weights' stream, by leaving it out (64-token decode
// of 896 experts, N 768, K 3584, when tokens came straight to the MFMA operands
// with four loads a step): tokens 17 of 150 us, scales 8, decode and MFMAs
// none; weights alone stream at 7.1 TB/s. Tokens loaded a KB at a time and
// passed through LDS took 151 to 142 us.
template <int FMT, int G, int DT, int MT, int RB, int W>
__global__ __launch_bounds__(64 * W, MT == 1 && W == 4 ? 3 : 2) void w4_kernel(W4Args a) {
  constexpr int L = w4_layout(FMT, G, DT);
  constexpr bool kInt = FMT == MOE_W4_INT4;
  constexpr bool kFold = FMT == MOE_W4_MXFP4 && DT == MOE_DTYPE_BF16;  // scale in the convert
  constexpr int D = w4_depth(MT);
  constexpr int kTile = 16 * MT;
  constexpr int kGroups = 128 / G;                   // groups of a step
  constexpr int kScale = kInt ? 2 : 1;               // bytes of a scale
  extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];
  __shared__ int32_t s_first[kMaxExperts + 1];  // grouped: row tiles before each expert
  __shared__ int32_t s_wave[W];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_index();
  const int nk = a.K >> 7, ng = (a.N + 15) >> 4;
  const int sets = W / a.kw;  // sets of weight groups in the block
  const int kpart = wv % a.kw, set = wv / a.kw;
  const int k0 = nk * kpart / a.kw, nsteps = nk * (kpart + 1) / a.kw - k0;
  const int ntn = (ng + RB * sets - 1) / (RB * sets);
  const int srow = nk * kGroups * kScale, zrow = nk * kGroups;  // bytes of a weight row's
  uint8_t* const s_scale = s_dyn + w4_token_bytes<MT, W>();
  uint8_t* const s_zero = s_scale + ((RB * sets * 16 * srow + 15) & ~15);

  int tiles = (a.M + kTile - 1) / kTile;
  if (a.offsets != nullptr) {
    constexpr int kPer = kMaxExperts / (64 * W);
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
    for (int i = 0; i < W; ++i) {
      if (i < wv) at += s_wave[i];
      tiles += s_wave[i];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s_first[tid * kPer + i] = at;
      at += c[i];
    }
    if (tid == 64 * W - 1) s_first[kMaxExperts] = at;
    __syncthreads();
    tiles = __builtin_amdgcn_readfirstlane(tiles);
  }
  // the launcher's bound, which offsets that decrease could pass: the loop below
  // must end without its index wrapping
  const int items = static_cast<int>(min(static_cast<int64_t>(tiles) * ntn, kW4MaxItems));

  const uint32_t xrow = static_cast<uint32_t>(a.ldx) * 2;
  const uint32_t gbytes = static_cast<uint32_t>(nk) * kPkBlock;  // a weight group's
  uint8_t* const s_tok = s_dyn + wv * MT * 4096;  // this wave's token tile

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    int e = 0, tn, row0, rows;
    bool once = tiles == 1;  // the weights are read by this task alone: past the caches
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
      const int first = s_first[e], te = __builtin_amdgcn_readfirstlane(s_first[e + 1] - first);
      once = te == 1;
      const int local = item - first * ntn;
      tn = local / te;
      const int m = local - tn * te;
      const int r0 = min(max(a.offsets[e], 0), a.M), r1 = min(a.offsets[e + 1], a.M);
      row0 = r0 + m * kTile;
      rows = min(kTile, r1 - row0);
    }
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);
    const int bg0 = __builtin_amdgcn_readfirstlane(tn) * RB * sets;  // the block's first weight group
    const int rg0 = bg0 + set * RB;                                  // the wave's

    // The scales of the block's weight rows, in one contiguous copy. Every wave
    // has passed the last task's barrier, and so has read the last of its scales.
    {
      const size_t row = static_cast<size_t>(e) * a.N + bg0 * 16;
      const int nrow = min(RB * sets * 16, a.N - bg0 * 16);
      block_to_lds<kInt ? 2 : 4, W>(s_scale, static_cast<const uint8_t*>(a.scales) + row * srow, nrow * srow);
      if (kInt && a.zeros != nullptr) block_to_lds<1, W>(s_zero, a.zeros + row * zrow, nrow * zrow);
    }

    // Rows past the tile's and weight groups past the last are out of the
    // buffers' range: loads of them return 0 and touch no memory.
    const __amdgpu_buffer_rsrc_t xb = make_rsrc(
        static_cast<const uint8_t*>(a.x) + static_cast<size_t>(row0) * xrow,
        static_cast<uint32_t>(rows - 1) * xrow + static_cast<uint32_t>(a.K) * 2);
    const int live = min(RB, ng - rg0);
    const __amdgpu_buffer_rsrc_t wb = make_rsrc(
        a.w + (static_cast<size_t>(e) * ng + rg0) * gbytes, live > 0 ? live * gbytes : 0);

    f32x4_t acc[RB][MT];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[b][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // The wave's K steps. XL: 1 KB loads of tokens a step, four rows each; TT:
    // 16-row tiles that hold rows (an expert may have fewer than MT).
    auto walk = [&](auto xlc, auto oncec) {
      constexpr int XL = decltype(xlc)::value, TT = XL <= 4 ? 1 : XL / 4;
      constexpr bool ONCE = decltype(oncec)::value;
      const int ln = opaque(lane), r = ln & 15, q = ln >> 4;
      const uint32_t woff = k0 * kPkBlock + r * 64 + q * 16;
      uint4 xg[D][XL], w[D][RB];
      uint32_t xoff[XL], xlds[XL];
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        const uint32_t row = 4 * i + q;  // piece r of row 4 i + q
        xoff[i] = row < static_cast<uint32_t>(rows) ? row * xrow + k0 * 256 + r * 16 : kNoRow;
        xlds[i] = row * 256 + ((r ^ row) & 15) * 16;
      }
      // The blocks of an XCD take a row tile's steps from different places on:
      // in step, all of them would ask one L2 channel for the same tokens, whose
      // rows are often a multiple of the channels' span apart. The place goes by matrix
      // and weight rows alone, so the order of a row's sums has nothing to do with where
      // in the batch it lies.
      const int turn = (((e * ntn + tn) >> 3) + kpart * (nsteps >> 2)) % max(nsteps, 1);
      auto place = [&](int step) { return step + turn < nsteps ? step + turn : step + turn - nsteps; };
      auto load = [&](int d, int step) {  // step: wave-uniform
        const bool in = step < nsteps;
        const int at = place(step);
#pragma unroll
        for (int i = 0; i < XL; ++i) xg[d][i] = bld16(xb, in ? xoff[i] + at * 256 : kNoRow);
#pragma unroll
        for (int b = 0; b < RB; ++b)
          w[d][b] = bld16_once<ONCE>(wb, in ? woff + b * gbytes + at * kPkBlock : kNoRow);
      };
#pragma unroll
      for (int d = 0; d < D; ++d) load(d, d);
      __syncthreads();  // scales are in LDS

      // INT4, lane (m, q): its share of the sums of row m's tokens that the zero
      // points meet, and the place of the scale and zero point of weight row n = m.
      // Groups of 64 and 128 leave half of the correction's four places free: it
      // takes two steps at once (kPair), the first in lanes q < 2 (64 of 256 experts,
      // K 7168, N 4096, groups of 64: 188 us step by step, 179 so).
      constexpr bool kPair = kInt && G >= 64 && D == 2;
      float xs[TT];
      int zplace = 0;
      auto compute = [&](int d, int ks, bool last) {
        // Tokens through the wave's own LDS tile: loaded whole rows a KB at a
        // time, read as the MFMAs want them. Piece c of row m lies at c ^ m, so
        // the sixteen rows' pieces fall on different banks. Lanes of rows that
        // were not loaded read one that was: their results are not stored. INT4:
        // the tokens in the order of the decoded codes.
#pragma unroll
        for (int i = 0; i < XL; ++i)
          *reinterpret_cast<uint4*>(s_tok + xlds[i]) = kInt ? even_odd(xg[d][i]) : xg[d][i];
        __builtin_amdgcn_wave_barrier();
        uint4 xf[TT][4];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint32_t m = XL < 4 ? r & (4 * XL - 1) : t * 16 + r;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            xf[t][j] = *reinterpret_cast<const uint4*>(
                s_tok + m * 256 + ((token_piece<L>(q, j) ^ m) & 15) * 16);
          if constexpr (kInt) {
            // MFMAs with ones for weights: every lane (m, q) gets row m's sum of
            // each group, and keeps its share of the one that its scales belong to
            const uint32_t one = DT == MOE_DTYPE_BF16 ? 0x3f803f80u : 0x3c003c00u;
            constexpr int kPer = 4 / kGroups;
            f32x4_t sum[kGroups];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j % kPer == 0) sum[j / kPer] = f32x4_t{0.f, 0.f, 0.f, 0.f};
              sum[j / kPer] = mfma_rows<DT>(uint4{one, one, one, one}, xf[t][j], sum[j / kPer]);
            }
            if constexpr (kPair) {
              const float own = G == 64 ? (q & 1 ? sum[kGroups - 1][0] : sum[0][0]) : 0.5f * sum[0][0];
              xs[t] = d == 0 ? (q < 2 ? own : 0.0f) : (q < 2 ? xs[t] : own);
            } else {
              xs[t] = sum[0][0];
#pragma unroll
              for (int g = 1; g < kGroups; ++g) xs[t] = q / kPer == g ? sum[g][0] : xs[t];
              xs[t] *= 1.0f / kPer;  // the group's kPer lanes add up to it
            }
          }
        }
        __builtin_amdgcn_wave_barrier();
        if constexpr (kPair) {
          const int here = ks * kGroups + (G == 64 ? q & 1 : 0);
          zplace = d == 0 || q >= 2 ? here : zplace;
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
              for (int t = 0; t < TT; ++t) acc[b][t] = mfma_rows<DT>(xf[t][j], f, acc[b][t]);
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
            f32x4_t part[TT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint4 f;
              if constexpr (kInt) f = decode_int4x8<DT>(dw[j]);
              else f = decode_fp4x8_f16(dw[j]);
#pragma unroll
              for (int t = 0; t < TT; ++t) {
                if (j % kPer == 0) part[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                part[t] = mfma_rows<DT>(xf[t][j], f, part[t]);
                if (j % kPer == kPer - 1) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) acc[b][t][i] += s[j / kPer] * part[t][i];
                }
              }
            }
            if constexpr (kPair) {
              if (d == 1 || last) {
                const float sz = scale16<DT>(*reinterpret_cast<const uint16_t*>(s_scale + wr * srow + 2 * zplace)) *
                                 (a.zeros != nullptr ? static_cast<float>(s_zero[wr * zrow + zplace]) : 8.0f);
#pragma unroll
                for (int t = 0; t < TT; ++t)
                  acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(xs[t], -sz, acc[b][t], 0, 0, 0);
              }
            } else if constexpr (kInt) {
              const int gq = q / kPer;
              float z = 8.0f, sq = s[0];
              if (a.zeros != nullptr) z = static_cast<float>(s_zero[wr * zrow + ks * kGroups + gq]);
#pragma unroll
              for (int g = 1; g < kGroups; ++g) sq = gq == g ? s[g] : sq;
#pragma unroll
              for (int t = 0; t < TT; ++t)
                acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(xs[t], -sq * z, acc[b][t], 0, 0, 0);
            }
          }
          __builtin_amdgcn_sched_barrier(0);  // one weight group's decode at a time: registers
        }
      };
      for (int s0 = 0; s0 < nsteps; s0 += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          if (s0 + d < nsteps) compute(d, k0 + place(s0 + d), s0 + d + 1 >= nsteps);
          __builtin_amdgcn_sched_barrier(0);
          load(d, s0 + d + D);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    const auto by_rows = [&](auto oncec) {
      if (rows <= 4) walk(std::integral_constant<int, 1>{}, oncec);
      else if (rows <= 8) walk(std::integral_constant<int, 2>{}, oncec);
      else if (MT == 1 || rows <= 16) walk(std::integral_constant<int, 4>{}, oncec);
      else if (rows <= 32) walk(std::integral_constant<int, 4 * std::min(MT, 2)>{}, oncec);
      else walk(std::integral_constant<int, 4 * MT>{}, oncec);
    };
    if constexpr (MT == 2) walk(std::integral_constant<int, 8>{}, std::true_type{});  // 17 to 32 rows in all
    else if (once) by_rows(std::true_type{});
    else by_rows(std::false_type{});

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
      const int ln = opaque(lane), r = ln & 15, q = ln >> 4;
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) store(t * 16 + q * 4 + i, (rg0 + b) * 16 + r, acc[b][t][i]);
      __syncthreads();  // before the next task's scales
    } else {
      // in place of the wave's tokens: [RB * MT][lane] of MT * 256 places
      static_assert(RB <= 4, "a wave's sums fit its token tile");
      f32x4_t* part = reinterpret_cast<f32x4_t*>(s_dyn);
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t) part[(wv * 4 * MT + b * MT + t) * kWave + opaque(lane)] = acc[b][t];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < RB * MT * 256; i += 64 * W) {
        const int at = i + opaque(tid), bt = at >> 8, m = (at >> 4) & 15, nn = at & 15;
        if (RB * MT * 256 % (64 * W) != 0 && at >= RB * MT * 256) break;
        float v = 0.0f;
#pragma unroll
        for (int u = 0; u < W; ++u)
          v += reinterpret_cast<const float*>(
              part + (u * 4 * MT + bt) * kWave + (m >> 2) * 16 + nn)[m & 3];
        store(bt % MT * 16 + m, (rg0 + bt / MT) * 16 + nn, v);
      }
    }
  }
}

// CUs of the current GPU and blocks of a kernel that one of them holds, by the
// block's LDS; blocks 0 where the runtime does not say. Kept for each kernel, GPU and
// KB of LDS: asking takes longer than a small launch. The kernel is the template's
// argument itself: instances have one type between them, and would share what is kept
// for a type.
struct W4Room {
  int cus, blocks;
};
template <auto Kernel>
W4Room w4_room(int threads, int lds) {
  constexpr int kGpus = 16;
  static std::atomic<int> kept[kGpus][161];  // cus << 8 | blocks
  int gpu = 0, blocks = 0, cus = 0;
  if (hipGetDevice(&gpu) == hipSuccess) {
    std::atomic<int>* const k = gpu < kGpus ? &kept[gpu][lds >> 10] : nullptr;
    const int v = k != nullptr ? k->load(std::memory_order_relaxed) : 0;
    if (v > 0) return {v >> 8, v & 255};
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, reinterpret_cast<const void*>(Kernel), threads,
                                                     (lds | 1023) + 1) == hipSuccess &&
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, gpu) == hipSuccess &&
        blocks > 0 && cus > 0) {
      if (k != nullptr) k->store(cus << 8 | blocks, std::memory_order_relaxed);
      return {cus, blocks};
    }
  }
  (void)hipGetLastError();  // a query's error is not the launch's
  return {256, 0};
}

// LDS of a block that splits K over kw waves, without the kernel's static tables.
template <int FMT, int G, int MT, int RB, int W>
int w4_lds(const W4Args& a, int kw) {
  constexpr bool kInt = FMT == MOE_W4_INT4;
  const int groups = (a.K >> 7) * (128 / G), nrow = RB * (W / kw) * 16;
  return w4_token_bytes<MT, W>() + ((nrow * groups * (kInt ? 2 : 1) + 15) & ~15) +
         (kInt && a.zeros != nullptr ? (nrow * groups + 15) & ~15 : 0);
}
constexpr int kW4MostLds = 150 << 10;   // of a CU's 160 KB, with room for the static tables
constexpr int kW4WholeLds = 52 << 10;   // kw = 1 with 16-row tiles: 16 KB of tokens, 36 of scales

// U: the 16-row weight groups that can be read (kw: see w4_rows).
template <int FMT, int G, int DT, int MT, int RB, int W>
void w4_go(const W4Args& a0, int64_t U, hipStream_t st) {
  constexpr auto kernel = w4_kernel<FMT, G, DT, MT, RB, W>;
  [[maybe_unused]] constexpr bool kInt = FMT == MOE_W4_INT4;
  W4Args a = a0;
  a.kw = W;
  int lds = w4_lds<FMT, G, MT, RB, W>(a, W);
  W4Room room = w4_room<kernel>(64 * W, lds);
  if (W == 4 && U >= 2048) {
    const int lds1 = w4_lds<FMT, G, MT, RB, W>(a, 1), nk = a.K >> 7;
    bool whole = false;
    if constexpr (MT == 1) {
      const int64_t blocks = int64_t{room.cus} * std::max(room.blocks, 1);
      const auto cost = [&](int64_t tasks, int steps) { return (tasks + blocks - 1) / blocks * (steps + 4); };
      whole = lds1 <= kW4WholeLds && cost(U / (W * RB), nk) <= cost(U / RB, (nk + W - 1) / W);
    } else if (lds1 <= kW4MostLds) {
      const int64_t m = a.offsets != nullptr ? a.M / a.E : a.M, tiles = (m + 16 * MT - 1) / (16 * MT);
      const auto cost = [&](int64_t tasks, int steps, int blocks) {
        const int64_t each = (tasks + room.cus - 1) / room.cus;
        return each * (2 * steps + (MT == 2 ? 5 : 4)) * (each > 1 && blocks > 1 ? 6 : kInt ? 10 : 8);
      };
      whole = cost(U * tiles / (W * RB), nk, w4_room<kernel>(64 * W, lds1).blocks) <
              cost(U * tiles / RB, (nk + W - 1) / W, room.blocks);
    }
    if (whole) {
      a.kw = 1;
      lds = lds1;
      room = w4_room<kernel>(64 * W, lds);
    }
  }
  const int64_t sets = W / a.kw;
  const int64_t ntn = ((a.N + 15) / 16 + RB * sets - 1) / (RB * sets);
  const int64_t tiles = (a.M + 16 * MT - 1) / (16 * MT) + (a.offsets != nullptr ? a.E : 0);
  const int64_t items = ntn * tiles;
  // as many blocks as are resident, each with tasks in turn: twice to sixteen times
  // as many were 0 to 14 % slower with experts and no faster with one matrix, and
  // only as many as share the tasks evenly 4 to 8 % slower
  const int64_t most = int64_t{room.cus} * std::max(room.blocks, 1);
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(items < most ? items : most)), dim3(64 * W), lds,
                     st, a);
}

// The variant of a shape. U is the number of 16-row weight groups that can be
// read (an expert without rows reads none), nk the K steps.
//
// - Many groups (U >= 2048): RB = 4 with 16-row tiles, whose loads of tokens serve
//   four groups, 2 with 32 and 64 rows. kw = 1 reads a group's whole K in one wave,
//   with no join, but takes tasks four times as long, and four times the scales in
//   LDS. It is chosen where its estimate is not the higher one:
//   16-row tiles (the weights' stream bounds them): rounds of resident blocks (three a
//   CU) times (steps + 4), the 4 for a task's start and end. K 384 x N 3584 of 896
//   experts: 97 us against 205 with kw = 4; K 7168 x N 4096 of 64 experts: 176 against
//   157. Up to 30 KB of scales a block leave room for three with kw = 1 too; from there
//   to the limit of 36 two fit, which costs MXFP4 little (K 4096: N 2816 of 60 experts
//   137 against 138, N 768 of 448 138 against 128) and INT4 nothing (groups of 64 with
//   zero points, K 2560: N 768 of 896 experts 173 against 197).
//   32 and 64 rows (decode, MFMAs and LDS bound them, so what the busiest CU has to do
//   counts): tasks a CU times (steps + 2.5 or 2), and where a CU has one block at a
//   time, which leaves its waits open, a third more with MXFP4, two with INT4.
//   N 129279, 64 rows: K 1024 48 us with kw = 1, 72 with 4; INT4 of 64 with zero
//   points at K 2048 149 and 126, at K 4096 262 and 204, since kw = 1 leaves room for
//   one block; N 65536, K 4096, 32 rows 47 and 51; 16 experts of 256 rows, K 3584,
//   N 4096 352 and 312.
// - Fewer: RB = 2, or 1 up to a group a CU, and K over eight waves from 16 steps on.
//   8192 x 8192, 1 and 16 tokens: 9.3 and 12.3 us with RB = 2 and eight waves, 9.7
//   and 15.3 with RB = 1, 13.4 and 15.6 with RB = 4 and four waves. 4096 x 4096:
//   5.6 and 7.2, 4.8 and 6.1, 8.4 and 9.7. 24576 x 2048, one token: 7.2 with RB = 2
//   and four waves, 8.8 with RB = 4.
// Row tiles of x a task takes (MT): 16 rows, whose tiles read their weights again
// from the caches, or 32 (up to 32 rows of one matrix) or 64, which share a decode.
// N 32768, K 4096, MXFP4, 32 and 64 rows: 26 and 42 us so, 27 and 45 in tiles of
// 16; INT4 of 64 32 and 55, 31 and 55. INT4 of 32 runs out of registers with 64
// rows (82 us against 75). The rows of an expert are not known here, only M / E,
// which counts those that live elsewhere too, so experts take tiles of 16 until
// M / E says many: K 2048 x N 4096, a quarter of 256 experts, M / E = 64 with 16
// rows each, 77 us in tiles of 16, 122 in tiles of 64; 16 experts of 256 rows
// (K 3584, N 768) 85 and 71.
template <int FMT, int G, int DT>
void w4_rows(const W4Args& a, hipStream_t st) {
  constexpr bool kWide = !(FMT == MOE_W4_INT4 && G == 32);
  const bool grouped = a.offsets != nullptr;
  int mt = grouped ? (a.M / a.E > 128 ? 4 : 1) : a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
  if (mt == 4 && !kWide) mt = 1;
  const int64_t U = static_cast<int64_t>((a.N + 15) / 16) * (grouped ? std::min(a.E, a.M) : 1);
  const int nk = a.K >> 7;
  if (mt == 4) {
    if constexpr (kWide) {
      if (U >= 512) w4_go<FMT, G, DT, 4, 2, 4>(a, U, st);
      else w4_go<FMT, G, DT, 4, 1, 4>(a, U, st);
    }
  } else if (mt == 2) {
    if (U >= 512) w4_go<FMT, G, DT, 2, 2, 4>(a, U, st);
    else w4_go<FMT, G, DT, 2, 1, 4>(a, U, st);
  } else if (U >= 2048) {
    w4_go<FMT, G, DT, 1, 4, 4>(a, U, st);
  } else if (U > 512 || nk < 16) {
    if (U > 256) w4_go<FMT, G, DT, 1, 2, 4>(a, U, st);
    else w4_go<FMT, G, DT, 1, 1, 4>(a, U, st);
  } else {
    if (U > 256) w4_go<FMT, G, DT, 1, 2, 8>(a, U, st);
    else w4_go<FMT, G, DT, 1, 1, 8>(a, U, st);
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
