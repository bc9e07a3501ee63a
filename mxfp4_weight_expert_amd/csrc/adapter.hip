// Low-rank adapters of many requests:
//   out[m, n] = base[m, n] + s[i] * sum over r of t[m, r] B[i, n, r],
//   t[m, r]   = sum over k of x[m, k] A[i, r, k],   i the adapter of row m.
// With few rows an adapter memory bounds it: A and B of the adapters that rows
// have, once each, and base and out.
//
// Two launches. The first makes t: a block takes 16 (or 64) sorted rows of one
// adapter and a part of K, so that few rows still spread over the card; the parts
// are summed, in order, by the second, whose blocks take the same rows and a span
// of N. Both read their operands from global memory straight into the 16x16x32
// MFMA (A's or B's rows as its rows, the rows of x as its columns): every element
// is used once by a wave, so LDS would only be a detour.
#include "rows.h"
#include "kernels.h"

#include <algorithm>

namespace moe {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
constexpr int kThreads = 256, kWaves = 4;

template <int DT>
__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
  if constexpr (DT == MOE_DTYPE_BF16)
    return mfma16x16x32(as_bf16x8(a), as_bf16x8(b), c);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                  0, 0, 0);
}

__device__ __forceinline__ uint4 keep(uint4 v, bool in) {
  return in ? v : uint4{0u, 0u, 0u, 0u};
}

// Tile number `tile` of TR sorted rows each, an adapter's tiles after the ones of the
// adapters below: its adapter and rows. Every block counts the tiles of all adapters.
struct AdapterTile {
  int adapter, row0, rows;  // rows 0: no such tile
};
template <int TR>
__device__ __forceinline__ AdapterTile find_tile(const AdapterArgs& a, int tile) {
  constexpr int kPer = kMaxExperts / kThreads;
  __shared__ int s_wave[kWaves];
  __shared__ int s_tile[3];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_index();
  if (tid == 0) s_tile[2] = 0;
  int lo[kPer], hi[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * kThreads + tid;  // adapters below kThreads in one load
    lo[i] = hi[i] = 0;
    if (i * kThreads < a.A && e < a.A) {
      lo[i] = min(max(a.offsets[e], 0), a.M);
      hi[i] = min(a.offsets[e + 1], a.M);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i * kThreads >= a.A) break;
    const int n = hi[i] > lo[i] ? (hi[i] - lo[i] + TR - 1) / TR : 0;
    const int incl = wave_incl_scan(n);
    __syncthreads();
    if (lane == kWave - 1) s_wave[wv] = incl;
    __syncthreads();
    int at = sum + incl - n;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wv) at += s_wave[w];
      sum += s_wave[w];
    }
    if (tile >= at && tile < at + n) {
      s_tile[0] = i * kThreads + tid;
      s_tile[1] = lo[i] + (tile - at) * TR;
      s_tile[2] = min(TR, hi[i] - s_tile[1]);
    }
  }
  __syncthreads();
  return {__builtin_amdgcn_readfirstlane(s_tile[0]), __builtin_amdgcn_readfirstlane(s_tile[1]),
          __builtin_amdgcn_readfirstlane(s_tile[2])};
}

// Row of x of a sorted row, or -1.
__device__ __forceinline__ int row_of(const AdapterArgs& a, int sorted) {
  const int r = a.row_slot[sorted];
  return r >= 0 && r < a.M ? r : -1;
}

// t of a tile's rows over one part of K. RB: 16-row blocks of A. OWN: a wave has 16
// rows of the tile (64 in all) and the whole part; else the waves split the part, and
// join in LDS.
template <int DT, int RB, bool OWN>
__global__ __launch_bounds__(kThreads) void adapter_down_kernel(AdapterArgs a) {
  constexpr int TR = OWN ? 64 : 16;
  constexpr int U = RB >= 4 ? 2 : 4;  // K steps of 32 loaded together
  const AdapterTile t = find_tile<TR>(a, blockIdx.x);
  if (t.rows == 0) return;
  const int lane = lane_id(), wv = wave_index(), c = lane & 15, q = lane >> 4;
  const int nk = (a.K + 31) >> 5, parts = a.splits * (OWN ? 1 : kWaves);
  const int part = blockIdx.y * (OWN ? 1 : kWaves) + (OWN ? 0 : wv);
  const int k0 = static_cast<int>(static_cast<int64_t>(nk) * part / parts);
  const int k1 = static_cast<int>(static_cast<int64_t>(nk) * (part + 1) / parts);
  const int first = OWN ? wv * 16 : 0, rows = min(16, t.rows - first);
  f32x4_t acc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (rows > 0) {
    // lanes of rows that are not there read the tile's first: their columns of the
    // result are not stored, and no column meets another (the same for rows of A)
    const int row = max(row_of(a, t.row0 + first + (c < rows ? c : 0)), 0);
    const uint16_t* const x = static_cast<const uint16_t*>(a.x) + row * a.ldx + q * 8;
    const uint16_t* w[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b)
      w[b] = static_cast<const uint16_t*>(a.a) +
             (static_cast<int64_t>(t.adapter) * a.R + min(b * 16 + c, a.R - 1)) * a.K + q * 8;
    const int whole = min(k1, a.K >> 5);
    int k = k0;
    for (; k + U <= whole; k += U) {
      uint4 xf[U], wf[U][RB];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xf[u] = ld16(x + (k + u) * 32);
#pragma unroll
        for (int b = 0; b < RB; ++b) wf[u][b] = ld16(w[b] + (k + u) * 32);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b] = mfma16<DT>(wf[u][b], xf[u], acc[b]);
    }
    for (; k < k1; ++k) {  // the rest, and pieces of 8 past the end of K
      const bool in = k * 32 + q * 8 < a.K;
      const int at = in ? k * 32 : 0;
      const uint4 xf = keep(ld16(in ? x + at : x - q * 8), in);
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[b] = mfma16<DT>(keep(ld16(in ? w[b] + at : w[b] - q * 8), in), xf, acc[b]);
    }
  }
  // lane (c, q), register v of block b: t[row c, 16 b + 4 q + v]
  float* const out = a.part + (static_cast<int64_t>(blockIdx.y) * a.M + t.row0 + first) * a.R;
  if constexpr (OWN) {
    if (c < rows)
#pragma unroll
      for (int b = 0; b < RB; ++b)
        if (b * 16 + q * 4 < a.R)
          *reinterpret_cast<f32x4_t*>(out + static_cast<int64_t>(c) * a.R + b * 16 + q * 4) = acc[b];
  } else {
    __shared__ f32x4_t s_part[kWaves][RB][kWave];
#pragma unroll
    for (int b = 0; b < RB; ++b) s_part[wv][b][lane] = acc[b];
    __syncthreads();
    for (int b = wv; b < RB; b += kWaves) {
      f32x4_t v = s_part[0][b][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += s_part[w][b][lane];
      if (c < rows && b * 16 + q * 4 < a.R)
        *reinterpret_cast<f32x4_t*>(out + static_cast<int64_t>(c) * a.R + b * 16 + q * 4) = v;
    }
  }
}

// Sixteen elements of a row of base or out, as floats; n of them there.
template <int OT>
__device__ __forceinline__ void load16(const void* p, int n, float (&f)[16]) {
  constexpr int kVec = Row<OT>::kVec;
  const uint8_t* const b = static_cast<const uint8_t*>(p);
  if (n >= 16) {
#pragma unroll
    for (int i = 0; i < 16; i += kVec) Row<OT>::unpack(ld16_any<false>(b + i * Row<OT>::kSize), f + i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = i < n ? Row<OT>::get(b + i * Row<OT>::kSize) : 0.0f;
  }
}
template <int OT>
__device__ __forceinline__ void store16(void* p, int n, const float (&f)[16]) {
  constexpr int kVec = Row<OT>::kVec;
  uint8_t* const b = static_cast<uint8_t*>(p);
  if (n >= 16) {
#pragma unroll
    for (int i = 0; i < 16; i += kVec) st16_any<false>(b + i * Row<OT>::kSize, Row<OT>::pack(f + i));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) Row<OT>::put(b + i * Row<OT>::kSize, f[i]);
  }
}

// out of a tile's rows and a span of N. RS: 32-steps of R; MT: 16-row blocks of the
// tile. t is summed over the parts of K and goes to LDS as two halves, t = hi + lo:
// B is exact in its type, so the products keep t to 2^-16 (bf16) or 2^-22 (fp16)
// at twice the MFMAs, which memory hides. In fp16 a row of t is first divided by a
// power of two that brings its largest value below 2, past neither end of the range.
//
// MFMA j of four on 64 columns takes column 16 (i / 4) + 4 j + i % 4 as its row i, so
// a lane's four results of four MFMAs are sixteen neighbours of a row of out.
template <int DT, int OT, int RS, int MT>
__global__ __launch_bounds__(kThreads) void adapter_up_kernel(AdapterArgs a, int tiles, int span) {
  constexpr int TR = 16 * MT, kPad = 8, kRow = RS * 32 + kPad;  // halves of a row of t in LDS
  constexpr int OS = Row<OT>::kSize;
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_index(), c = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.y * span, n1 = min(a.N, n0 + span);
  uint8_t* const out = static_cast<uint8_t*>(a.out);
  const uint8_t* const base = static_cast<const uint8_t*>(a.base);
  if (static_cast<int>(blockIdx.x) >= tiles) {
    // rows without an adapter, where out is an array of its own
    const int r0 = (blockIdx.x - tiles) * TR;
    for (int r = r0 + wv; r < min(a.M, r0 + TR); r += kWaves) {
      if (a.slot_row[r] >= 0) continue;
      for (int n = n0 + lane * 16; n < n1; n += kWave * 16) {
        float f[16] = {};
        const int left = min(16, n1 - n);
        if (base != nullptr) load16<OT>(base + (r * a.ldb + n) * OS, left, f);
        store16<OT>(out + (r * a.ldo + n) * OS, left, f);
      }
    }
    return;
  }
  __shared__ __attribute__((aligned(16))) uint16_t s_hi[TR * kRow], s_lo[TR * kRow];
  __shared__ float s_scale[TR];
  __shared__ int s_row[TR];
  const AdapterTile t = find_tile<TR>(a, blockIdx.x);
  if (t.rows == 0) return;
  // t: sixteen threads a row, 8 RS / 4 values each
  constexpr int kPer = RS * 2;
  for (int m = tid >> 4; m < TR; m += kThreads / 16) {
    const int r = (tid & 15) * kPer;
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
    if (m < t.rows) {
      const float* p = a.part + static_cast<int64_t>(t.row0 + m) * a.R + r;
      for (int s = 0; s < a.splits; ++s, p += static_cast<int64_t>(a.M) * a.R)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (r + i < a.R) v[i] += p[i];
    }
    float f = a.scale != nullptr ? a.scale[t.adapter] : 1.0f;
    if constexpr (DT == MOE_DTYPE_FP16) {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) most = fmaxf(most, fabsf(v[i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor(most, o, 16));
      // infinities and NaN stay what they are
      const int e = most > 0.0f && most < __builtin_inff() ? ilogbf(most) : 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = ldexpf(v[i], -e);
      f = ldexpf(f, e);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float hi;
      if constexpr (DT == MOE_DTYPE_BF16) {
        const uint16_t h = f32_to_bf16(v[i]);
        hi = bf16_to_f32(h);
        s_hi[m * kRow + r + i] = h;
      } else {
        const _Float16 h = static_cast<_Float16>(v[i]);
        hi = static_cast<float>(h);
        s_hi[m * kRow + r + i] = __builtin_bit_cast(uint16_t, h);
      }
      const float lo = fabsf(hi) < __builtin_inff() ? v[i] - hi : 0.0f;  // nothing beside an infinity or NaN
      if constexpr (DT == MOE_DTYPE_BF16) s_lo[m * kRow + r + i] = f32_to_bf16(lo);
      else s_lo[m * kRow + r + i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(lo));
    }
    if ((tid & 15) == 0) {
      s_scale[m] = f;
      s_row[m] = m < t.rows ? row_of(a, t.row0 + m) : -1;
    }
  }
  __syncthreads();
  int row[MT];
  float scale[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    row[m] = s_row[m * 16 + c];
    scale[m] = s_scale[m * 16 + c];
  }
  const uint16_t* const b = static_cast<const uint16_t*>(a.b) + static_cast<int64_t>(t.adapter) * a.N * a.R;
  for (int n = n0 + wv * 64; n < n1; n += kWaves * 64) {
    uint4 w[4][RS];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = min(n + 16 * (c >> 2) + 4 * j + (c & 3), a.N - 1);
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const int r = s * 32 + q * 8;
        w[j][s] = keep(ld16(b + static_cast<int64_t>(at) * a.R + (r < a.R ? r : 0)), r < a.R);
      }
    }
    const int col = n + q * 16, left = min(16, n1 - col);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m * 16 >= t.rows) break;
      float f[16] = {};
      const bool in = row[m] >= 0 && left > 0;
      if (in && base != nullptr) load16<OT>(base + (row[m] * a.ldb + col) * OS, left, f);
      f32x4_t acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const int at = (m * 16 + c) * kRow + s * 32 + q * 8;
        const uint4 hi = *reinterpret_cast<const uint4*>(s_hi + at), lo = *reinterpret_cast<const uint4*>(s_lo + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = mfma16<DT>(w[j][s], hi, mfma16<DT>(w[j][s], lo, acc[j]));
      }
      if (!in) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) f[4 * j + v] += scale[m] * acc[j][v];
      store16<OT>(out + (row[m] * a.ldo + col) * OS, left, f);
    }
  }
}

// Rows of an adapter that a tile takes: 64 where M / A says many. Tiles there are at
// most one for each row, and one for each adapter beside the full ones.
bool many_rows(int64_t M, int64_t A) { return M >= 32 * A; }
int64_t tile_bound(const AdapterArgs& a) {
  const int tr = many_rows(a.M, a.A) ? 64 : 16;
  return std::min<int64_t>(a.M, a.M / tr + a.A);
}

template <int DT, int RB>
void down(const AdapterArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(tile_bound(a)), static_cast<unsigned>(a.splits));
  if (many_rows(a.M, a.A))
    hipLaunchKernelGGL((adapter_down_kernel<DT, RB, true>), grid, dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((adapter_down_kernel<DT, RB, false>), grid, dim3(kThreads), 0, st, a);
}

template <int DT, int OT, int RS>
void up(const AdapterArgs& a, hipStream_t st) {
  const bool many = many_rows(a.M, a.A);
  const int tr = many ? 64 : 16;
  const int64_t tiles = tile_bound(a);
  // rows without an adapter need a copy only where out is not base
  const int64_t others = a.out == a.base ? 0 : (a.M + tr - 1) / tr;
  const int64_t n64 = (a.N + 63) / 64;
  // spans of N: enough blocks for the card, each with at least one piece a wave
  const int64_t want = std::max<int64_t>(1, 2048 / std::max<int64_t>(tiles, 1));
  const int64_t per = std::max<int64_t>(kWaves, (n64 + want - 1) / want);
  const int span = static_cast<int>((per + kWaves - 1) / kWaves * kWaves * 64);
  const dim3 grid(static_cast<unsigned>(tiles + others), static_cast<unsigned>((a.N + span - 1) / span));
  if (many)
    hipLaunchKernelGGL((adapter_up_kernel<DT, OT, RS, 4>), grid, dim3(kThreads), 0, st, a, static_cast<int>(tiles), span);
  else
    hipLaunchKernelGGL((adapter_up_kernel<DT, OT, RS, 1>), grid, dim3(kThreads), 0, st, a, static_cast<int>(tiles), span);
}

template <int DT, int OT>
void up_rank(const AdapterArgs& a, hipStream_t st) {
  if (a.R <= 32) up<DT, OT, 1>(a, st);
  else if (a.R <= 64) up<DT, OT, 2>(a, st);
  else up<DT, OT, 4>(a, st);
}

template <int DT>
void both(const AdapterArgs& a, hipStream_t st) {
  if (a.R <= 16) down<DT, 1>(a, st);
  else if (a.R <= 32) down<DT, 2>(a, st);
  else if (a.R <= 64) down<DT, 4>(a, st);
  else down<DT, 8>(a, st);
  if (a.out_dtype == MOE_DTYPE_FP32) up_rank<DT, MOE_DTYPE_FP32>(a, st);
  else up_rank<DT, DT>(a, st);
}

}  // namespace

int adapter_splits(int64_t M, int64_t A, int64_t K) {
  const bool many = many_rows(M, A);
  const int64_t tiles = std::max<int64_t>(1, std::min<int64_t>(M, M / (many ? 64 : 16) + std::min(A, M)));
  const int64_t steps = (K + 31) / 32 / (many ? 1 : kWaves);  // a wave's, unsplit
  const int64_t by_card = (many ? 1024 : 512) / tiles, by_steps = steps / 4;
  return static_cast<int>(std::clamp<int64_t>(std::min(by_card, by_steps), 1, 16));
}

hipError_t launch_adapter(const AdapterArgs& a, hipStream_t st) {
  if (a.dtype == MOE_DTYPE_BF16) both<MOE_DTYPE_BF16>(a, st);
  else both<MOE_DTYPE_FP16>(a, st);
  return hipGetLastError();
}

}  // namespace moe
