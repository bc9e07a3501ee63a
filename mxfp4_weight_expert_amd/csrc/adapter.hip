// Low-rank adapters of many requests:
//   out[m, n] = base[m, n] + s[i] * sum over r of t[m, r] B[i, n, r],
//   t[m, r]   = sum over k of x[m, k] A[i, r, k],   i the adapter of row m.
// With few rows an adapter memory bounds it: A and B of the adapters that rows
// have, once each, and base and out; a handful of rows the two launches one after the
// other (1 row, rank 16, K 7168, N 2048: 4.3 and 4.7 us). 8191 rows, 8 adapters of rank
// 64, K 3584, N 7168: 27 us and 77, where x alone takes 12 at the rate of a large copy and
// base and out 48 (191 MB read, 118 written). Spans of N by XCD, so that each reads its part
// of B alone, and non-temporal base and out gained nothing or lost (108 us, 116).
//
// Two launches. The first makes t: a block takes 16 (or 32) sorted rows of one
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
// adapters below: its adapter and rows. Every wave counts the tiles of all adapters up to
// it, 256 at a time.
struct AdapterTile {
  int adapter, row0, rows;  // rows 0: no such tile
};
template <int TR>
__device__ __forceinline__ AdapterTile find_tile(const AdapterArgs& a, int tile) {
  const int lane = lane_id();
  int below = 0;  // tiles of the adapters looked at
  for (int e0 = 0; e0 < a.A; e0 += 4 * kWave) {
    int lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + i * kWave + lane;
      lo[i] = a.offsets[min(e, a.A)];
      hi[i] = a.offsets[min(e + 1, a.A)];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int first = min(max(lo[i], 0), a.M), last = min(hi[i], a.M);
      const int n = last > first ? (last - first + TR - 1) / TR : 0, at = below + wave_incl_scan(n) - n;
      const uint64_t mine = ballot(tile >= at && tile < at + n);
      if (mine != 0) {
        const int l = __builtin_ctzll(mine);
        const int row0 = __builtin_amdgcn_readlane(first + (tile - at) * TR, l);
        return {e0 + i * kWave + l, row0, min(TR, __builtin_amdgcn_readlane(last, l) - row0)};
      }
      below = __builtin_amdgcn_readlane(at + n, kWave - 1);
    }
  }
  return {0, 0, 0};
}

// Row of x of a sorted row, or -1.
__device__ __forceinline__ int row_of(const AdapterArgs& a, int sorted) {
  const int r = a.row_slot[sorted];
  return r >= 0 && r < a.M ? r : -1;
}

// t of a tile's rows over one part of K, which the four waves split again and join in
// LDS. RB, MT: 16-row blocks of A and of the tile.
template <int DT, int RB, int MT>
__global__ __launch_bounds__(kThreads, RB * MT >= 16 ? 2 : 4) void adapter_down_kernel(AdapterArgs a) {
  constexpr int D = RB + MT <= 2 ? 4 : RB + MT <= 5 ? 2 : 1;  // steps of 64 of K in flight
  const AdapterTile t = find_tile<16 * MT>(a, blockIdx.x);
  if (t.rows == 0) return;
  const int lane = lane_id(), wv = wave_index(), c = lane & 15, q = lane >> 4;
  const int nk = (a.K + 63) >> 6, parts = a.splits * kWaves, part = blockIdx.y * kWaves + wv;
  const int k0 = static_cast<int>(static_cast<int64_t>(nk) * part / parts);
  const int nsteps = static_cast<int>(static_cast<int64_t>(nk) * (part + 1) / parts) - k0;
  // lanes of rows that are not there read the tile's first: their columns of the result
  // are not stored, and no column meets another
  const uint16_t* x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = m * 16 + c;
    x[m] = static_cast<const uint16_t*>(a.x) + max(row_of(a, t.row0 + (r < t.rows ? r : 0)), 0) * a.ldx;
  }
  const __amdgpu_buffer_rsrc_t wb = make_rsrc(
      static_cast<const uint16_t*>(a.a) + static_cast<int64_t>(t.adapter) * a.R * a.K, kNoRow);
  uint32_t woff[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) woff[b] = b * 16 + c < a.R ? (b * 16 + c) * static_cast<uint32_t>(a.K) * 2 : kNoRow;
  f32x4_t acc[RB][MT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[b][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint4 xf[D][MT][2], wf[D][RB][2];
  auto load = [&](int d, int step) {  // both halves of a row's 128 bytes together
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = (k0 + min(step, nsteps - 1)) * 64 + j * 32 + q * 8;
      const bool in = k < a.K;  // pieces past the end of K count as zeros on both sides
#pragma unroll
      for (int m = 0; m < MT; ++m) xf[d][m][j] = ld16(x[m] + (in ? k : 0));
#pragma unroll
      for (int b = 0; b < RB; ++b) wf[d][b][j] = bld16(wb, in ? woff[b] + k * 2 : kNoRow);
    }
  };
  if (nsteps > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, d);
    for (int s0 = 0; s0 < nsteps; s0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (s0 + d < nsteps) {
          const int k = (k0 + s0 + d) * 64;
          if (k + 64 > a.K) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int m = 0; m < MT; ++m) xf[d][m][j] = keep(xf[d][m][j], k + j * 32 + q * 8 < a.K);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
              for (int m = 0; m < MT; ++m) acc[b][m] = mfma16<DT>(wf[d][b][j], xf[d][m][j], acc[b][m]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (s0 + d + D < nsteps) load(d, s0 + d + D);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // lane (c, q), register v of block (b, m): t[row 16 m + c, 16 b + 4 q + v]
  constexpr int kBlocks = RB * MT, kOnce = kBlocks < 8 ? kBlocks : 8;  // blocks joined at a time
  __shared__ f32x4_t s_part[kWaves][kOnce][kWave];
  float* const out = a.part + (static_cast<int64_t>(blockIdx.y) * a.M + t.row0) * a.R;
#pragma unroll
  for (int at = 0; at < kBlocks; at += kOnce) {
    if (at > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < kOnce; ++i) s_part[wv][i][lane] = acc[(at + i) / MT][(at + i) % MT];
    __syncthreads();
    for (int i = wv; i < kOnce; i += kWaves) {
      f32x4_t v = s_part[0][i][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += s_part[w][i][lane];
      const int r = (at + i) / MT * 16 + q * 4, m = (at + i) % MT * 16 + c;
      if (m < t.rows && r < a.R) *reinterpret_cast<f32x4_t*>(out + static_cast<int64_t>(m) * a.R + r) = v;
    }
  }
}

// A lane's 16-byte pieces of a row of base or out, of which n elements are there.
template <int OT>
__device__ __forceinline__ uint4 load_piece(const void* p, int n) {
  constexpr int kVec = Row<OT>::kVec, kSize = Row<OT>::kSize;
  if (n >= kVec) return ld16_any<false>(p);
  uint4 v = {0u, 0u, 0u, 0u};
  float f[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] = i < n ? Row<OT>::get(static_cast<const uint8_t*>(p) + i * kSize) : 0.0f;
  v = Row<OT>::pack(f);
  return v;
}
template <int OT>
__device__ __forceinline__ void store_piece(void* p, int n, const float* f) {
  constexpr int kVec = Row<OT>::kVec, kSize = Row<OT>::kSize;
  if (n >= kVec) {
    st16_any<false>(p, Row<OT>::pack(f));
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) Row<OT>::put(static_cast<uint8_t*>(p) + i * kSize, f[i]);
  }
}

// out of a tile's rows and a span of N. RS: 32-steps of R; MT: 16-row blocks of the
// tile. t is summed over the parts of K and goes to LDS as a sum of terms in B's type:
// hi + lo keep t to 2^-16 in bfloat16 (2^-22 in half), which is past a 16-bit result;
// results in 32 bits from bfloat16 take a third term (2^-24). The MFMAs this costs hide
// behind memory. In half a row of t is first divided by a power of two that brings its
// largest value below 2, past neither end of the range.
//
// Of four MFMAs on 64 columns, number j takes column col(j, i / 4) + i % 4 as its row i: so
// a lane's results are 16-byte pieces of a row of out, and the pieces of four lanes lie
// side by side.
template <int DT, int OT, int RS, int MT>
__global__ __launch_bounds__(kThreads) void adapter_up_kernel(AdapterArgs a, int tiles, int span, int spans) {
  constexpr int TR = 16 * MT, kPad = 8, kRow = RS * 32 + kPad;  // halves of a row of t in LDS
  constexpr int kTerms = DT == MOE_DTYPE_BF16 && OT == MOE_DTYPE_FP32 ? 3 : 2;
  constexpr int OS = Row<OT>::kSize, kVec = Row<OT>::kVec, kPieces = 16 / kVec;
  constexpr auto col = [](int j, int q) { return OS == 4 ? j * 16 + q * 4 : (j >> 1) * 32 + q * 8 + (j & 1) * 4; };
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_index(), c = lane & 15, q = lane >> 4;
  // spans of the same rows are neighbours
  const int tile = blockIdx.x / spans, n0 = (blockIdx.x - tile * spans) * span, n1 = min(a.N, n0 + span);
  uint8_t* const out = static_cast<uint8_t*>(a.out);
  const uint8_t* const base = static_cast<const uint8_t*>(a.base);
  if (tile >= tiles) {
    // rows without an adapter, where out is an array of its own
    const int r0 = (tile - tiles) * TR;
    for (int r = r0 + wv; r < min(a.M, r0 + TR); r += kWaves) {
      if (a.slot_row[r] >= 0) continue;
      for (int n = n0 + lane * kVec; n < n1; n += kWave * kVec) {
        float f[kVec] = {};
        if (base != nullptr) Row<OT>::unpack(load_piece<OT>(base + (r * a.ldb + n) * OS, n1 - n), f);
        store_piece<OT>(out + (r * a.ldo + n) * OS, n1 - n, f);
      }
    }
    return;
  }
  __shared__ __attribute__((aligned(16))) uint16_t s_t[kTerms][TR * kRow];
  __shared__ float s_scale[TR];
  const AdapterTile t = find_tile<TR>(a, tile);
  if (t.rows == 0) return;
  // The loads that need no t go out first.
  int row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) row[m] = m * 16 + c < t.rows ? row_of(a, t.row0 + m * 16 + c) : -1;
  const uint16_t* const b = static_cast<const uint16_t*>(a.b) + static_cast<int64_t>(t.adapter) * a.N * a.R;
  uint4 w[4][RS], old[MT][kPieces];
  auto load = [&](int n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = min(n + col(j, c >> 2) + (c & 3), a.N - 1);
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const int r = s * 32 + q * 8;
        w[j][s] = ld16(b + static_cast<int64_t>(at) * a.R + (r < a.R ? r : 0));
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = n + col(i * kVec / 4, q);
        old[m][i] = uint4{0u, 0u, 0u, 0u};
        if (base != nullptr && row[m] >= 0 && at < n1)
          old[m][i] = load_piece<OT>(base + (row[m] * a.ldb + at) * OS, n1 - at);
      }
  };
  int n = n0 + wv * 64;
  if (n < n1) load(n);
  // t: sixteen threads a row, 2 RS values each
  constexpr int kPer = RS * 2, kOnce = 4;
  typedef float vec_t __attribute__((ext_vector_type(kPer), aligned(8)));
  const float factor = a.scale != nullptr ? a.scale[t.adapter] : 1.0f;
#pragma unroll
  for (int m0 = 0; m0 < TR; m0 += kThreads / 16) {
    const int m = m0 + (tid >> 4), r = (tid & 15) * kPer;
    // R is a multiple of 8: a thread's values are all there or none is
    const bool in = m < t.rows && r < a.R;
    const float* p = a.part + static_cast<int64_t>(t.row0 + (in ? m : 0)) * a.R + (in ? r : 0);
    const int64_t step = static_cast<int64_t>(a.M) * a.R;
    vec_t v = {};
    for (int s = 0; s < a.splits; s += kOnce) {
      vec_t u[kOnce];
#pragma unroll
      for (int i = 0; i < kOnce; ++i) u[i] = *reinterpret_cast<const vec_t*>(p + min(s + i, a.splits - 1) * step);
#pragma unroll
      for (int i = 0; i < kOnce; ++i)
        if (s + i < a.splits) v += u[i];
    }
    if (!in) v = vec_t{};
    float f = factor;
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
      float left = v[i];
#pragma unroll
      for (int k = 0; k < kTerms; ++k) {
        uint16_t h;
        Row<DT>::put(&h, left);
        s_t[k][m * kRow + r + i] = h;
        const float term = Row<DT>::get(&h);
        left = fabsf(term) < __builtin_inff() ? left - term : 0.0f;  // nothing beside an infinity or NaN
      }
    }
    if ((tid & 15) == 0) s_scale[m] = f;
  }
  __syncthreads();
  float scale[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) scale[m] = s_scale[m * 16 + c];
  for (; n < n1; n += kWaves * 64) {
    if (a.R % 32 != 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < RS; ++s) w[j][s] = keep(w[j][s], s * 32 + q * 8 < a.R);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m * 16 >= t.rows) break;
      f32x4_t acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < RS; ++s) {
#pragma unroll
        for (int k = kTerms - 1; k >= 0; --k) {
          const uint4 term = *reinterpret_cast<const uint4*>(&s_t[k][(m * 16 + c) * kRow + s * 32 + q * 8]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = mfma16<DT>(w[j][s], term, acc[j]);
        }
      }
      if (row[m] < 0) continue;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = n + col(i * kVec / 4, q);
        if (at >= n1) continue;
        float f[kVec];
        Row<OT>::unpack(old[m][i], f);
#pragma unroll
        for (int v = 0; v < kVec; ++v) f[v] += scale[m] * acc[i * kVec / 4 + v / 4][v % 4];
        store_piece<OT>(out + (row[m] * a.ldo + at) * OS, n1 - at, f);
      }
    }
    if (n + kWaves * 64 < n1) load(n + kWaves * 64);
  }
}

// Sixteens of rows that a tile takes. Two halve the reads of A and B from the caches, which
// pays for long rows of t and rows enough to fill the card all the same (8192 rows of 2
// adapters, K 3584, N 4096: rank 64 61 us, four sixteens 73; rank 128 93, 134 with one; rank
// 8 45, 44 with one; 2683 rows of 16, K 808, N 1456, rank 32: 14.5, 12.0 with one).
int tile_rows(int64_t M, int64_t A, int64_t R) { return M >= 32 * A && R > 16 && M * R >= 100000 ? 2 : 1; }

// Tiles there are at most one for each row, and one for each adapter beside the full ones.
int64_t tile_bound(const AdapterArgs& a, int tr) { return std::min<int64_t>(a.M, a.M / (16 * tr) + std::min(a.A, a.M)); }

template <int DT, int RB>
void down(const AdapterArgs& a, hipStream_t st) {
  const int tr = tile_rows(a.M, a.A, a.R);
  const dim3 grid(static_cast<unsigned>(tile_bound(a, tr)), static_cast<unsigned>(a.splits));
  if (tr == 2)
    hipLaunchKernelGGL((adapter_down_kernel<DT, RB, 2>), grid, dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((adapter_down_kernel<DT, RB, 1>), grid, dim3(kThreads), 0, st, a);
}

template <int DT, int OT, int RS>
void up(const AdapterArgs& a, hipStream_t st) {
  const int tr = tile_rows(a.M, a.A, a.R);
  const int64_t tiles = tile_bound(a, tr);
  // rows without an adapter need a copy only where out is not base
  const int64_t others = a.out == a.base ? 0 : (a.M + 16 * tr - 1) / (16 * tr);
  // Spans of N: about four blocks a CU, of a piece a wave or more, and all of one length
  // where that is not under half of it (4096 rows of 32 adapters, K 3584, N 4096, rank 64:
  // 43 us, 49 with a shorter last one); eight where tiles of 32 rows alone make one, whose
  // shorter spans then lie nearer to each other in memory. Eight and four (us): rank 64, K
  // 3584, N 7168, 8 adapters: 8191 rows 106 and 113, 12000 161 and 176, 16000 202 and 206;
  // N 4096, 32 adapters: 65 and 64, 119 and 125, 140 and 153. Below 256 tiles: 2048 rows 37
  // and 34, 6000 68 and 69. Short rows (K 1024, N 2048, 2 adapters) the same, but of rank
  // 128 from 12000 rows on 68 and 61.
  const int64_t pieces = (a.N + 64 * kWaves - 1) / (64 * kWaves);
  const int64_t want = std::clamp<int64_t>((tr == 2 && tiles >= 256 ? 2048 : 1024) / std::max<int64_t>(tiles, 1), 1, pieces);
  int64_t per = (pieces + want - 1) / want;
  for (int64_t p = per; p >= (per + 1) / 2; --p) {
    if (pieces % p != 0) continue;
    per = p;
    break;
  }
  const int span = static_cast<int>(per) * kWaves * 64;
  const int spans = (a.N + span - 1) / span, count = static_cast<int>(tiles);
  const dim3 grid(static_cast<unsigned>((tiles + others) * spans));
  if (tr == 2)
    hipLaunchKernelGGL((adapter_up_kernel<DT, OT, RS, 2>), grid, dim3(kThreads), 0, st, a, count, span, spans);
  else
    hipLaunchKernelGGL((adapter_up_kernel<DT, OT, RS, 1>), grid, dim3(kThreads), 0, st, a, count, span, spans);
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

// Parts of K: a block a CU, or with tiles of 32 rows two, as these load more than a wave
// holds in flight; every part is also one more of t to sum (64 requests 11.5 us, 12.2 with
// twice the parts; 4096 rows of 32 adapters, rank 64: 49, 54 with half of them).
int adapter_splits(int64_t M, int64_t A, int64_t K, int64_t R) {
  const int tr = tile_rows(M, A, R);
  const int64_t tiles = std::max<int64_t>(1, std::min<int64_t>(M, M / (16 * tr) + std::min(A, M)));
  const int64_t steps = (K + 63) / 64 / kWaves;  // a wave's, unsplit
  return static_cast<int>(std::clamp<int64_t>(std::min(tr > 1 ? 512 / tiles : (255 + tiles) / tiles, steps / 2), 1, 16));
}

hipError_t launch_adapter(const AdapterArgs& a, hipStream_t st) {
  if (a.dtype == MOE_DTYPE_BF16) both<MOE_DTYPE_BF16>(a, st);
  else both<MOE_DTYPE_FP16>(a, st);
  return hipGetLastError();
}

}  // namespace moe
