// Combine: expert rows weighted and summed back to token order, and its
// gradients. Each row and each token is read or written once; memory bounds
// all three. Sums are 32-bit, in an order fixed by the sizes (no atomics).
#include "rows.h"
#include "kernels.h"

#include <type_traits>

namespace moe {

// out[t] = sum over k of w[t, k] * rows[row(t, k)] (w = nullptr: 1, the
// gradient of dispatch). A one-wave block takes 64 16-byte pieces of one
// token; it first packs the token's rows and weights into LDS in ascending k,
// so the sum has no branches and its loads go out eight at a time. Rows and
// result pass the caches: 1 GB for 8191 tokens of 8 rows of 14 KB took 210 us with
// plain loads, 198 with non-temporal ones, 179 (5.9 TB/s) with the stores so too;
// two to seven pieces a lane, or sixteen loads at a time, were slower.
template <int DT>
__global__ __launch_bounds__(64) void combine_kernel(const uint8_t* __restrict__ rows,
                                                     const int32_t* __restrict__ slot_row,
                                                     const float* __restrict__ topk_w, int topk,
                                                     int nslots, int H, int npiece,
                                                     uint8_t* __restrict__ out) {
  using R = Row<DT>;
  constexpr int V = R::kVec;
  __shared__ int32_t s_row[kMaxTopK];
  __shared__ float s_w[kMaxTopK];
  const int t = blockIdx.x / npiece;
  const int c = (blockIdx.x - t * npiece) * kWave + lane_id();
  const int k = lane_id();
  const size_t slot = static_cast<size_t>(t) * topk + k;
  const int row = k < topk ? slot_row[slot] : -1;
  const float w = k < topk && topk_w != nullptr ? topk_w[slot] : 1.0f;  // with the row: one latency
  const bool valid = static_cast<uint32_t>(row) < static_cast<uint32_t>(nslots);
  const uint64_t m = ballot(valid);
  if (valid) {
    const int pos = popc_below(m);
    s_row[pos] = row;
    s_w[pos] = w;
  }
  __syncthreads();
  const int n = __popcll(m);
  const int nvec = H / V;
  const size_t row_bytes = static_cast<size_t>(H) * R::kSize;
  const uint8_t* src = rows + 16 * static_cast<size_t>(c);
  uint8_t* dst = out + static_cast<size_t>(t) * row_bytes + 16 * static_cast<size_t>(c);
  if (c < nvec) {
    float acc[V], f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int k0 = 0; k0 < n; k0 += 8) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (k0 + u < n) v[u] = ld16_any<true>(src + s_row[k0 + u] * row_bytes);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (k0 + u < n) {
          R::unpack(v[u], f);
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] += s_w[k0 + u] * f[i];
        }
      }
    }
    st16_any<true>(dst, R::pack(acc));
  } else if (c == nvec) {
    for (int i = 0; i < H - nvec * V; ++i) {
      float acc = 0.0f;
      for (int u = 0; u < n; ++u) acc += s_w[u] * R::get(src + s_row[u] * row_bytes + i * R::kSize);
      R::put(dst + i * R::kSize, acc);
    }
  }
}

// Gradients of combine: a wave per slot writes w * dout[t] to the slot's row
// and reduces <dout[t], row> over its lanes. The token's other waves find dout in
// the caches; rows in and out pass them. 1 GB for 4096 tokens of 8 rows of 14 KB:
// 206 us with plain accesses one piece at a time, 189 now, 5.3 TB/s (a copy of
// 2 GiB on this card: 4.9).
template <int DT>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const uint8_t* __restrict__ dout, const uint8_t* __restrict__ rows,
    const int32_t* __restrict__ slot_row, const float* __restrict__ topk_w, int topk, int nslots,
    int H, uint8_t* __restrict__ drows, float* __restrict__ dtopk_w) {
  using R = Row<DT>;
  constexpr int V = R::kVec;
  // Consecutive blocks go to the eight XCDs in turn: each XCD takes a run of slots
  // of its own, so that a token's blocks find its dout in one L2 (the 4096 tokens
  // above: 192 -> 189 us, and 59 MB less read).
  const int per = gridDim.x >> 3, b = blockIdx.x;
  const int block = b < 8 * per ? (b & 7) * per + (b >> 3) : b;
  const int s = block * 4 + wave_index();
  if (s >= nslots) return;
  const int lane = lane_id();
  const int row = slot_row[s];
  const float w = topk_w[s];
  if (static_cast<uint32_t>(row) >= static_cast<uint32_t>(nslots)) {
    if (lane == 0) dtopk_w[s] = 0.0f;
    return;
  }
  const size_t row_bytes = static_cast<size_t>(H) * R::kSize;
  const uint8_t* g = dout + static_cast<size_t>(s / topk) * row_bytes;
  const uint8_t* y = rows + row * row_bytes;
  uint8_t* d = drows + row * row_bytes;
  const int nvec = H / V;
  float dot = 0.0f;
  auto piece = [&](const uint4& vg, const uint4& vy, size_t at) {
    float fg[V], fy[V];
    R::unpack(vg, fg);
    R::unpack(vy, fy);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dot += fg[i] * fy[i];
      fg[i] *= w;
    }
    st16_any<true>(d + at, R::pack(fg));
  };
  // U pieces a lane at once; lanes past the row's end load its last piece again.
  // Rows of more than four pieces a lane take eight (64 tokens x 16 rows of 7 KB:
  // 4.4 us, 5.7 with four and the rest one by one), shorter ones no more than they
  // have (2000 x 8 rows of 1 KB: 12.9 us, 16.5 with eight).
  auto walk = [&](auto uc) {
    constexpr int U = decltype(uc)::value;
    for (int c0 = 0; c0 < nvec; c0 += U * kWave) {
      uint4 vg[U], vy[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (U == 4 && c0 + u * kWave >= nvec) break;
        const size_t at = 16 * static_cast<size_t>(min(c0 + u * kWave + lane, nvec - 1));
        vy[u] = ld16_any<true>(y + at);
        vg[u] = ld16_any<false>(g + at);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * kWave + lane;
        if (U == 4 && c0 + u * kWave >= nvec) break;
        if (c < nvec) piece(vg[u], vy[u], 16 * static_cast<size_t>(c));
      }
    }
  };
  if (nvec > 4 * kWave) walk(std::integral_constant<int, 8>{});
  else walk(std::integral_constant<int, 4>{});
  const int i = nvec * V + lane;
  if (i < H) {
    const size_t at = static_cast<size_t>(i) * R::kSize;
    const float fg = R::get(g + at);
    dot += fg * R::get(y + at);
    R::put(d + at, w * fg);
  }
  dot = wave_sum_f(dot);
  if (lane == 0) dtopk_w[s] = dot;
}

namespace {
template <class F>
hipError_t by_dtype(int dtype, F f) {
  if (dtype == MOE_DTYPE_BF16) f(std::integral_constant<int, MOE_DTYPE_BF16>{});
  else if (dtype == MOE_DTYPE_FP16) f(std::integral_constant<int, MOE_DTYPE_FP16>{});
  else f(std::integral_constant<int, MOE_DTYPE_FP32>{});
  return hipGetLastError();
}
}  // namespace

hipError_t launch_combine(const CombineArgs& a, hipStream_t st) {
  return by_dtype(a.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const int npiece = (a.H + Row<DT>::kVec * kWave - 1) / (Row<DT>::kVec * kWave);
    hipLaunchKernelGGL((combine_kernel<DT>), dim3(static_cast<unsigned>(a.T) * npiece), dim3(64), 0,
                       st, a.rows, a.slot_row, a.topk_w, a.topk, a.T * a.topk, a.H, npiece, a.out);
  });
}

hipError_t launch_combine_backward(const CombineArgs& a, hipStream_t st) {
  return by_dtype(a.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const int nslots = a.T * a.topk;
    hipLaunchKernelGGL((combine_backward_kernel<DT>), dim3((nslots + 3) / 4), dim3(256), 0, st,
                       a.dout, a.rows, a.slot_row, a.topk_w, a.topk, nslots, a.H, a.out, a.dtopk_w);
  });
}

}  // namespace moe
