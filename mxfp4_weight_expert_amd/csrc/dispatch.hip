// Dispatch: token rows into expert order. Slot s = t * topk + k with local
// expert e(s) goes to row
//   row(s) = #{s' : e(s') < e(s)} + #{s' < s : e(s') = e(s)},
// so rows follow the experts and, within one, the slots, whatever order the
// blocks run in. What it cannot do without: the ids, each token once, each
// row once; memory bounds it.
#include "rows.h"
#include "kernels.h"

namespace moe {

// Local expert of a global id, or -1.
__device__ __forceinline__ int local_expert(int id, int offset, int E) {
  return id >= offset && id - offset < E ? id - offset : -1;
}

// One wave copies a row of `bytes` (a multiple of 2).
__device__ __forceinline__ void wave_copy_row(const uint8_t* src, uint8_t* dst, uint32_t bytes) {
  const uint32_t n = bytes >> 4, lane = lane_id();
  uint32_t c = lane;
  for (; c + 192 < n; c += 256) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = ld16_any<false>(src + 16 * static_cast<size_t>(c + 64 * u));
#pragma unroll
    for (int u = 0; u < 4; ++u) st16_any<false>(dst + 16 * static_cast<size_t>(c + 64 * u), v[u]);
  }
  for (; c < n; c += 64)
    st16_any<false>(dst + 16 * static_cast<size_t>(c), ld16_any<false>(src + 16 * static_cast<size_t>(c)));
  const uint32_t at = (n << 4) + 2 * lane;
  if (at < bytes)
    *reinterpret_cast<uint16_t*>(dst + at) = *reinterpret_cast<const uint16_t*>(src + at);
}

// Few slots: one launch. Every block reads all ids and keys slot s by
// (expert, s), expert E for slots without one; a wave counts the keys below
// its slot's, which is its row, and copies the token there. The last block
// counts the slots of each expert and scans the counts. The counting grows with
// the square of the slots: up to kFusedSlots it stays below the four launches of
// the path for many (896 experts, 7 KB rows: 4.6 us against 16 at 1024 slots, 14
// against 18 at 4096, 41 against 24 at 8192).
__global__ __launch_bounds__(256) void dispatch_fused_kernel(
    const uint8_t* __restrict__ x, const int32_t* __restrict__ ids, int nslots, int topk, int E,
    int expert_offset, uint32_t row_bytes, uint8_t* __restrict__ rows,
    int32_t* __restrict__ offsets, int32_t* __restrict__ row_slot, int32_t* __restrict__ slot_row) {
  __shared__ __attribute__((aligned(16))) uint32_t s_key[kFusedSlots];
  __shared__ int s_wave[4];
  const int tid = threadIdx.x, lane = lane_id(), w = wave_index();
  if (blockIdx.x == gridDim.x - 1) {
    int* cnt = reinterpret_cast<int*>(s_key);  // kMaxExperts counters
    for (int e = tid; e < kMaxExperts; e += 256) cnt[e] = 0;
    __syncthreads();
    for (int s = tid; s < nslots; s += 256) {
      const int e = local_expert(ids[s], expert_offset, E);
      if (e >= 0) atomicAdd(&cnt[e], 1);  // whole numbers: the order changes nothing
    }
    __syncthreads();
    constexpr int kPer = kMaxExperts / 256;
    int c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] = cnt[tid * kPer + i];
      sum += c[i];
    }
    const int incl = wave_incl_scan(sum);
    if (lane == kWave - 1) s_wave[w] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int i = 0; i < w; ++i) at += s_wave[i];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      if (e <= E) offsets[e] = at;  // counters from E on are 0: offsets[E] is the total
      at += c[i];
    }
    if (E == kMaxExperts && tid == 255) offsets[E] = at;
    return;
  }
  const int nkeys = (nslots + 255) & ~255;
  for (int s = tid; s < nkeys; s += 256) {
    const int e = s < nslots ? local_expert(ids[s], expert_offset, E) : -1;
    s_key[s] = static_cast<uint32_t>(e >= 0 ? e : E) * kFusedSlots + s;
  }
  __syncthreads();
  const int s = blockIdx.x * 4 + w;
  if (s >= nslots) return;
  const uint32_t key = s_key[s];
  if (key >= static_cast<uint32_t>(E) * kFusedSlots) {
    if (lane == 0) slot_row[s] = -1;
    return;
  }
  int row = 0;
  for (int i = 0; i < nkeys; i += 4 * kWave) {
    const uint4 k = *reinterpret_cast<const uint4*>(s_key + i + 4 * lane);
    row += __popcll(ballot(k.x < key)) + __popcll(ballot(k.y < key)) +
           __popcll(ballot(k.z < key)) + __popcll(ballot(k.w < key));
  }
  if (lane == 0) {
    slot_row[s] = row;
    row_slot[row] = s;
  }
  wave_copy_row(x + static_cast<size_t>(s / topk) * row_bytes,
                rows + static_cast<size_t>(row) * row_bytes, row_bytes);
}

// Many slots: the maps come from launch_sort_maps;
// then a one-wave block takes 1 KB of a token, reads it once and writes it to
// the token's rows, past the caches (131k rows of 7 KB, 1 GB in all: 188 us with
// plain stores, 175 with these, 5.7 TB/s; a wave a whole row, or blocks of 256
// threads with 4 KB, the same or slower; a plain fill writes at 6.9).
__global__ __launch_bounds__(64) void dispatch_copy_kernel(const uint8_t* __restrict__ x,
                                                           const int32_t* __restrict__ slot_row,
                                                           int topk, uint32_t row_bytes, int npiece,
                                                           uint8_t* __restrict__ rows) {
  const int t = blockIdx.x / npiece;
  const uint32_t c = (blockIdx.x - t * npiece) * kWave + lane_id();
  const uint32_t n = row_bytes >> 4, tail = row_bytes & 15;
  const uint8_t* src = x + static_cast<size_t>(t) * row_bytes + 16 * static_cast<size_t>(c);
  const int32_t* map = slot_row + static_cast<size_t>(t) * topk;
  uint4 v = {0, 0, 0, 0};
  if (c < n) v = ld16_any<false>(src);
  for (int k = 0; k < topk; ++k) {
    const int row = map[k];
    if (row < 0) continue;
    uint8_t* dst = rows + static_cast<size_t>(row) * row_bytes + 16 * static_cast<size_t>(c);
    if (c < n) {
      st16_any<true>(dst, v);
    } else if (c == n) {
      for (uint32_t b = 0; b < tail; b += 2)
        *reinterpret_cast<uint16_t*>(dst + b) = *reinterpret_cast<const uint16_t*>(src + b);
    }
  }
}

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t st) {
  const uint32_t row_bytes = static_cast<uint32_t>(a.H) * a.elem;
  const int nslots = a.T * a.topk;
  if (nslots <= kFusedSlots) {
    hipLaunchKernelGGL(dispatch_fused_kernel, dim3((nslots + 3) / 4 + 1), dim3(256), 0, st, a.x,
                       a.ids, nslots, a.topk, a.E, a.expert_offset, row_bytes, a.rows, a.offsets,
                       a.row_slot, a.slot_row);
    return hipGetLastError();
  }
  SortMapsArgs m;
  m.ids = a.ids;
  m.nslots = nslots;
  m.E = a.E;
  m.expert_offset = a.expert_offset;
  m.range_counts = a.range_counts;
  m.counts = a.counts;
  m.offsets = a.offsets;
  m.row_slot = a.row_slot;
  m.slot_row = a.slot_row;
  const hipError_t err = launch_sort_maps(m, st);
  if (err != hipSuccess || row_bytes == 0) return err;  // no rows: the maps alone
  const int npiece = static_cast<int>((row_bytes + 1023) / 1024);
  hipLaunchKernelGGL(dispatch_copy_kernel, dim3(static_cast<unsigned>(a.T) * npiece), dim3(64), 0,
                     st, a.x, a.slot_row, a.topk, row_bytes, npiece, a.rows);
  return hipGetLastError();
}

}  // namespace moe
