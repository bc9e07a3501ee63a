// Row access of the dispatch and combine kernels: rows of any length in
// bfloat16, half or float, moved in 16-byte pieces whatever the row's
// alignment (global loads and stores of gfx950 take any address; an odd H
// puts every second 16-bit row off a 4-byte boundary).
#pragma once

#include "common.h"
#include "moe_ops.h"

namespace moe {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <bool NT>
__device__ __forceinline__ uint4 ld16_any(const void* p) {
  const u32x4_any* q = static_cast<const u32x4_any*>(p);
  if constexpr (NT)
    return __builtin_bit_cast(uint4, static_cast<u32x4_t>(__builtin_nontemporal_load(q)));
  else
    return __builtin_bit_cast(uint4, static_cast<u32x4_t>(*q));
}
template <bool NT>
__device__ __forceinline__ void st16_any(void* p, const uint4& v) {
  u32x4_any* q = static_cast<u32x4_any*>(p);
  const u32x4_any u = __builtin_bit_cast(u32x4_t, v);
  if constexpr (NT)
    __builtin_nontemporal_store(u, q);
  else
    *q = u;
}

// Element type DT (MOE_DTYPE_*): 16-byte pieces to floats and back. The only
// rounding is pack's, to the nearest even.
template <int DT>
struct Row;
template <>
struct Row<MOE_DTYPE_BF16> {
  static constexpr int kVec = 8, kSize = 2;
  __device__ static void unpack(const uint4& v, float* f) {
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(d[i] << 16);
      f[2 * i + 1] = __uint_as_float(d[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float* f) {
    return uint4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                 pack_bf16x2(f[6], f[7])};
  }
  __device__ static float get(const void* p) {
    return bf16_to_f32(*static_cast<const uint16_t*>(p));
  }
  __device__ static void put(void* p, float f) { *static_cast<uint16_t*>(p) = f32_to_bf16(f); }
};
template <>
struct Row<MOE_DTYPE_FP16> {
  static constexpr int kVec = 8, kSize = 2;
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  __device__ static void unpack(const uint4& v, float* f) {
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const h2 h = __builtin_bit_cast(h2, d[i]);
      f[2 * i] = static_cast<float>(h.x);
      f[2 * i + 1] = static_cast<float>(h.y);
    }
  }
  __device__ static uint32_t pack2(float a, float b) {
    const h2 h = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
    return __builtin_bit_cast(uint32_t, h);
  }
  __device__ static uint4 pack(const float* f) {
    return uint4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
  }
  __device__ static float get(const void* p) {
    return static_cast<float>(*static_cast<const _Float16*>(p));
  }
  __device__ static void put(void* p, float f) {
    *static_cast<_Float16*>(p) = static_cast<_Float16>(f);
  }
};
template <>
struct Row<MOE_DTYPE_FP32> {
  static constexpr int kVec = 4, kSize = 4;
  __device__ static void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float* f) {
    return uint4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                 __float_as_uint(f[3])};
  }
  __device__ static float get(const void* p) { return *static_cast<const float*>(p); }
  __device__ static void put(void* p, float f) { *static_cast<float*>(p) = f; }
};

}  // namespace moe
