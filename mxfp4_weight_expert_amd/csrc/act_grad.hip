// Gradient of the gated product's activation: dg, du from dh and the
// pre-activations g, u of the rows that experts own. Elementwise; memory bounds
// it: three arrays read and two written, M * I elements each (8192 rows, I 2048, bf16: 168
// MB in 29 us, 5.8 TB/s, a large copy 4.9). dgu is rounded before the products that take
// it, which read it as 16-bit operands; what the rounding leaves goes to an array of its
// own where the caller asks for two terms, and the products take both.
#include "rows.h"
#include "kernels.h"

namespace moe {

namespace {

// d act / d g and d act / d u, times dh (act as act_apply of common.h).
__device__ __forceinline__ void act_grad(float dh, float g, float u, const ActArgs& a, float& dg, float& du) {
  if (a.kind == MOE_ACT_SITU) {
    const float s = 1.0f / (1.0f + __expf(-g)), tg = tanhf(g * a.inv_beta), tu = tanhf(u * a.inv_lb);
    dg = dh * (a.lb * tu) * (s * ((1.0f - tg * tg) + a.beta * tg * (1.0f - s)));
    du = dh * (a.beta * tg * s) * (1.0f - tu * tu);
    return;
  }
  bool in_g = true, in_u = true;
  if (a.limit > 0.0f) {
    in_g = !(g > a.limit);  // NaN is not cut off
    in_u = !(fabsf(u) > a.limit);
    g = clamp_gate(g, a.limit);
    u = clamp_up(u, a.limit);
  }
  const float s = 1.0f / (1.0f + __expf(-g));
  dg = in_g ? dh * u * (s * (1.0f + g * (1.0f - s))) : 0.0f;
  du = in_u ? dh * (g * s) : 0.0f;
}

// Eight values rounded, and what is left of each (nothing beside an infinity or NaN).
template <int DT>
__device__ __forceinline__ void store_terms(const float* v, uint16_t* to, uint16_t* rest) {
  const uint4 p = Row<DT>::pack(v);
  *reinterpret_cast<uint4*>(to) = p;
  if (rest == nullptr) return;
  float r[8];
  Row<DT>::unpack(p, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = fabsf(r[i]) < __builtin_inff() ? v[i] - r[i] : 0.0f;
  *reinterpret_cast<uint4*>(rest) = Row<DT>::pack(r);
}

template <int DT>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a) {
  int lo = 0, hi = a.M;
  if (a.offsets != nullptr) {
    lo = min(max(a.offsets[0], 0), a.M);
    hi = min(a.offsets[a.E], a.M);
  }
  const int pieces = a.I >> 3;  // of a row, eight elements each
  const int64_t n = static_cast<int64_t>(hi - lo) * pieces, step = static_cast<int64_t>(gridDim.x) * 256;
  const uint16_t* const dh = static_cast<const uint16_t*>(a.dh);
  const uint16_t* const gu = static_cast<const uint16_t*>(a.gu);
  uint16_t* const out = static_cast<uint16_t*>(a.dgu);
  uint16_t* const rest = static_cast<uint16_t*>(a.rest);
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < n; at += step) {
    const int64_t row = lo + at / pieces;
    const int i = static_cast<int>(at % pieces) * 8;
    float d[8], g[8], u[8], dg[8], du[8];
    Row<DT>::unpack(ld16(dh + row * a.I + i), d);
    Row<DT>::unpack(ld16(gu + row * 2 * a.I + i), g);
    Row<DT>::unpack(ld16(gu + row * 2 * a.I + a.I + i), u);
#pragma unroll
    for (int v = 0; v < 8; ++v) act_grad(d[v], g[v], u[v], a.act, dg[v], du[v]);
    const int64_t to = row * 2 * a.I + i;
    store_terms<DT>(dg, out + to, rest != nullptr ? rest + to : nullptr);
    store_terms<DT>(du, out + to + a.I, rest != nullptr ? rest + to + a.I : nullptr);
  }
}

}  // namespace

hipError_t launch_act_grad(const ActGradArgs& a, hipStream_t st) {
  const int64_t want = (static_cast<int64_t>(a.M) * (a.I >> 3) + 255) / 256;
  const dim3 grid(static_cast<unsigned>(want < 4096 ? want : 4096));
  if (a.dtype == MOE_DTYPE_BF16)
    hipLaunchKernelGGL(act_grad_kernel<MOE_DTYPE_BF16>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(act_grad_kernel<MOE_DTYPE_FP16>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace moe
