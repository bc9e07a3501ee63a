// C ABI of the 16-bit products (moe_linear.h): argument checks, then the launches.
#include "checks.h"
#include "common.h"
#include "kernels.h"
#include "moe_linear.h"

#include <cmath>

using namespace moe;

namespace {

// Elements of a row or from row to row, and of a matrix: byte offsets inside a tile
// (256 rows) and inside a matrix stay below the 2^31 that buffer accesses of the
// kernels count to.
constexpr int64_t kMaxLd = int64_t{1} << 20;
constexpr int64_t kMaxMatrix = int64_t{1} << 30;

bool half_type(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_FP16; }

// A product of M rows of K elements with E matrices of N rows.
struct Product {
  int64_t M, N, K, E, ldx, ldo, out_cols;  // out_cols: elements of a row of the result
  int dtype, out_dtype;
};

int check(const Product& p) {
  if (p.M < 0 || p.N < 1 || p.K < 1 || p.E < 1) return MOE_ERR_INVALID;
  if (p.N % 8 != 0 || p.K % 8 != 0 || p.ldx % 8 != 0 || p.ldo % 8 != 0 || p.out_cols % 8 != 0) return MOE_ERR_INVALID;
  if ((p.ldx != 0 && p.ldx < p.K) || (p.ldo != 0 && p.ldo < p.out_cols)) return MOE_ERR_INVALID;
  if (p.M > kMaxSlots || p.N > kMaxLd || p.K > kMaxLd || p.ldx > kMaxLd || p.ldo > kMaxLd || p.E > kMaxExperts ||
      p.N * p.K > kMaxMatrix || !half_type(p.dtype) || (p.out_dtype != p.dtype && p.out_dtype != MOE_DTYPE_FP32))
    return MOE_ERR_UNSUPPORTED;
  if ((p.M / 16 + p.E + 1) * (p.N / 16 + 1) >= kMaxTileItems) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check(const moe_linear_shape* s, Product& p) {
  if (s == nullptr) return MOE_ERR_INVALID;
  p = {s->M, s->N, s->K, s->E, s->ldx, s->ldo, s->N, s->dtype, s->out_dtype};
  return check(p);
}

int check(const moe_gated_shape* s, Product& p) {
  if (s == nullptr || s->I < 1) return MOE_ERR_INVALID;
  p = {s->M, int64_t{2} * s->I, s->H, s->E, s->ldx, s->ldo, s->I, s->dtype, s->dtype};
  const bool situ = s->activation == MOE_ACT_SITU;
  if (!std::isfinite(s->swiglu_limit) || s->dgu_terms < 0 || s->dgu_terms > 2) return MOE_ERR_INVALID;
  if (situ && !(std::isfinite(s->act_beta) && s->act_beta > 0.0f && std::isfinite(s->act_linear_beta) &&
                s->act_linear_beta > 0.0f))
    return MOE_ERR_INVALID;
  const int rc = check(p);
  if (rc != MOE_OK) return rc;
  return situ || s->activation == MOE_ACT_SWIGLU ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

ActArgs act_args(const moe_gated_shape& s) {
  const bool situ = s.activation == MOE_ACT_SITU;
  ActArgs a{};
  a.kind = s.activation;
  a.limit = s.swiglu_limit;
  a.beta = s.act_beta;
  a.inv_beta = situ ? 1.0f / s.act_beta : 0.0f;
  a.lb = s.act_linear_beta;
  a.inv_lb = situ ? 1.0f / s.act_linear_beta : 0.0f;
  return a;
}

struct Range {
  const void* p;
  int64_t bytes;
};
// Whether an output meets an input or another output.
template <int NO, int NI>
bool meet(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (const Range& r : in)
      if (overlap(out[i].p, out[i].bytes, r.p, r.bytes)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
  }
  return false;
}

int64_t offsets_bytes(const Product& p) { return (p.E + 1) * 4; }

TileArgs tile_args(const Product& p, const int32_t* offsets) {
  TileArgs a{};
  a.offsets = offsets;
  a.M = static_cast<int>(p.M);
  a.E = static_cast<int>(p.E);
  a.pstride = p.N * p.K;
  a.dtype = p.dtype;
  a.out_dtype = p.dtype;
  a.terms = 1;
  return a;
}

int forward(const Product& p, const void* x, const int32_t* offsets, const void* w, void* out, void* gu,
            const ActArgs* act, void* stream) {
  if (offsets == nullptr && p.E != 1) return MOE_ERR_INVALID;
  if (p.M == 0) return MOE_OK;
  if (x == nullptr || w == nullptr || out == nullptr) return MOE_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(gu, 16) || !aligned(offsets, 4))
    return MOE_ERR_INVALID;
  const int64_t ldx = p.ldx != 0 ? p.ldx : p.K, ldo = p.ldo != 0 ? p.ldo : p.out_cols, so = size_of(p.out_dtype);
  const Range outs[2] = {{out, ((p.M - 1) * ldo + p.out_cols) * so}, {gu, p.M * p.N * 2}};
  const Range ins[2] = {{w, p.E * p.N * p.K * 2}, {offsets, offsets_bytes(p)}};
  if (meet(outs, ins) || overlap(gu, outs[1].bytes, x, ((p.M - 1) * ldx + p.K) * 2) ||
      rows_overlap(x, p.K * 2, ldx * 2, out, p.out_cols * so, ldo * so, p.M))
    return MOE_ERR_INVALID;
  TileArgs a = tile_args(p, offsets);
  a.p = w;
  a.q = x;
  a.out = out;
  a.gu = gu;
  a.R = static_cast<int>(p.out_cols);
  a.I = static_cast<int>(p.K);
  a.ldp = p.K;
  a.ldq = ldx;
  a.ldo = ldo;
  a.out_dtype = p.out_dtype;
  if (act != nullptr) a.act = *act;
  return status(launch_tile_forward(a, act != nullptr, static_cast<hipStream_t>(stream)));
}

// What both backward passes ask of their shape.
int check_backward(const Product& p, const int32_t* offsets) {
  if (p.ldx != 0 || p.ldo != 0 || (offsets == nullptr && p.E != 1)) return MOE_ERR_INVALID;
  // tiles of the rows' gradient (those of the matrices' are below by N * K and E)
  if ((p.M / 16 + p.E + 1) * (p.K / 16 + 1) >= kMaxTileItems) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// dx and dw from the gradient of the product, the sum of `terms` arrays that follow each
// other; either of them null.
int gradients(const Product& p, const void* dout, int terms, const void* x, const int32_t* offsets, const void* w,
              void* dx, void* dw, hipStream_t st) {
  TileArgs row = tile_args(p, offsets);
  row.terms = terms;
  row.qterm = p.M * p.N;
  TileArgs mat = row;
  row.p = w;
  row.q = dout;
  row.out = dx;
  row.R = static_cast<int>(p.K);
  row.I = static_cast<int>(p.N);
  row.ldp = row.ldo = p.K;
  row.ldq = p.N;
  mat.p = x;
  mat.q = dout;
  mat.out = dw;
  mat.R = static_cast<int>(p.K);
  mat.C = static_cast<int>(p.N);
  mat.ldp = mat.ldo = p.K;
  mat.ldq = p.N;
  mat.out_dtype = p.out_dtype;
  const bool rows = dx != nullptr && p.M > 0;
  if (rows && dw != nullptr) return status(launch_tile_gradients(mat, row, st));
  if (rows) return status(launch_tile_row_grad(row, st));
  return dw != nullptr ? status(launch_tile_mat_grad(mat, st)) : MOE_OK;
}

int check(const moe_adapter_shape* s) {
  if (s == nullptr) return MOE_ERR_INVALID;
  if (s->M < 0 || s->N < 1 || s->K < 1 || s->R < 1 || s->A < 1) return MOE_ERR_INVALID;
  if (s->K % 8 != 0 || s->R % 8 != 0 || s->ldx % 8 != 0) return MOE_ERR_INVALID;
  if ((s->ldx != 0 && s->ldx < s->K) || (s->ldb != 0 && s->ldb < s->N) || (s->ldo != 0 && s->ldo < s->N))
    return MOE_ERR_INVALID;
  if (s->M > kMaxSlots || s->N > kMaxLd || s->K > kMaxLd || s->R > 128 || s->A > kMaxExperts || s->ldx > kMaxLd ||
      s->ldb > kMaxLd || s->ldo > kMaxLd || !half_type(s->dtype) ||
      (s->out_dtype != s->dtype && s->out_dtype != MOE_DTYPE_FP32))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// t by part of K; the maps' workspace where it is larger.
uint64_t adapter_ws(const moe_adapter_shape& s) {
  const uint64_t part = static_cast<uint64_t>(adapter_splits(s.M, s.A, s.K, s.R)) * s.M * s.R * 4;
  const uint64_t both = part > maps_ws(s.M, s.A).bytes ? part : maps_ws(s.M, s.A).bytes;
  return (both + 255) / 256 * 256;
}

}  // namespace

extern "C" {

int moe_linear_adapter_query(const moe_adapter_shape* shape, uint64_t* workspace_bytes) {
  if (workspace_bytes == nullptr) return MOE_ERR_INVALID;
  const int rc = check(shape);
  if (rc != MOE_OK) return rc;
  *workspace_bytes = adapter_ws(*shape);
  return MOE_OK;
}

int moe_linear_adapter_maps(const int32_t* ids_dev, const moe_adapter_shape* shape,
                            int32_t* offsets_dev, int32_t* row_slot_dev, int32_t* slot_row_dev,
                            void* workspace_dev, uint64_t workspace_bytes, void* stream) {
  const int rc = check(shape);
  if (rc != MOE_OK) return rc;
  const moe_adapter_shape& s = *shape;
  if (offsets_dev == nullptr || !aligned(offsets_dev, 4) || !aligned(ids_dev, 4) || !aligned(row_slot_dev, 4) ||
      !aligned(slot_row_dev, 4))
    return MOE_ERR_INVALID;
  if (s.M > 0 && (ids_dev == nullptr || row_slot_dev == nullptr || slot_row_dev == nullptr)) return MOE_ERR_INVALID;
  const int64_t map = int64_t{4} * s.M;
  const MapsWs ws = maps_ws(s.M, s.A);
  const Range ids[1] = {{ids_dev, map}};
  const Range maps[3] = {{offsets_dev, (int64_t{s.A} + 1) * 4}, {row_slot_dev, map}, {slot_row_dev, map}};
  if (meet(maps, ids)) return MOE_ERR_INVALID;
  if (workspace_dev == nullptr || !aligned(workspace_dev, 256) || workspace_bytes < ws.bytes) return MOE_ERR_WORKSPACE;
  const Range work[1] = {{workspace_dev, static_cast<int64_t>(ws.bytes)}};
  if (meet(work, ids) || meet(work, maps)) return MOE_ERR_INVALID;
  DispatchArgs a{};
  a.ids = ids_dev;
  a.T = s.M;
  a.E = s.A;
  a.topk = 1;
  a.offsets = offsets_dev;
  a.row_slot = row_slot_dev;
  a.slot_row = slot_row_dev;
  a.range_counts = static_cast<int32_t*>(workspace_dev);
  a.counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace_dev) + ws.counts);
  return status(launch_dispatch(a, static_cast<hipStream_t>(stream)));
}

int moe_linear_adapter(const void* x_dev, const int32_t* offsets_dev, const int32_t* row_slot_dev,
                       const int32_t* slot_row_dev, const void* a_dev, const void* b_dev,
                       const float* scale_dev, const moe_adapter_shape* shape, const void* base_dev,
                       void* out_dev, void* workspace_dev, uint64_t workspace_bytes, void* stream) {
  const int rc = check(shape);
  if (rc != MOE_OK || shape->M == 0) return rc;
  const moe_adapter_shape& s = *shape;
  if (x_dev == nullptr || offsets_dev == nullptr || row_slot_dev == nullptr || slot_row_dev == nullptr ||
      a_dev == nullptr || b_dev == nullptr || out_dev == nullptr)
    return MOE_ERR_INVALID;
  const int64_t so = size_of(s.out_dtype);
  if (!aligned(x_dev, 16) || !aligned(a_dev, 16) || !aligned(b_dev, 16) || !aligned(offsets_dev, 4) ||
      !aligned(row_slot_dev, 4) || !aligned(slot_row_dev, 4) || !aligned(scale_dev, 4) ||
      !aligned(base_dev, static_cast<uintptr_t>(so)) || !aligned(out_dev, static_cast<uintptr_t>(so)))
    return MOE_ERR_INVALID;
  const int64_t ldx = s.ldx != 0 ? s.ldx : s.K, ldb = s.ldb != 0 ? s.ldb : s.N, ldo = s.ldo != 0 ? s.ldo : s.N;
  const int64_t M = s.M, N = s.N, A = s.A, R = s.R;
  const Range out = {out_dev, ((M - 1) * ldo + N) * so};
  const Range ins[6] = {{offsets_dev, (A + 1) * 4}, {row_slot_dev, M * 4}, {slot_row_dev, M * 4},
                        {a_dev, A * R * s.K * 2},   {b_dev, A * N * R * 2}, {scale_dev, A * 4}};
  const Range rows[2] = {{x_dev, ((M - 1) * ldx + s.K) * 2}, {base_dev, ((M - 1) * ldb + N) * so}};
  const Range outs[1] = {out};
  if (meet(outs, ins) || rows_overlap(x_dev, int64_t{s.K} * 2, ldx * 2, out_dev, N * so, ldo * so, M)) return MOE_ERR_INVALID;
  const bool same = base_dev == out_dev && ldb == ldo;
  if (base_dev != nullptr && !same && rows_overlap(base_dev, N * so, ldb * so, out_dev, N * so, ldo * so, M))
    return MOE_ERR_INVALID;
  const int splits = adapter_splits(M, A, s.K, s.R);
  const int64_t bytes = splits * M * R * 4;
  if (workspace_dev == nullptr || !aligned(workspace_dev, 256) || workspace_bytes < static_cast<uint64_t>(bytes))
    return MOE_ERR_WORKSPACE;
  const Range work[1] = {{workspace_dev, bytes}};
  if (meet(work, ins) || meet(work, rows) || meet(work, outs)) return MOE_ERR_INVALID;
  AdapterArgs a{};
  a.x = x_dev;
  a.offsets = offsets_dev;
  a.row_slot = row_slot_dev;
  a.slot_row = slot_row_dev;
  a.a = a_dev;
  a.b = b_dev;
  a.scale = scale_dev;
  a.base = base_dev;
  a.out = out_dev;
  a.part = static_cast<float*>(workspace_dev);
  a.M = s.M;
  a.N = s.N;
  a.K = s.K;
  a.R = s.R;
  a.A = s.A;
  a.splits = splits;
  a.dtype = s.dtype;
  a.out_dtype = s.out_dtype;
  a.ldx = ldx;
  a.ldb = ldb;
  a.ldo = ldo;
  return status(launch_adapter(a, static_cast<hipStream_t>(stream)));
}

int moe_linear_grouped(const void* x_dev, const int32_t* offsets_dev, const void* w_dev,
                       const moe_linear_shape* shape, void* out_dev, void* stream) {
  Product p;
  const int rc = check(shape, p);
  return rc != MOE_OK ? rc : forward(p, x_dev, offsets_dev, w_dev, out_dev, nullptr, nullptr, stream);
}

int moe_linear_grouped_backward(const void* dout_dev, const void* x_dev, const int32_t* offsets_dev,
                                const void* w_dev, const moe_linear_shape* shape, void* dx_dev,
                                void* dw_dev, void* stream) {
  Product p;
  int rc = check(shape, p);
  if (rc == MOE_OK) rc = check_backward(p, offsets_dev);
  if (rc != MOE_OK) return rc;
  if (p.M > 0 && ((dx_dev != nullptr && w_dev == nullptr) || (dw_dev != nullptr && x_dev == nullptr) ||
                  ((dx_dev != nullptr || dw_dev != nullptr) && dout_dev == nullptr)))
    return MOE_ERR_INVALID;
  if (!aligned(dout_dev, 16) || !aligned(x_dev, 16) || !aligned(w_dev, 16) || !aligned(dx_dev, 16) ||
      !aligned(dw_dev, 16) || !aligned(offsets_dev, 4))
    return MOE_ERR_INVALID;
  const int64_t matrices = p.E * p.N * p.K;
  const Range outs[2] = {{dx_dev, p.M * p.K * 2}, {dw_dev, matrices * size_of(p.out_dtype)}};
  const Range ins[4] = {{dout_dev, p.M * p.N * 2},
                        {x_dev, dw_dev != nullptr ? p.M * p.K * 2 : 0},
                        {w_dev, dx_dev != nullptr ? matrices * 2 : 0},
                        {offsets_dev, offsets_bytes(p)}};
  if (meet(outs, ins)) return MOE_ERR_INVALID;
  return gradients(p, dout_dev, 1, x_dev, offsets_dev, w_dev, dx_dev, dw_dev, static_cast<hipStream_t>(stream));
}

int moe_linear_gated(const void* x_dev, const int32_t* offsets_dev, const void* w13_dev,
                     const moe_gated_shape* shape, void* h_dev, void* gu_dev, void* stream) {
  Product p;
  const int rc = check(shape, p);
  if (rc != MOE_OK) return rc;
  const ActArgs act = act_args(*shape);
  return forward(p, x_dev, offsets_dev, w13_dev, h_dev, gu_dev, &act, stream);
}

int moe_linear_gated_backward(const void* dh_dev, const void* x_dev, const int32_t* offsets_dev,
                              const void* gu_dev, const void* w13_dev, const moe_gated_shape* shape,
                              void* dgu_dev, void* dx_dev, void* dw_dev, void* stream) {
  Product p;
  int rc = check(shape, p);
  if (rc == MOE_OK) rc = check_backward(p, offsets_dev);
  if (rc != MOE_OK) return rc;
  if (p.M > 0 && (dh_dev == nullptr || gu_dev == nullptr || dgu_dev == nullptr ||
                  (dx_dev != nullptr && w13_dev == nullptr) || (dw_dev != nullptr && x_dev == nullptr)))
    return MOE_ERR_INVALID;
  if (!aligned(dh_dev, 16) || !aligned(x_dev, 16) || !aligned(gu_dev, 16) || !aligned(w13_dev, 16) ||
      !aligned(dgu_dev, 16) || !aligned(dx_dev, 16) || !aligned(dw_dev, 16) || !aligned(offsets_dev, 4))
    return MOE_ERR_INVALID;
  const int64_t matrices = p.E * p.N * p.K * 2, pre = p.M * p.N * 2, rows = p.M * p.K * 2;
  const int terms = shape->dgu_terms == 2 ? 2 : 1;
  const Range outs[3] = {{dgu_dev, terms * pre}, {dx_dev, rows}, {dw_dev, matrices}};
  const Range ins[5] = {{dh_dev, pre / 2}, {gu_dev, pre}, {x_dev, dw_dev != nullptr ? rows : 0},
                        {w13_dev, dx_dev != nullptr ? matrices : 0}, {offsets_dev, offsets_bytes(p)}};
  if (meet(outs, ins)) return MOE_ERR_INVALID;
  if (p.M > 0) {
    ActGradArgs g{};
    g.dh = dh_dev;
    g.gu = gu_dev;
    g.dgu = dgu_dev;
    g.rest = terms > 1 ? static_cast<uint8_t*>(dgu_dev) + pre : nullptr;
    g.offsets = offsets_dev;
    g.M = shape->M;
    g.I = shape->I;
    g.E = shape->E;
    g.dtype = shape->dtype;
    g.act = act_args(*shape);
    rc = status(launch_act_grad(g, static_cast<hipStream_t>(stream)));
    if (rc != MOE_OK) return rc;
  }
  return gradients(p, dgu_dev, terms, x_dev, offsets_dev, w13_dev, dx_dev, dw_dev, static_cast<hipStream_t>(stream));
}

}  // extern "C"
