// C ABI of the dispatch, combine and 4-bit product operators (moe_ops.h):
// argument checks, then the launches.
#include "common.h"
#include "kernels.h"
#include "moe_ops.h"

using namespace moe;

namespace {

constexpr int64_t kMaxSlots = int64_t{1} << 23;
constexpr int64_t kMaxRowLen = int64_t{1} << 24;  // H, N, ldx, ldo
// T * H: keeps the grids (a one-wave block for 1 KB of a token) within the 2^32
// threads of a launch
constexpr int64_t kMaxElems = int64_t{1} << 33;

bool known_dtype(int d) {
  return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_FP16 || d == MOE_DTYPE_FP32;
}
int64_t size_of(int dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) &&
         y < x + static_cast<uintptr_t>(na);
}

// Rows of two matrices, `rows` of each, na and nb bytes long and sa and sb apart. With
// the same stride the rows of the one may lie between those of the other; with
// different ones the ranges decide.
bool rows_overlap(const void* a, int64_t na, int64_t sa, const void* b, int64_t nb, int64_t sb,
                  int64_t rows) {
  if (!overlap(a, (rows - 1) * sa + na, b, (rows - 1) * sb + nb)) return false;
  if (sa != sb) return true;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const int64_t at = (d % sa + sa) % sa;  // from a row of a to the next row of b
  return at < na || at + nb > sa;
}

int check(const moe_ops_dispatch_shape* s) {
  if (s == nullptr) return MOE_ERR_INVALID;
  if (s->T < 0 || s->E < 1 || s->topk < 1 || s->H < 1 || s->expert_offset < 0)
    return MOE_ERR_INVALID;
  if (s->topk > kMaxTopK || s->E > kMaxExperts || s->H > kMaxRowLen || !known_dtype(s->dtype))
    return MOE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s->T) * s->topk > kMaxSlots ||
      static_cast<int64_t>(s->T) * s->H > kMaxElems)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct DispatchWs {
  uint64_t counts, bytes;  // range counts at 0
};
DispatchWs dispatch_ws(const moe_ops_dispatch_shape& s) {
  const uint64_t slots = static_cast<uint64_t>(s.T) * s.topk;
  if (slots <= static_cast<uint64_t>(kFusedSlots)) return {0, 256};
  const uint64_t len = map_range_slots(static_cast<int64_t>(slots));
  const uint64_t ranges = (slots + len - 1) / len;
  const uint64_t counts = (ranges * s.E * 4 + 255) / 256 * 256;
  return {counts, counts + (static_cast<uint64_t>(s.E) * 4 + 255) / 256 * 256};
}

int status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Bytes of the token and slot arrays of a shape.
struct Extents {
  int64_t tokens, rows, map;
  explicit Extents(const moe_ops_dispatch_shape& s)
      : tokens(static_cast<int64_t>(s.T) * s.H * size_of(s.dtype)),
        rows(tokens * s.topk),
        map(static_cast<int64_t>(s.T) * s.topk * 4) {}
};

// The forward sum of combine and dispatch's gradient.
int combine_impl(const void* rows, const int32_t* slot_row, const float* w, bool weighted,
                 const moe_ops_dispatch_shape* shape, void* out, void* stream) {
  const int rc = check(shape);
  if (rc != MOE_OK || shape->T == 0) return rc;
  const moe_ops_dispatch_shape& s = *shape;
  const uintptr_t al = static_cast<uintptr_t>(size_of(s.dtype));
  if (rows == nullptr || slot_row == nullptr || out == nullptr || (weighted && w == nullptr))
    return MOE_ERR_INVALID;
  if (!aligned(rows, al) || !aligned(out, al) || !aligned(slot_row, 4) || !aligned(w, 4))
    return MOE_ERR_INVALID;
  const Extents n(s);
  if (overlap(out, n.tokens, rows, n.rows) || overlap(out, n.tokens, slot_row, n.map) ||
      overlap(out, n.tokens, w, n.map))
    return MOE_ERR_INVALID;
  CombineArgs a{};
  a.rows = static_cast<const uint8_t*>(rows);
  a.slot_row = slot_row;
  a.topk_w = w;
  a.T = s.T;
  a.topk = s.topk;
  a.H = s.H;
  a.dtype = s.dtype;
  a.out = static_cast<uint8_t*>(out);
  return status(launch_combine(a, static_cast<hipStream_t>(stream)));
}

int check_w4(const moe_ops_w4_shape* s) {
  if (s == nullptr) return MOE_ERR_INVALID;
  if (s->M < 0 || s->N < 1 || s->K < 1 || s->E < 1) return MOE_ERR_INVALID;
  if ((s->ldx != 0 && s->ldx < s->K) || (s->ldo != 0 && s->ldo < s->N)) return MOE_ERR_INVALID;
  if (s->ldx % 8 != 0) return MOE_ERR_INVALID;
  if (s->K % 128 != 0 || s->K > kMaxTiledK || s->N > kMaxRowLen || s->M > kMaxSlots ||
      s->E > kMaxExperts || s->ldx > kMaxRowLen || s->ldo > kMaxRowLen)
    return MOE_ERR_UNSUPPORTED;
  if (s->format == MOE_W4_MXFP4) {
    if (s->group != 32) return MOE_ERR_UNSUPPORTED;
  } else if (s->format == MOE_W4_INT4) {
    if (s->group != 32 && s->group != 64 && s->group != 128) return MOE_ERR_UNSUPPORTED;
  } else {
    return MOE_ERR_UNSUPPORTED;
  }
  if (s->dtype != MOE_DTYPE_BF16 && s->dtype != MOE_DTYPE_FP16) return MOE_ERR_UNSUPPORTED;
  if (!known_dtype(s->out_dtype)) return MOE_ERR_UNSUPPORTED;
  // work items (row tiles x weight sets) are counted in 32 bits
  if ((static_cast<int64_t>(s->M) / 16 + s->E + 1) * (static_cast<int64_t>(s->N) / 16 + 1) >=
      kW4MaxItems)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int w4_impl(const void* x, const int32_t* offsets, bool grouped, const uint8_t* w,
            const void* scales, const uint8_t* zeros, const void* bias,
            const moe_ops_w4_shape* shape, void* out, void* stream) {
  const int rc = check_w4(shape);
  if (rc != MOE_OK) return rc;
  const moe_ops_w4_shape& s = *shape;
  if (!grouped && s.E != 1) return MOE_ERR_INVALID;
  if (zeros != nullptr && s.format == MOE_W4_MXFP4) return MOE_ERR_INVALID;
  if (s.M == 0) return MOE_OK;
  if (x == nullptr || w == nullptr || scales == nullptr || out == nullptr ||
      (grouped && offsets == nullptr))
    return MOE_ERR_INVALID;
  // vector loads of x and w; scales and zero points in dwords where a K step
  // has four bytes of them or more
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(scales, 4) || !aligned(zeros, 4) ||
      !aligned(bias, 2) || !aligned(out, static_cast<uintptr_t>(size_of(s.out_dtype))) ||
      !aligned(offsets, 4))
    return MOE_ERR_INVALID;
  const int64_t ldx = s.ldx != 0 ? s.ldx : s.K, ldo = s.ldo != 0 ? s.ldo : s.N;
  const int64_t osize = size_of(s.out_dtype), no = ((s.M - 1) * ldo + s.N) * osize;
  const int64_t np = (static_cast<int64_t>(s.N) + 15) / 16 * 16;
  const int64_t ngroup = static_cast<int64_t>(s.E) * s.N * (s.K / s.group);
  if (rows_overlap(x, static_cast<int64_t>(s.K) * 2, ldx * 2, out, s.N * osize, ldo * osize, s.M) ||
      overlap(out, no, w, s.E * np * (s.K / 2)) ||
      overlap(out, no, scales, ngroup * (s.format == MOE_W4_MXFP4 ? 1 : 2)) ||
      overlap(out, no, zeros, ngroup) || overlap(out, no, bias, static_cast<int64_t>(s.E) * s.N * 2) ||
      overlap(out, no, offsets, (static_cast<int64_t>(s.E) + 1) * 4))
    return MOE_ERR_INVALID;
  W4Args a{};
  a.x = x;
  a.offsets = grouped ? offsets : nullptr;
  a.w = w;
  a.scales = scales;
  a.zeros = zeros;
  a.bias = bias;
  a.out = out;
  a.M = s.M;
  a.N = s.N;
  a.K = s.K;
  a.E = s.E;
  a.format = s.format;
  a.group = s.group;
  a.dtype = s.dtype;
  a.out_dtype = s.out_dtype;
  a.ldx = ldx;
  a.ldo = ldo;
  return status(launch_w4(a, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int moe_ops_dispatch_query(const moe_ops_dispatch_shape* shape, uint64_t* workspace_bytes) {
  if (workspace_bytes == nullptr) return MOE_ERR_INVALID;
  const int rc = check(shape);
  if (rc != MOE_OK) return rc;
  *workspace_bytes = dispatch_ws(*shape).bytes;
  return MOE_OK;
}

int moe_ops_dispatch(const void* x_dev, const int32_t* topk_ids_dev,
                     const moe_ops_dispatch_shape* shape, void* rows_dev, int32_t* offsets_dev,
                     int32_t* row_slot_dev, int32_t* slot_row_dev, void* workspace_dev,
                     uint64_t workspace_bytes, void* stream) {
  const int rc = check(shape);
  if (rc != MOE_OK) return rc;
  const moe_ops_dispatch_shape& s = *shape;
  const uintptr_t al = static_cast<uintptr_t>(size_of(s.dtype));
  if (offsets_dev == nullptr || !aligned(offsets_dev, 4)) return MOE_ERR_INVALID;
  struct Range {
    const void* p;
    int64_t bytes;
  };
  const Extents n(s);
  const Range in[2] = {{x_dev, n.tokens}, {topk_ids_dev, n.map}};
  const Range out[4] = {{rows_dev, n.rows}, {offsets_dev, (static_cast<int64_t>(s.E) + 1) * 4},
                        {row_slot_dev, n.map}, {slot_row_dev, n.map}};
  const auto meet = [](const Range& a, const Range& b) { return overlap(a.p, a.bytes, b.p, b.bytes); };
  if (s.T > 0) {
    if (x_dev == nullptr || topk_ids_dev == nullptr || rows_dev == nullptr ||
        row_slot_dev == nullptr || slot_row_dev == nullptr)
      return MOE_ERR_INVALID;
    if (!aligned(x_dev, al) || !aligned(rows_dev, al) || !aligned(topk_ids_dev, 4) ||
        !aligned(row_slot_dev, 4) || !aligned(slot_row_dev, 4))
      return MOE_ERR_INVALID;
    for (int i = 0; i < 4; ++i) {
      if (meet(out[i], in[0]) || meet(out[i], in[1])) return MOE_ERR_INVALID;
      for (int j = 0; j < i; ++j)
        if (meet(out[i], out[j])) return MOE_ERR_INVALID;
    }
  }
  const DispatchWs ws = dispatch_ws(s);
  if (workspace_dev == nullptr || !aligned(workspace_dev, 256) || workspace_bytes < ws.bytes)
    return MOE_ERR_WORKSPACE;
  const Range work = {workspace_dev, static_cast<int64_t>(ws.bytes)};
  for (const Range& r : in)
    if (meet(work, r)) return MOE_ERR_INVALID;
  for (const Range& r : out)
    if (meet(work, r)) return MOE_ERR_INVALID;
  DispatchArgs a{};
  a.x = static_cast<const uint8_t*>(x_dev);
  a.ids = topk_ids_dev;
  a.T = s.T;
  a.E = s.E;
  a.topk = s.topk;
  a.H = s.H;
  a.expert_offset = s.expert_offset;
  a.elem = static_cast<int>(al);
  a.rows = static_cast<uint8_t*>(rows_dev);
  a.offsets = offsets_dev;
  a.row_slot = row_slot_dev;
  a.slot_row = slot_row_dev;
  a.range_counts = static_cast<int32_t*>(workspace_dev);
  a.counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace_dev) + ws.counts);
  return status(launch_dispatch(a, static_cast<hipStream_t>(stream)));
}

int moe_ops_dispatch_backward(const void* drows_dev, const int32_t* slot_row_dev,
                              const moe_ops_dispatch_shape* shape, void* dx_dev, void* stream) {
  return combine_impl(drows_dev, slot_row_dev, nullptr, false, shape, dx_dev, stream);
}

int moe_ops_combine(const void* rows_dev, const int32_t* slot_row_dev, const float* topk_w_dev,
                    const moe_ops_dispatch_shape* shape, void* out_dev, void* stream) {
  return combine_impl(rows_dev, slot_row_dev, topk_w_dev, true, shape, out_dev, stream);
}

int moe_ops_combine_backward(const void* dout_dev, const void* rows_dev,
                             const int32_t* slot_row_dev, const float* topk_w_dev,
                             const moe_ops_dispatch_shape* shape, void* drows_dev,
                             float* dtopk_w_dev, void* stream) {
  const int rc = check(shape);
  if (rc != MOE_OK || shape->T == 0) return rc;
  const moe_ops_dispatch_shape& s = *shape;
  const uintptr_t al = static_cast<uintptr_t>(size_of(s.dtype));
  if (dout_dev == nullptr || rows_dev == nullptr || slot_row_dev == nullptr ||
      topk_w_dev == nullptr || drows_dev == nullptr || dtopk_w_dev == nullptr)
    return MOE_ERR_INVALID;
  if (!aligned(dout_dev, al) || !aligned(rows_dev, al) || !aligned(drows_dev, al) ||
      !aligned(slot_row_dev, 4) || !aligned(topk_w_dev, 4) || !aligned(dtopk_w_dev, 4))
    return MOE_ERR_INVALID;
  const Extents n(s);
  const void* in[4] = {dout_dev, rows_dev, slot_row_dev, topk_w_dev};
  const int64_t nin[4] = {n.tokens, n.rows, n.map, n.map};
  for (int i = 0; i < 4; ++i)
    if (overlap(drows_dev, n.rows, in[i], nin[i]) || overlap(dtopk_w_dev, n.map, in[i], nin[i]))
      return MOE_ERR_INVALID;
  if (overlap(drows_dev, n.rows, dtopk_w_dev, n.map)) return MOE_ERR_INVALID;
  CombineArgs a{};
  a.dout = static_cast<const uint8_t*>(dout_dev);
  a.rows = static_cast<const uint8_t*>(rows_dev);
  a.slot_row = slot_row_dev;
  a.topk_w = topk_w_dev;
  a.T = s.T;
  a.topk = s.topk;
  a.H = s.H;
  a.dtype = s.dtype;
  a.out = static_cast<uint8_t*>(drows_dev);
  a.dtopk_w = dtopk_w_dev;
  return status(launch_combine_backward(a, static_cast<hipStream_t>(stream)));
}

int moe_ops_w4_linear(const void* x_dev, const uint8_t* w_dev, const void* scales_dev,
                      const uint8_t* zeros_dev, const void* bias_dev,
                      const moe_ops_w4_shape* shape, void* out_dev, void* stream) {
  return w4_impl(x_dev, nullptr, false, w_dev, scales_dev, zeros_dev, bias_dev, shape, out_dev,
                 stream);
}

int moe_ops_w4_grouped_linear(const void* x_dev, const int32_t* offsets_dev, const uint8_t* w_dev,
                              const void* scales_dev, const uint8_t* zeros_dev,
                              const void* bias_dev, const moe_ops_w4_shape* shape, void* out_dev,
                              void* stream) {
  return w4_impl(x_dev, offsets_dev, true, w_dev, scales_dev, zeros_dev, bias_dev, shape, out_dev,
                 stream);
}

}  // extern "C"
