/*
 * moe_ops.h - C ABI of the operators around the expert layer for AMD
 * Instinct MI355X (gfx950), in the same library as moe_mxfp4.h:
 *
 *   - dispatch: token rows copied into expert order, with the maps there and
 *     back, and the gradient of the tokens;
 *   - combine: expert rows weighted and summed back to token order, and the
 *     gradients of the rows and of the routing weights;
 *   - w4_linear: a few tokens times one 4-bit weight matrix with group scales;
 *   - w4_grouped_linear: the rows that dispatch sorted, each times its
 *     expert's 4-bit weight matrix.
 *
 * They are the steps of moe_mxfp4_forward as operators of their own, for
 * programs that train the routed part, put other products or activations
 * between the steps, or hold 4-bit weights outside the layer.
 *
 * Conventions, as in moe_mxfp4.h: pointers named *_dev are device pointers
 * owned by the caller; no function allocates, synchronises or reads device
 * memory from the host, so every call can be captured in a graph; shapes are
 * passed by host pointer and read during the call only; every function
 * returns MOE_OK or an MOE_ERR_* code of moe_mxfp4.h, and argument errors
 * come before anything is enqueued. `stream` is a hipStream_t of the current
 * device (NULL: its default stream); the pointers must be usable there.
 * Outputs must not overlap inputs or each other (MOE_ERR_INVALID where their
 * ranges do; rows of the products' x and out that are the same number of bytes
 * apart may lie between each other, as columns of one matrix). Nothing of a
 * call is kept for the next; the products keep how many blocks of a kernel a
 * GPU holds.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of tokens, rows and results. */
#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_FP16 1
#define MOE_DTYPE_FP32 2

/*
 * Shape of dispatch and combine.
 *
 *   T              tokens (0 allowed)
 *   E              local experts, 1..2048
 *   topk           columns (slots) per token, 1..32
 *   H              elements per token row, >= 1: any length; rows whose byte
 *                  length is a multiple of 16 run fastest
 *   expert_offset  global id of local expert 0, >= 0
 *   dtype          MOE_DTYPE_* of the rows; sums are held in 32 bits and
 *                  rounded once, to the nearest even
 *
 * T * topk is at most 2^23 slots, T * H at most 2^33. Slot t * topk + k is column k of token t.
 */
typedef struct moe_ops_dispatch_shape {
  int32_t T;
  int32_t E;
  int32_t topk;
  int32_t H;
  int32_t expert_offset;
  int32_t dtype;
} moe_ops_dispatch_shape;

/*
 * Check a shape and return the workspace bytes that moe_ops_dispatch needs
 * (at least 256). Host only. MOE_ERR_INVALID: null pointer, T < 0, E, topk or
 * H < 1, expert_offset < 0; MOE_ERR_UNSUPPORTED: topk > 32, E > 2048,
 * T * topk > 2^23, H > 2^24, T * H > 2^33, unknown dtype.
 */
int moe_ops_dispatch_query(const moe_ops_dispatch_shape* shape, uint64_t* workspace_bytes);

/*
 * Tokens into expert order. A slot whose id lies in [expert_offset,
 * expert_offset + E) gets a row; any other id (-1 among them) gets none. Rows
 * are ordered by expert, within an expert by slot; every slot with a row gets
 * its own, also where a token names an expert twice. With R rows in all:
 *
 *   x_dev         [T, H]            tokens
 *   topk_ids_dev  int32 [T, topk]   global expert ids
 *   rows_dev      [T * topk, H]     row r is the token of slot row_slot[r];
 *                                   rows from R on are left as they were
 *   offsets_dev   int32 [E + 1]     first row of each expert; offsets[E] = R
 *   row_slot_dev  int32 [T * topk]  row -> slot; entries from R on are left
 *                                   as they were
 *   slot_row_dev  int32 [T, topk]   slot -> row, or -1
 *
 * Deterministic. T = 0 writes zeros to offsets and reads nothing. Alignment:
 * rows their element size, maps 4 bytes, workspace 256 bytes.
 * MOE_ERR_WORKSPACE: workspace NULL, too small or misaligned; MOE_ERR_INVALID:
 * its first bytes, as many as are needed, on an input or output. Calls that
 * may overlap in time need workspaces of their own (two captured graphs that
 * can run at once among them).
 */
int moe_ops_dispatch(const void* x_dev, const int32_t* topk_ids_dev,
                     const moe_ops_dispatch_shape* shape, void* rows_dev, int32_t* offsets_dev,
                     int32_t* row_slot_dev, int32_t* slot_row_dev, void* workspace_dev,
                     uint64_t workspace_bytes, void* stream);

/*
 * Gradient of dispatch: dx[t] = sum over k of drows[slot_row[t, k]], columns
 * without a row adding nothing (a token without any gets zeros). slot_row as
 * moe_ops_dispatch wrote it; entries outside [0, T * topk) count as -1. Rows
 * that no slot names are not read.
 */
int moe_ops_dispatch_backward(const void* drows_dev, const int32_t* slot_row_dev,
                              const moe_ops_dispatch_shape* shape, void* dx_dev, void* stream);

/*
 * Rows back to token order: out[t] = sum over k of w[t, k] *
 * rows[slot_row[t, k]], in ascending k; columns without a row add nothing,
 * whatever their weight. rows [T * topk, H], topk_w float [T, topk], out
 * [T, H].
 */
int moe_ops_combine(const void* rows_dev, const int32_t* slot_row_dev, const float* topk_w_dev,
                    const moe_ops_dispatch_shape* shape, void* out_dev, void* stream);

/*
 * Gradients of combine from dout [T, H]:
 *   drows[slot_row[t, k]] = w[t, k] * dout[t]          (rows that no slot
 *       names are left as they were)
 *   dtopk_w[t, k] = <dout[t], rows[slot_row[t, k]]>    (float; 0 without a row)
 * Two slots must not name the same row (dispatch never makes such a map).
 */
int moe_ops_combine_backward(const void* dout_dev, const void* rows_dev,
                             const int32_t* slot_row_dev, const float* topk_w_dev,
                             const moe_ops_dispatch_shape* shape, void* drows_dev,
                             float* dtopk_w_dev, void* stream);

/* 4-bit weight formats: a weight is scale * (value of its code). */
#define MOE_W4_MXFP4 0 /* E2M1 codes; an E8M0 scale byte for 32 weights along K
                          (byte 255 is NaN), as the layer's weights */
#define MOE_W4_INT4 1  /* codes 0..15 minus a zero point; a scale in the tokens'
                          type for each group of 32, 64 or 128 along K */

/*
 * Shape of the 4-bit products: out[m, n] = bias[n] + sum over k of
 * x[m, k] * weight[n, k].
 *
 *   M          rows of x and out (0 allowed)
 *   N          weight rows, 1..2^24
 *   K          inner length, a multiple of 128 up to 8192
 *   E          matrices: 1 for w4_linear, the experts (1..2048) for
 *              w4_grouped_linear
 *   format     MOE_W4_MXFP4 or MOE_W4_INT4
 *   group      weights that share a scale: 32 (MXFP4), 32, 64 or 128 (INT4)
 *   dtype      MOE_DTYPE_BF16 or MOE_DTYPE_FP16: x, bias and the INT4 scales
 *   out_dtype  MOE_DTYPE_*: the result, rounded once from 32 bits
 *   ldx, ldo   elements from one row of x / out to the next; 0 stands for K / N
 *
 * The products are exact in 32 bits before they are summed, whatever the
 * format: codes are exact in the tokens' type and a group's scale meets its
 * sum in 32 bits. With bfloat16 tokens MXFP4 scales are applied to the codes,
 * which is exact too: scale bytes up to 252 (then no weight passes the
 * type's range; bytes 253 and 254 may give infinities). INT4 zero points come
 * off a group's sum: the 32-bit rounding goes by the sum of |s| (c + z) |x|, not
 * |s| |c - z| |x|, so weights that equal their zero points need not give exactly
 * 0, and NaN comes out where x is infinite or s times the sum of c x or of z x
 * passes the 32-bit range.
 *
 * Deterministic. For one shape a row's result depends, to the bit, on the row and
 * its matrix alone: not on its place in x, nor on the other rows and their experts.
 * Another shape (M among its fields) may sum in another order.
 */
typedef struct moe_ops_w4_shape {
  int32_t M;
  int32_t N;
  int32_t K;
  int32_t E;
  int32_t format;
  int32_t group;
  int32_t dtype;
  int32_t out_dtype;
  int64_t ldx;
  int64_t ldo;
} moe_ops_w4_shape;

/*
 * A few tokens times one matrix (E = 1). Made for decode: the weights are
 * read once for up to 64 rows of x (INT4 with groups of 32: 16, beyond 32 rows);
 * more rows are taken that many at a time.
 *
 *   x_dev       [M, K] rows ldx apart, 16-byte aligned, ldx % 8 == 0
 *   w_dev       uint8 [Np, K / 2], Np = N rounded up to 16: two codes a byte,
 *               the even K in the low nibble, in the packed layout of
 *               moe_mxfp4_prepack (rows from N on may hold anything)
 *   scales_dev  uint8 [N, K / 32] E8M0 (MXFP4) or dtype [N, K / group] (INT4),
 *               row-major, 4-byte aligned
 *   zeros_dev   uint8 [N, K / group] zero points (INT4; 4-byte aligned), or
 *               NULL: 8
 *   bias_dev    dtype [N], or NULL
 *   out_dev     out_dtype [M, N] rows ldo apart; nothing between them is written
 *
 * MOE_ERR_INVALID: null or misaligned pointers, sizes below their range,
 * strides shorter than a row, ldx % 8, zeros with MXFP4, E != 1;
 * MOE_ERR_UNSUPPORTED: K % 128, K > 8192, N, ldx or ldo > 2^24, M > 2^23,
 * (M / 16 + E + 1) * (N / 16 + 1) >= 2^30, unknown format, group or type.
 */
int moe_ops_w4_linear(const void* x_dev, const uint8_t* w_dev, const void* scales_dev,
                      const uint8_t* zeros_dev, const void* bias_dev,
                      const moe_ops_w4_shape* shape, void* out_dev, void* stream);

/*
 * Rows times their expert's matrix: row r of x in [offsets[e],
 * offsets[e + 1]) with matrix e. offsets int32 [E + 1], non-decreasing from
 * >= 0, as moe_ops_dispatch writes them; values past M count as M. Rows of out
 * that no expert owns are left as they were, those of x are not read.
 * w [E, Np, K / 2], scales and zeros [E, N, K / group], bias [E, N]: the
 * matrices of w4_linear one after another. Meant for few rows an expert: an
 * expert's weights are read once for 16 of its rows (64 where M / E is large).
 */
int moe_ops_w4_grouped_linear(const void* x_dev, const int32_t* offsets_dev, const uint8_t* w_dev,
                              const void* scales_dev, const uint8_t* zeros_dev,
                              const void* bias_dev, const moe_ops_w4_shape* shape, void* out_dev,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
