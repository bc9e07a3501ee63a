/*
 * moe_linear.h - C ABI of the 16-bit products around the expert layer for AMD
 * Instinct MI355X (gfx950), in the same library as moe_mxfp4.h and moe_ops.h:
 *
 *   - moe_linear_grouped: rows times their expert's matrix (or one matrix for
 *     all rows), and its gradients;
 *   - moe_linear_gated: rows times their expert's gate and up matrices, the
 *     activation and the product in one kernel, and its gradients;
 *   - moe_linear_adapter: low-rank products of many requests, each row with its
 *     adapter, added to a shared projection's result.
 *
 * With dispatch and combine of moe_ops.h the first two are the routed part of
 * a layer that trains; the third goes beside any projection, the 4-bit ones of
 * moe_ops.h among them.
 *
 * Conventions as in moe_ops.h: pointers named *_dev are device pointers owned
 * by the caller; no function allocates, synchronises or reads device memory
 * from the host, so every call can be captured in a graph; shapes are passed by
 * host pointer and read during the call only; every function returns MOE_OK or
 * an MOE_ERR_* code, and argument errors come before anything is enqueued;
 * `stream` is a hipStream_t of the current device (NULL: its default stream).
 * Outputs must not overlap inputs or each other (MOE_ERR_INVALID where their
 * ranges do; rows of x and out that are the same number of bytes apart may lie
 * between each other, as columns of one matrix). Types are MOE_DTYPE_* of
 * moe_ops.h. Every sum is held in 32 bits and rounded once, to the nearest
 * even. All calls are deterministic.
 */
#ifndef MOE_LINEAR_H
#define MOE_LINEAR_H

#include "moe_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Shape of the grouped product out[m, n] = sum over k of x[m, k] w[e, n, k],
 * e the expert of row m.
 *
 *   M          rows of x and out (0 allowed)
 *   N, K       rows and columns of a matrix, multiples of 8
 *   E          matrices, 1..2048
 *   dtype      MOE_DTYPE_BF16 or MOE_DTYPE_FP16: x, w and dx
 *   out_dtype  dtype or MOE_DTYPE_FP32: out, or in the backward pass dw
 *   ldx, ldo   elements from one row of x / out to the next, multiples of 8;
 *              0 stands for K / N. The backward pass takes 0 alone.
 */
typedef struct moe_linear_shape {
  int32_t M;
  int32_t N;
  int32_t K;
  int32_t E;
  int32_t dtype;
  int32_t out_dtype;
  int64_t ldx;
  int64_t ldo;
} moe_linear_shape;

/*
 * x_dev [M, K], w_dev [E, N, K], out_dev [M, N]; every array 16-byte aligned.
 * offsets_dev: int32 [E + 1], non-decreasing from >= 0, as moe_ops_dispatch
 * writes them: rows [offsets[e], offsets[e + 1]) are expert e's; values past M
 * count as M. NULL with E = 1: all rows. Rows of out that no expert owns are
 * left as they were, those of x are not read.
 *
 * MOE_ERR_INVALID: null or misaligned pointers, sizes below their range, N, K
 * or a stride that is no multiple of 8, strides shorter than a row, overlaps,
 * offsets NULL with E > 1; MOE_ERR_UNSUPPORTED: M > 2^23, N, K or a stride
 * > 2^20, N * K > 2^30, E > 2048, unknown type, (M / 16 + E + 1) * (N / 16 + 1)
 * >= 2^30.
 */
int moe_linear_grouped(const void* x_dev, const int32_t* offsets_dev, const void* w_dev,
                       const moe_linear_shape* shape, void* out_dev, void* stream);

/*
 * Gradients from dout [M, N] (dtype):
 *   dx[m, k] = sum over n of dout[m, n] w[e, n, k]      (dtype; rows that no
 *       expert owns are left as they were)
 *   dw[e, n, k] = sum over the rows m of e of dout[m, n] x[m, k]  (out_dtype;
 *       zeros for an expert without rows)
 * dx_dev or dw_dev NULL: not computed (and w, or x, may be NULL), the other
 * with the same bits. Besides the above MOE_ERR_UNSUPPORTED: (M / 16 + E + 1) *
 * (K / 16 + 1) >= 2^30.
 */
int moe_linear_grouped_backward(const void* dout_dev, const void* x_dev, const int32_t* offsets_dev,
                                const void* w_dev, const moe_linear_shape* shape, void* dx_dev,
                                void* dw_dev, void* stream);

/*
 * Shape of the gated product h = act(g, u), g[m, i] = sum over k of x[m, k]
 * w13[e, i, k], u[m, i] the same with w13[e, I + i, k].
 *
 *   M, E, dtype  as above (x, w13, h, the pre-activations and all gradients)
 *   I, H         features of h and elements of a row of x, multiples of 8
 *   activation, swiglu_limit, act_beta, act_linear_beta
 *                as in moe_mxfp4_shape; the sums enter it in 32 bits. The clamp of
 *                swiglu_limit cuts infinities off and leaves NaN NaN
 *   dgu_terms    1, or 0 which stands for it, or 2: the values of dtype whose sum
 *                the backward pass keeps the gradient of the pre-activations as
 *   ldx, ldo     elements from one row of x / h to the next, multiples of 8; 0
 *                stands for H / I. The backward pass takes 0 alone.
 */
typedef struct moe_gated_shape {
  int32_t M;
  int32_t I;
  int32_t H;
  int32_t E;
  int32_t dtype;
  int32_t activation;
  float swiglu_limit;
  float act_beta;
  float act_linear_beta;
  int32_t dgu_terms;
  int64_t ldx;
  int64_t ldo;
} moe_gated_shape;

/*
 * x_dev [M, H], offsets_dev as above, w13_dev [E, 2 I, H] (rows [0, I) gate,
 * [I, 2 I) up), h_dev [M, I]. gu_dev [M, 2 I], or NULL: the pre-activations (g,
 * then u, of each row), rounded to dtype, for the backward pass. Rows that no
 * expert owns are left as they were in both. Errors as above with N = 2 I,
 * K = H, and MOE_ERR_INVALID for values of the activation's that
 * moe_mxfp4_query refuses.
 */
int moe_linear_gated(const void* x_dev, const int32_t* offsets_dev, const void* w13_dev,
                     const moe_gated_shape* shape, void* h_dev, void* gu_dev, void* stream);

/*
 * Gradients from dh [M, I] at the pre-activations gu [M, 2 I]:
 *   dgu[m, (g, u)] = dh times the derivative of act, rounded to dtype; 0 where
 *       the clamp of swiglu_limit > 0 cut off (g > L, |u| > L; on the limit and
 *       for NaN it does not)
 *   dx = dgu w13 and dw13 = dgu^T x, as moe_linear_grouped_backward
 * dgu_dev [M, 2 I] is written, and read, in the rows that experts own: the
 * caller's scratch, or the gradient of the pre-activations. dx_dev or dw_dev
 * NULL: not computed.
 *
 * Rounding dgu once makes dx and dw about 1.4 times as far off as their own
 * rounding does. With dgu_terms 2 dgu_dev is [2, M, 2 I], the second array what
 * the rounding to the first left, rounded too: their sum is dgu to 2^-16 of it
 * (bf16) or 2^-22 (fp16; 2^-25 where that is more), and both products take
 * both, in one and a half to two times the time.
 */
int moe_linear_gated_backward(const void* dh_dev, const void* x_dev, const int32_t* offsets_dev,
                              const void* gu_dev, const void* w13_dev, const moe_gated_shape* shape,
                              void* dgu_dev, void* dx_dev, void* dw_dev, void* stream);

/*
 * Shape of the adapters' product out[m, n] = base[m, n] + scale[i] * sum over r
 * of t[m, r] b[i, n, r], t[m, r] = sum over k of x[m, k] a[i, r, k], i the
 * adapter of row m; a row without one gets base[m, n].
 *
 *   M             rows (0 allowed), up to 2^23
 *   N             elements of a row of out, 1..2^20: any length
 *   K             elements of a row of x, a multiple of 8 up to 2^20
 *   R             rank: a multiple of 8, 8..128 (adapters of lower rank end in
 *                 zeros)
 *   A             adapters, 1..2048
 *   dtype         MOE_DTYPE_BF16 or MOE_DTYPE_FP16: x, a and b
 *   out_dtype     dtype or MOE_DTYPE_FP32: base and out
 *   ldx, ldb, ldo elements from one row of x / base / out to the next; 0 stands
 *                 for K / N / N; ldx a multiple of 8; each up to 2^20
 *
 * t is held in 32 bits and enters the second product as two values of dtype
 * whose sum is t to 2^-16 of it in bf16 and in fp16 to 2^-22 of it, or 2^-25 of
 * the row's largest |t| where that is more; or as three, to 2^-24, where dtype
 * is bf16 and out_dtype fp32. An infinity in b gives infinities or NaN.
 */
typedef struct moe_adapter_shape {
  int32_t M;
  int32_t N;
  int32_t K;
  int32_t R;
  int32_t A;
  int32_t dtype;
  int32_t out_dtype;
  int64_t ldx;
  int64_t ldb;
  int64_t ldo;
} moe_adapter_shape;

/*
 * Check a shape and return the workspace bytes of both calls below (at least
 * 256). Host only. MOE_ERR_INVALID: null pointer, sizes below their range, K, R
 * or ldx no multiple of 8, strides shorter than a row; MOE_ERR_UNSUPPORTED:
 * sizes above theirs, unknown type.
 */
int moe_linear_adapter_query(const moe_adapter_shape* shape, uint64_t* workspace_bytes);

/*
 * Maps that sort the rows by adapter, for all calls with the same ids. ids_dev
 * int32 [M]: a row's adapter, any value outside [0, A) for none. offsets_dev
 * int32 [A + 1], row_slot_dev and slot_row_dev int32 [M]: as moe_ops_dispatch
 * writes them for one column, row_slot's entries from offsets[A] on left as
 * they were. Errors as moe_ops_dispatch.
 */
int moe_linear_adapter_maps(const int32_t* ids_dev, const moe_adapter_shape* shape,
                            int32_t* offsets_dev, int32_t* row_slot_dev, int32_t* slot_row_dev,
                            void* workspace_dev, uint64_t workspace_bytes, void* stream);

/*
 * x_dev [M, K] and a_dev [A, R, K], b_dev [A, N, R] 16-byte aligned; scale_dev
 * float [A], or NULL: 1; base_dev [M, N], or NULL: 0; out_dev [M, N], which may
 * be base_dev with the same stride (rows without an adapter are then not
 * touched). Entries of row_slot outside [0, M) are left out. Alignment: base
 * and out their element size, maps and scale 4 bytes, workspace 256 bytes.
 *
 * MOE_ERR_WORKSPACE: workspace NULL, too small or misaligned; MOE_ERR_INVALID:
 * null or misaligned pointers, out overlapping an input (base apart, as above)
 * or the workspace anything. Calls that may overlap in time need workspaces of
 * their own.
 */
int moe_linear_adapter(const void* x_dev, const int32_t* offsets_dev, const int32_t* row_slot_dev,
                       const int32_t* slot_row_dev, const void* a_dev, const void* b_dev,
                       const float* scale_dev, const moe_adapter_shape* shape, const void* base_dev,
                       void* out_dev, void* workspace_dev, uint64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LINEAR_H */
