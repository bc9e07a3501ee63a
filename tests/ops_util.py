"""References in 64 bits for the dispatch, combine and 4-bit product operators,
written from their definitions (loops over slots and experts), and the bounds
their tests hold the kernels to."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# smallest step of a type: a rounding near zero is off by at most half of it
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def ref_maps(ids: np.ndarray, E: int, offset: int):
    """(offsets, row_slot, slot_row): rows by expert, then by slot."""
    flat = ids.reshape(-1).astype(np.int64) - offset
    by = [np.nonzero(flat == e)[0] for e in range(E)]
    offsets = np.concatenate([[0], np.cumsum([len(b) for b in by])])
    row_slot = np.concatenate(by) if by else np.zeros(0, np.int64)
    slot_row = np.full(flat.shape, -1, np.int64)
    slot_row[row_slot] = np.arange(len(row_slot))
    return offsets, row_slot, slot_row.reshape(ids.shape)


def ref_combine(rows: np.ndarray, slot_row: np.ndarray, w: np.ndarray):
    """(out, sum of magnitudes): columns without a row take no part."""
    T, K = slot_row.shape
    out, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for k in range(K):
        t = np.nonzero(slot_row[:, k] >= 0)[0]
        term = w[t, k, None] * rows[slot_row[t, k]]
        out[t] += term
        mag[t] += np.abs(term)
    return out, mag


def ref_combine_backward(dout, rows, slot_row, w):
    """(drows with NaN where nothing is written, dw, sum of magnitudes of dw)."""
    drows = np.full(rows.shape, np.nan)
    dw, mag = np.zeros(w.shape), np.zeros(w.shape)
    for t in range(w.shape[0]):
        for k in range(w.shape[1]):
            r = slot_row[t, k]
            if r >= 0:
                drows[r] = w[t, k] * dout[t]
                dw[t, k] = np.dot(dout[t], rows[r])
                mag[t, k] = np.dot(np.abs(dout[t]), np.abs(rows[r]))
    return drows, dw, mag


def round_tol(ref: np.ndarray, dtype: str, err32) -> np.ndarray:
    """Bound on a result rounded once to dtype whose 32-bit value is off by at
    most err32: half a step of the rounded value, plus err32 itself."""
    return (np.abs(ref) + err32) * torch.finfo(TORCH[dtype]).eps / 2 + TINY[dtype] / 2 + err32


def pack_rows(codes: np.ndarray) -> np.ndarray:
    """Codes [..., N, K] (0..15) -> bytes [..., Np, K / 2], even K in the low
    nibble; the rows added to reach a multiple of 16 hold 0xff."""
    b = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    pad = -b.shape[-2] % 16
    return np.concatenate([b, np.full((*b.shape[:-2], pad, b.shape[-1]), 0xff, np.uint8)], -2)


def ref_weights(codes, scales, zeros, fmt, group):
    """(weights, their magnitudes before the zero point comes off) in 64 bits."""
    if fmt == "mxfp4":
        s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
        v = E2M1[codes]
        m = np.abs(v)
    else:
        z = np.repeat(np.full(scales.shape, 8.0) if zeros is None else zeros.astype(np.float64), group, -1)
        s, v, m = scales, codes - z, codes + z
    s = np.repeat(s, group, -1)
    with np.errstate(invalid="ignore"):  # 0 times an infinite scale
        return v * s, m * np.abs(s)


def sum_tol(K: int) -> float:
    """Relative bound on a 32-bit sum of K products, of the sum of magnitudes.
    A product passes at most 32 additions inside its MFMA, one for each of the
    K / 32 MFMAs after it (a group's sum and its scale: two), and 8 more (waves,
    zero points, bias); an addition in the matrix unit is taken as off by a
    whole step, 2^-23, as one that cuts off would be."""
    return (40 + 2 * (K // 32)) * 2.0 ** -23
