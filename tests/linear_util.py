"""References in 64 bits for the 16-bit products and adapters, from their
definitions, and the bounds their tests hold the kernels to."""
from __future__ import annotations

import numpy as np
import torch

from ops_util import TORCH, f64, round_tol, sum_tol

EPS = {"bf16": 2.0 ** -7, "fp16": 2.0 ** -10, "fp32": 2.0 ** -23}  # a step at 1


def normal(rng, scale, dtype, *size):
    return torch.from_numpy(scale * rng.standard_normal(size)).to(TORCH[dtype]).cuda()


def owned(off, E, M):
    """(expert, first row, row after its last) of experts with rows."""
    if off is None:
        return [(0, 0, M)]
    o = [int(v) for v in off]
    return [(e, max(o[e], 0), min(o[e + 1], M)) for e in range(E) if min(o[e + 1], M) > max(o[e], 0)]


def ref_forward(x, w, off):
    """(rows times their matrix, sum of magnitudes); NaN where no expert owns a row."""
    out = np.full((x.shape[0], w.shape[1]), np.nan)
    mag = np.zeros(out.shape)
    for e, lo, hi in owned(off, w.shape[0], x.shape[0]):
        out[lo:hi] = x[lo:hi] @ w[e].T
        mag[lo:hi] = np.abs(x[lo:hi]) @ np.abs(w[e]).T
    return out, mag


def ref_backward(d, x, w, off, slack=None):
    """dx (NaN where no expert owns a row) and dw with bounds on their 32-bit values:
    the sums', and what an error of up to `slack` in d adds."""
    dx, ex = np.full(x.shape, np.nan), np.zeros(x.shape)
    dw, ew = np.zeros(w.shape), np.zeros(w.shape)
    for e, lo, hi in owned(off, w.shape[0], x.shape[0]):
        a, b = np.abs(d[lo:hi]), 0 if slack is None else slack[lo:hi]
        dx[lo:hi], dw[e] = d[lo:hi] @ w[e], d[lo:hi].T @ x[lo:hi]
        ex[lo:hi] = (sum_tol(w.shape[1]) * (a + b) + b) @ np.abs(w[e])
        ew[e] = (sum_tol(hi - lo) * (a + b) + b).T @ np.abs(x[lo:hi])
    return dx, ex, dw, ew


def act(g, u, kind, limit, beta=4.0, lb=25.0):
    """The activation and its derivatives by g and u."""
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
        if kind == "situ":
            tg, tu = np.tanh(g / beta), np.tanh(u / lb)
            return (beta * tg * s * lb * tu, lb * tu * (s * (1 - tg ** 2) + beta * tg * s * (1 - s)),
                    beta * tg * s * (1 - tu ** 2))
        L = limit if limit > 0 else np.inf
        gc, uc = np.minimum(g, L), np.clip(u, -L, L)
        s = 1 / (1 + np.exp(-gc))
        return gc * s * uc, np.where(g <= L, uc * (s + gc * s * (1 - s)), 0), np.where(np.abs(u) <= L, gc * s, 0)


def act_err(g, u, kind, beta=4.0, lb=25.0):
    """Bound on what 32-bit arithmetic adds to the activation or a derivative, of
    1 + |u|: each is a product of at most eight terms no larger than 2 (1 + |g|) and
    (1 + |u|), each of them off by a few steps and, by the exponential of a rounded
    product, |g| steps."""
    return (16 + 2 * np.abs(g)) * 2.0 ** -23 * (2 + np.abs(g)) * (1 + np.abs(u)) * (4 if kind == "situ" else 1)


def close(got, ref, tol, what):
    """Within the bound where the reference is a number; untouched rows are checked apart."""
    got = f64(got)
    has = ~np.isnan(ref)
    err = np.abs(got[has] - ref[has])
    t = np.broadcast_to(tol, ref.shape)[has]
    bad = ~(err <= t)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / t):.2f} tolerances"
