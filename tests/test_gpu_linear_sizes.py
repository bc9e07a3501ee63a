"""The 16-bit products at sizes that take each of their kernels (tiles of 64, 128 and 256,
short and long stages, few rows, both gradients in one launch), against their definitions
in 64 bits on the GPU."""
import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe

from gpu_util import say
from ops_util import TINY, TORCH, sum_tol

pytestmark = pytest.mark.gpu


def _normal(g, scale, dtype, *size):
    return (scale * torch.randn(*size, generator=g, device="cuda")).to(TORCH[dtype])


def _offsets(rng, M, E, skew=1.0):
    """Uneven experts, some without rows, a few rows before the first and behind the last."""
    share = rng.dirichlet(np.full(E, skew))
    share[rng.random(E) < 0.1] = 0
    counts = np.floor(share / max(share.sum(), 1e-9) * (M - 7)).astype(int)
    return (3 + np.concatenate([[0], np.cumsum(counts)])).tolist()


def _close(got, ref, bound, dtype, what):
    """bound: of the 32-bit value's error; half a step of the rounded value beside it."""
    tol = (ref.abs() + bound) * (torch.finfo(TORCH[dtype]).eps / 2) + TINY[dtype] / 2 + bound
    worst = float(((got.double() - ref).abs() / tol).max()) if ref.numel() else 0.0
    assert worst <= 1, f"{what}: worst {worst:.2f} tolerances"


def _spans(off, M):
    return [(0, 0, M)] if off is None else [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e + 1] > off[e]]


SHAPES = [  # M, E, N, K
    (9000, 40, 2048, 520), (3000, 24, 1288, 2312), (1000, 40, 1536, 1000), (2500, 1, 5128, 4104), (7000, 1, 4616, 4616),
    (300, 12, 2048, 1024), (5000, 2, 1032, 2056), (4000, 1, 2056, 2056), (40, 40, 1000, 1032), (40, 40, 1000, 520),
    (3, 1, 4096, 2056), (2048, 4, 392, 1544), (5800, 19, 368, 5152),
]


@pytest.mark.parametrize("M,E,N,K", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "fp32"), ("fp16", "fp16")])
def test_products_and_gradients(M, E, N, K, dtype, out):
    say(f"[linear] {M} {E} {N} {K} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(M + N)
    off = None if E == 1 else _offsets(np.random.default_rng(K), M, E)
    at = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    x, w, d = _normal(g, 1, dtype, M, K), _normal(g, K ** -0.5, dtype, E, N, K), _normal(g, 1, dtype, M, N)
    s = moe.LinearShape(M=M, N=N, K=K, E=E, dtype=dtype, out_dtype=out)
    y = torch.zeros(M, N, dtype=TORCH[out], device="cuda")
    dx = torch.zeros(M, K, dtype=TORCH[dtype], device="cuda")
    moe.grouped_linear(x, at, w, s, out=y)
    dx, dw = moe.grouped_linear_backward(d, x, at, w, s, dx=dx)
    alone = torch.zeros_like(dx)
    moe.grouped_linear_backward(d, None, at, w, s, dx=alone, dw=False)
    assert torch.equal(alone, dx)
    assert torch.equal(moe.grouped_linear_backward(d, x, at, None, s, dx=False)[1], dw)
    seen = torch.zeros(M, dtype=torch.bool, device="cuda")
    for e, lo, hi in _spans(off, M):
        a, b, c = x[lo:hi].double(), w[e].double(), d[lo:hi].double()
        _close(y[lo:hi], a @ b.t(), sum_tol(K) * (a.abs() @ b.abs().t()), out, f"out of {e}")
        _close(dx[lo:hi], c @ b, sum_tol(N) * (c.abs() @ b.abs()), dtype, f"dx of {e}")
        _close(dw[e], c.t() @ a, sum_tol(hi - lo) * (c.abs().t() @ a.abs()), out, f"dw of {e}")
        seen[lo:hi] = True
    assert bool((y[~seen] == 0).all()) and bool((dx[~seen] == 0).all())
    for e in set(range(E)) - {e for e, _, _ in _spans(off, M)}:
        assert bool((dw[e] == 0).all())


@pytest.mark.parametrize("M,E,I,K", [(9000, 40, 1024, 520), (3000, 24, 648, 2312), (2500, 1, 2568, 4104), (300, 12, 1024, 1024),
                                     (40, 40, 504, 1032), (40, 40, 504, 520), (200, 1, 200, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated_pre_activations_and_result(M, E, I, K, dtype):
    # h at the pre-activations' 32-bit values, which are gu's up to its rounding
    say(f"[linear] gated {M} {E} {I} {K} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(M + I)
    off = None if E == 1 else _offsets(np.random.default_rng(K), M, E)
    at = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    x, w = _normal(g, 1, dtype, M, K), _normal(g, K ** -0.5, dtype, E, 2 * I, K)
    s = moe.GatedShape(M=M, I=I, H=K, E=E, dtype=dtype)
    gu = torch.zeros(M, 2 * I, dtype=TORCH[dtype], device="cuda")
    h = torch.zeros(M, I, dtype=TORCH[dtype], device="cuda")
    moe.gated_linear(x, at, w, s, out=h, gu=gu)
    for e, lo, hi in _spans(off, M):
        a, b = x[lo:hi].double(), w[e].double()
        pre, bound = a @ b.t(), sum_tol(K) * (a.abs() @ b.abs().t())
        _close(gu[lo:hi], pre, bound, dtype, f"gu of {e}")
        p, u, ep, eu = pre[:, :I], pre[:, I:], bound[:, :I], bound[:, I:]
        silu = p * torch.sigmoid(p)
        # |silu'| <= 1.1, and 32-bit arithmetic: an exponential, a division and three
        # products, off by a few steps and, by the exponent's rounding, |p| steps
        err = 1.1 * ep * (u.abs() + eu) + silu.abs() * eu + (8 + p.abs()) * 2.0 ** -23 * (silu * u).abs()
        _close(h[lo:hi], silu * u, err, dtype, f"h of {e}")
