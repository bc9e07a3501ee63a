"""The gated product's gradients on the GPU with the pre-activations' gradient kept in two
terms: both products against their definition in 64 bits, with no rounding of it to 16 bits
in the bound."""
import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe

from gpu_util import say
from ops_util import TINY, TORCH, sum_tol

pytestmark = pytest.mark.gpu

MARK = -3.0
# what two terms leave of a value: half a step of half a step, or half the smallest number
REST = {"bf16": (2.0 ** -16, 2.0 ** -134), "fp16": (2.0 ** -22, 2.0 ** -25)}


def _act_grads(g, u, kind, limit, beta=4.0, lb=25.0):
    """The activation's derivatives by g and u, in 64 bits."""
    s = torch.sigmoid(g)
    if kind == "situ":
        tg, tu = torch.tanh(g / beta), torch.tanh(u / lb)
        return lb * tu * (s * (1 - tg ** 2) + beta * tg * s * (1 - s)), beta * tg * s * (1 - tu ** 2)
    if limit <= 0:
        return u * (s + g * s * (1 - s)), g * s
    gc, uc = g.clamp(max=limit), u.clamp(-limit, limit)
    s = torch.sigmoid(gc)
    return (g <= limit) * uc * (s + gc * s * (1 - s)), (u.abs() <= limit) * gc * s


def _offsets(M, E):
    """Uneven experts, one without rows, rows before the first and behind the last."""
    if E == 1:
        return None
    cut = sorted(np.random.default_rng(M).integers(2, M - 2, size=E - 1).tolist())
    off = [2, *cut, M - 2]
    off[E // 2] = off[E // 2 - 1]
    return off


# tiles of 64, 128 and 256, short and long stages, one launch for both gradients and two
SIZES = [(1, 1, 8, 8), (45, 3, 24, 40), (70, 4, 136, 264), (300, 12, 1024, 1024), (3, 1, 2048, 2056), (2048, 4, 200, 1544),
         (1000, 40, 768, 1000), (3000, 24, 648, 2312), (5800, 19, 184, 5152), (2500, 1, 2568, 4104), (7000, 1, 2312, 4616),
         (9000, 40, 1024, 520)]


@pytest.mark.parametrize("M,E,I,K", SIZES)
@pytest.mark.parametrize("dtype,kind,limit", [("bf16", "swiglu", 1.5), ("bf16", "situ", 0.0), ("fp16", "swiglu", 0.0)])
def test_two_terms(M, E, I, K, dtype, kind, limit):
    say(f"[terms] {M} {E} {I} {K} {dtype} {kind}")
    gen = torch.Generator(device="cuda").manual_seed(M + I)
    n = lambda scale, *size: torch.randn(*size, generator=gen, device="cuda").mul_(scale).to(TORCH[dtype])  # noqa: E731
    x, w, dh, gu = n(1, M, K), n(K ** -0.5, E, 2 * I, K), n(1, M, I), n(1.5, M, 2 * I)
    off = _offsets(M, E)
    at = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    args = dict(M=M, I=I, H=K, E=E, dtype=dtype, activation=kind, swiglu_limit=limit)
    one, two = moe.GatedShape(**args), moe.GatedShape(**args, dgu_terms=2)
    full = lambda *size: torch.full(size, MARK, dtype=TORCH[dtype], device="cuda")  # noqa: E731
    dgu1 = full(M, 2 * I)
    moe.gated_linear_backward(dh, x, at, gu, w, one, dx=False, dw=False, dgu=dgu1)
    dgu, dx = full(2, M, 2 * I), full(M, K)
    got, dw = moe.gated_linear_backward(dh, x, at, gu, w, two, dx=dx, dgu=dgu)
    assert got is dx and torch.equal(dgu[0], dgu1)
    # each gradient by itself is the same, and terms made by the call too
    alone, none = moe.gated_linear_backward(dh, None, at, gu, w, two, dx=full(M, K), dw=False)
    assert none is None and torch.equal(alone, dx)
    assert torch.equal(moe.gated_linear_backward(dh, x, at, gu, None, two, dx=False)[1], dw)
    rest, least = REST[dtype]
    half = torch.finfo(TORCH[dtype]).eps / 2
    spans = [(0, 0, M)] if off is None else [(e, off[e], off[e + 1]) for e in range(E)]
    seen = torch.zeros(M, dtype=torch.bool, device="cuda")

    def check(got, ref, bound, what):
        """Half a step of the result's one rounding beside what its 32-bit value is off by."""
        tol = (ref.abs() + bound) * half + TINY[dtype] / 2 + bound
        worst = float(((got.double() - ref).abs() / tol).max())
        assert worst <= 1, f"{what}: worst {worst:.2f} tolerances"

    for e, lo, hi in spans:
        if lo == hi:
            assert bool((dw[e] == 0).all())
            continue
        seen[lo:hi] = True
        g, u, d = gu[lo:hi, :I].double(), gu[lo:hi, I:].double(), dh[lo:hi].double()
        by_g, by_u = _act_grads(g, u, kind, limit)
        pre = torch.cat([by_g * d, by_u * d], 1)
        # 32-bit arithmetic of the derivatives: at most eight terms of 2 (1 + |g|)(1 + |u|),
        # each off by a few steps and, by a rounded exponent, |g| steps
        a32 = (16 + 2 * g.abs()) * 2.0 ** -23 * (2 + g.abs()) * (1 + u.abs()) * (4 if kind == "situ" else 1)
        slack = (a32 * d.abs()).repeat(1, 2)
        slack = slack + (pre.abs() + slack) * rest + least
        value = dgu[0, lo:hi].double() + dgu[1, lo:hi].double()
        assert float(((value - pre).abs() / slack).max()) <= 1
        # the terms' magnitudes sum to at most (1 + 2^-8) of the value's; a sum has twice as
        # many terms
        mag = (pre.abs() + slack) * (1 + 2.0 ** -7)
        X, W = x[lo:hi].double(), w[e].double()
        check(dx[lo:hi], pre @ W, (sum_tol(4 * I) * mag + slack) @ W.abs(), f"dx of {e}")
        check(dw[e], pre.t() @ X, (sum_tol(2 * (hi - lo)) * mag + slack).t() @ X.abs(), f"dw of {e}")
    assert bool((dx[~seen] == MARK).all()) and bool((dgu[:, ~seen] == MARK).all())


def test_terms_of_values_that_are_no_numbers():
    # NaN and infinities have nothing beside them, and stay in their rows
    gen = torch.Generator(device="cuda").manual_seed(1)
    M, I, K = 40, 16, 24
    x, w, dh, gu = (torch.randn(*n, generator=gen, device="cuda").bfloat16() for n in ((M, K), (2 * I, K), (M, I), (M, 2 * I)))
    s = moe.GatedShape(M=M, I=I, H=K, dgu_terms=2)
    clean = moe.gated_linear_backward(dh, x, None, gu, w, s)[0]
    dh[3, 5], dh[4, 6] = float("nan"), float("inf")
    dgu = torch.empty(2, M, 2 * I, dtype=torch.bfloat16, device="cuda")
    dx, _ = moe.gated_linear_backward(dh, x, None, gu, w, s, dgu=dgu)
    row = torch.arange(M, device="cuda")
    same = (row != 3) & (row != 4)
    assert torch.equal(dx[same], clean[same]) and bool(dx[3].isnan().all()) and not bool(dx[4].isfinite().any())
    odd = ~dgu[0].isfinite()
    assert odd.sum() == 4 and bool((dgu[1][odd] == 0).all())


def test_two_terms_without_rows_and_in_a_graph():
    z = lambda *n: torch.zeros(*n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    dx, dw = moe.gated_linear_backward(z(0, 8), z(0, 24), off, z(0, 16), z(2, 16, 24), moe.GatedShape(M=0, I=8, H=24, E=2, dgu_terms=2))
    assert dx.shape == (0, 24) and bool((dw == 0).all())
    M, I, K = 50, 16, 24
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, w, dh, gu = (torch.randn(*n, generator=gen, device="cuda").bfloat16() for n in ((M, K), (2 * I, K), (M, I), (M, 2 * I)))
    s, dx, dw, dgu = moe.GatedShape(M=M, I=I, H=K, dgu_terms=2), z(M, K), z(1, 2 * I, K), z(2, M, 2 * I)
    call = lambda: moe.gated_linear_backward(dh, x, None, gu, w, s, dx=dx, dw=dw, dgu=dgu)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for turn in range(3):
        dh.copy_(torch.randn(M, I, generator=gen, device="cuda"))
        for t in (dx, dw, dgu):
            t.fill_(turn)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (dx, dw, dgu)]
        call()
        assert all(torch.equal(a, b) for a, b in zip(got, (dx, dw, dgu)))
