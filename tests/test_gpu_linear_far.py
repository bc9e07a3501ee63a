"""The 16-bit products and adapters where arrays pass 4 GiB: results, pre-activations,
gradients, strided rows and the matrices themselves, of which the last rows or the last
expert's are used."""
import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe

from gpu_util import say
from linear_util import act, act_err, close, normal, ref_backward, ref_forward
from ops_util import f64, round_tol, sum_tol

pytestmark = pytest.mark.gpu

GB4 = 1 << 32
MARK = -3.0
LAST = 40  # rows that an expert owns, the last ones


def _bf(*size, value=None):
    e = torch.empty(*size, dtype=torch.bfloat16, device="cuda")
    return e if value is None else e.fill_(value)


def _far(t):
    """The array's last rows lie behind 32-bit byte offsets."""
    span = sum((n - 1) * s for n, s in zip(t.shape, t.stride())) * t.element_size()
    assert span > GB4
    return t


def _owns_last(M, E=1):
    return torch.tensor([0] * E + [M], dtype=torch.int32, device="cuda") if E > 1 else torch.tensor([M - LAST, M], dtype=torch.int32, device="cuda")


def _tail_only(t, value=MARK):
    return bool((t[:-LAST] == value).all())


def test_results_and_rows_gradients():
    M, N, K = 300_000, 8192, 64
    say("[far] out, dx")
    rng = np.random.default_rng(1)
    x, w = _bf(M, K, value=7), normal(rng, K ** -0.5, "bf16", N, K)
    x[-LAST:] = normal(rng, 1, "bf16", LAST, K)
    out = _far(_bf(M, N, value=MARK))
    moe.grouped_linear(x, _owns_last(M), w, moe.LinearShape(M=M, N=N, K=K), out=out)
    want, mag = ref_forward(f64(x[-LAST:]), f64(w)[None], None)
    close(out[-LAST:], want, round_tol(want, "bf16", sum_tol(K) * mag), "out")
    assert _tail_only(out)
    # the same array as dx of a product of 64 columns, and as x of its matrix's gradient
    d, wt = x, w.t().contiguous()
    back = moe.LinearShape(M=M, N=K, K=N)
    dx = out.fill_(MARK)
    rows = normal(rng, 1, "bf16", LAST, N)
    moe.grouped_linear_backward(d, None, _owns_last(M), wt, back, dx=dx, dw=False)
    close(dx[-LAST:], want, round_tol(want, "bf16", sum_tol(K) * mag), "dx")
    assert _tail_only(dx)
    far = dx
    far[-LAST:] = rows
    _, dw = moe.grouped_linear_backward(d, far, _owns_last(M), None, back, dx=False)
    _, _, rw, ew = ref_backward(f64(d[-LAST:]), f64(rows), f64(wt)[None], None)
    close(dw, rw, round_tol(rw, "bf16", ew), "dw")


def test_gated_pre_activations_and_their_gradient():
    M, I, K, L = 300_000, 4096, 64, 1.5
    say("[far] gu, dgu")
    rng = np.random.default_rng(2)
    x, w = _bf(M, K, value=7), normal(rng, K ** -0.5, "bf16", 1, 2 * I, K)
    x[-LAST:] = normal(rng, 1, "bf16", LAST, K)
    for terms in (1, 2):
        s = moe.GatedShape(M=M, I=I, H=K, swiglu_limit=L, dgu_terms=terms)
        gu, h = _far(_bf(M, 2 * I, value=MARK)), _bf(M, I, value=MARK)
        moe.gated_linear(x, _owns_last(M), w, s, out=h, gu=gu)
        want, mag = ref_forward(f64(x[-LAST:]), f64(w), None)
        close(gu[-LAST:], want, round_tol(want, "bf16", sum_tol(K) * mag), "gu")
        assert _tail_only(gu) and _tail_only(h)
        g, u, eg, eu = (v[:, p] for v in (want, sum_tol(K) * mag) for p in (slice(0, I), slice(I, None)))
        act_want, by_g, by_u = act(g, u, "swiglu", L)
        # the derivatives change by less than (2 + |u|) times the sums' errors over them; at
        # the border, where they drop to 0, the larger side counts
        err = eg * (np.abs(by_g) + (2 + np.abs(u)) * eg) + eu * (np.abs(by_u) + 2 * eg) + act_err(g, u, "swiglu")
        err = err + 2 * (1 + np.abs(u)) * eg * (np.abs(g - L) <= eg) + 2 * (1 + np.abs(g)) * eu * (np.abs(np.abs(u) - L) <= eu)
        close(h[-LAST:], act_want, round_tol(act_want, "bf16", err), "h")
        dh = h
        dh[-LAST:] = normal(rng, 1, "bf16", LAST, I)
        dgu = _bf(*((2,) if terms == 2 else ()), M, 2 * I, value=MARK)
        dx = _bf(M, K, value=MARK)
        dx, dw = moe.gated_linear_backward(dh, x, _owns_last(M), gu, w, s, dx=dx, dgu=_far(dgu))
        g, u = f64(gu[-LAST:])[:, :I], f64(gu[-LAST:])[:, I:]
        _, by_g, by_u = act(g, u, "swiglu", L)
        d = np.concatenate([by_g, by_u], 1) * np.tile(f64(dh[-LAST:]), 2)
        err = np.tile(np.abs(f64(dh[-LAST:])) * act_err(g, u, "swiglu"), 2)
        slack = round_tol(d, "bf16", err)
        first = dgu if terms == 1 else dgu[0]
        close(first[-LAST:], d, slack, "dgu")
        if terms == 2:
            close(dgu[1, -LAST:], d - f64(first[-LAST:]), err + 2.0 ** -16 * np.abs(d) + 2.0 ** -134, "the rest")
            assert _tail_only(dgu[1])
        rx, ex, rw, ew = ref_backward(d, f64(x[-LAST:]), f64(w), None, slack)
        close(dx[-LAST:], rx, round_tol(rx, "bf16", ex), "dx")
        close(dw, rw, round_tol(rw, "bf16", ew), "dw")
        assert _tail_only(first) and _tail_only(dx)
        del gu, h, dh, dgu, first, dx


@pytest.mark.parametrize("M", [LAST, 5000])  # few rows an expert on average, and tiles
def test_matrices(M):
    say(f"[far] matrices {M}")
    E, N, K = 600, 1024, 4096
    rng = np.random.default_rng(3)
    w, dw = _far(_bf(E, N, K, value=1)), _far(_bf(E, N, K, value=MARK))
    w[-1] = normal(rng, K ** -0.5, "bf16", N, K)
    x, d = _bf(M, K, value=0), _bf(M, N, value=0)
    x[-LAST:], d[-LAST:] = normal(rng, 1, "bf16", LAST, K), normal(rng, 1, "bf16", LAST, N)
    off = torch.full((E + 1,), M - LAST, dtype=torch.int32, device="cuda")
    off[-1] = M
    s = moe.LinearShape(M=M, N=N, K=K, E=E)
    out, dx = _bf(M, N, value=MARK), _bf(M, K, value=MARK)
    moe.grouped_linear(x, off, w, s, out=out)
    want, mag = ref_forward(f64(x[-LAST:]), f64(w[-1:]), None)
    close(out[-LAST:], want, round_tol(want, "bf16", sum_tol(K) * mag), "out")
    moe.grouped_linear_backward(d, x, off, w, s, dx=dx, dw=dw)
    rx, ex, rw, ew = ref_backward(f64(d[-LAST:]), f64(x[-LAST:]), f64(w[-1:]), None)
    close(dx[-LAST:], rx, round_tol(rx, "bf16", ex), "dx")
    close(dw[-1:], rw, round_tol(rw, "bf16", ew), "dw")
    assert bool((dw[:-1] == 0).all()) and _tail_only(out) and _tail_only(dx)
    if M > LAST:  # dw in 32 bits
        wide = _far(torch.full((E, N, K), MARK, dtype=torch.float32, device="cuda"))
        moe.grouped_linear_backward(d, x, off, None, moe.LinearShape(M=M, N=N, K=K, E=E, out_dtype="fp32"), dx=False, dw=wide)
        close(wide[-1:], rw, round_tol(rw, "fp32", ew), "dw in 32 bits")
        assert bool((wide[:-1] == 0).all())


@pytest.mark.parametrize("gated", [False, True])
def test_strided_rows_of_few_an_expert(gated):
    say(f"[far] strides {gated}")
    M, E, N, K, ld = 16384, 2048, 64, 72, 1 << 18
    rng = np.random.default_rng(4)
    x, out = _far(_bf(M, ld)[:, 8:8 + K]), _far(_bf(M, ld)[:, 16:16 + N])
    out.fill_(MARK)
    x[-LAST:] = normal(rng, 1, "bf16", LAST, K)
    w = _bf(E, N * (2 if gated else 1), K, value=1)
    w[-1] = normal(rng, K ** -0.5, "bf16", *w.shape[1:])
    off = torch.full((E + 1,), M - LAST, dtype=torch.int32, device="cuda")
    off[-1] = M
    near = x[-LAST:].contiguous()
    if gated:
        moe.gated_linear(x, off, w, moe.GatedShape(M=M, I=N, H=K, E=E), out=out)
        pre, mag = ref_forward(f64(near), f64(w[-1:]), None)
        g, u, eg, eu = pre[:, :N], pre[:, N:], sum_tol(K) * mag[:, :N], sum_tol(K) * mag[:, N:]
        want, by_g, by_u = act(g, u, "swiglu", 0.0)
        # the derivatives change by less than (2 + |u|) times the sums' errors over them
        err = eg * (np.abs(by_g) + (2 + np.abs(u)) * eg) + eu * (np.abs(by_u) + 2 * eg) + act_err(g, u, "swiglu")
        close(out[-LAST:], want, round_tol(want, "bf16", err), "h")
    else:
        moe.grouped_linear(x, off, w, moe.LinearShape(M=M, N=N, K=K, E=E), out=out)
        want, mag = ref_forward(f64(near), f64(w[-1:]), None)
        close(out[-LAST:], want, round_tol(want, "bf16", sum_tol(K) * mag), "out")
    assert _tail_only(out)


def test_adapters():
    M, N, K, R, A = 300_000, 8200, 8200, 128, 2048
    say("[far] adapters")
    rng = np.random.default_rng(5)
    x, base = _far(_bf(M, K, value=1)), _far(_bf(M, N, value=MARK))
    x[-LAST:], base[-LAST:] = normal(rng, 1, "bf16", LAST, K), normal(rng, 1, "bf16", LAST, N)
    a, b = _far(_bf(A, R, K, value=1)), _far(_bf(A, N, R, value=1))
    a[-1], b[-1] = normal(rng, K ** -0.5, "bf16", R, K), normal(rng, R ** -0.5, "bf16", N, R)
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[-LAST:] = A - 1
    s = moe.AdapterShape(M=M, N=N, K=K, R=R, A=A)
    maps = moe.adapter_maps(ids, s)
    t, tm = f64(x[-LAST:]) @ f64(a[-1]).T, np.abs(f64(x[-LAST:])) @ np.abs(f64(a[-1])).T
    B, was = f64(b[-1]), f64(base[-LAST:])
    want = was + t @ B.T
    # t's sum and its two terms, the second sum over both, the addition
    et = sum_tol(K) * tm + 2.0 ** -16 * np.abs(t)
    tol = 2.0 ** -23 * np.abs(was) + et @ np.abs(B).T + (sum_tol(2 * R) + 2.0 ** -22) * (np.abs(t) @ np.abs(B).T)
    out = _far(_bf(M, N, value=0))
    moe.adapter_linear(x, *maps, a, b, None, s, base=base, out=out)
    close(out[-LAST:], want, round_tol(want, "bf16", tol), "out")
    assert _tail_only(out)
    moe.adapter_linear(x, *maps, a, b, None, s, base=base, out=base)
    assert torch.equal(base[-LAST:], out[-LAST:]) and _tail_only(base)
