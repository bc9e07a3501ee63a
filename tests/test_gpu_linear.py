"""The 16-bit grouped and gated products and their gradients on the GPU, against
their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe

from gpu_util import say
from linear_util import EPS, act, act_err, close, normal, owned, ref_backward, ref_forward
from ops_util import TORCH, f64, round_tol, sum_tol

pytestmark = pytest.mark.gpu

MARK = -3.0  # what outputs hold before a call

# rows of each expert: none, a few, ends of the 32-row blocks and 256-row tiles;
# (rows before the first expert's, counts, rows behind the last)
ROWS = {
    "one": (0, [1], 0),
    "few": (0, [0, 3, 1, 0, 0, 5, 2], 4),
    "sixteen": (2, [16, 17, 15, 0, 1, 33], 3),
    "blocks": (0, [31, 32, 33, 64, 65, 0], 7),
    "tiles": (5, [255, 0, 256, 257], 1),
    "more": (0, [600, 130], 0),
    "none": (3, [0, 0, 0], 5),
}


def _offsets(rows):
    before, counts, behind = ROWS[rows]
    off = before + np.concatenate([[0], np.cumsum(counts)])
    return off, len(counts), int(off[-1]) + behind


def _gpu(off):
    return torch.as_tensor(np.asarray(off), dtype=torch.int32).cuda()


def _untouched(out, off, E, M, what):
    keep = np.ones(M, bool)
    for _, lo, hi in owned(off, E, M):
        keep[lo:hi] = False
    assert np.all(f64(out)[keep] == MARK), f"{what}: rows without an expert were written"


SIZES = [(8, 8), (40, 24), (256, 32), (248, 1000), (264, 72), (520, 264)]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32")])
def test_grouped(rows, N, K, dtype, out):
    say(f"[linear] {rows} {N} {K} {dtype}")
    rng = np.random.default_rng(N * K)
    off, E, M = _offsets(rows)
    x, w = normal(rng, 1, dtype, M, K), normal(rng, K ** -0.5, dtype, E, N, K)
    shape = moe.LinearShape(M=M, N=N, K=K, E=E, dtype=dtype, out_dtype=out)
    got = torch.full((M, N), MARK, dtype=TORCH[out], device="cuda")
    assert moe.grouped_linear(x, _gpu(off), w, shape, out=got) is got
    ref, mag = ref_forward(f64(x), f64(w), off)
    close(got, ref, round_tol(ref, out, sum_tol(K) * mag), "out")
    _untouched(got, off, E, M, "out")
    again = torch.full_like(got, MARK)
    moe.grouped_linear(x, _gpu(off), w, shape, out=again)
    assert torch.equal(got, again)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("dtype,out", [("bf16", "fp32"), ("fp16", "fp16")])
def test_grouped_backward(rows, N, K, dtype, out):
    say(f"[linear] backward {rows} {N} {K} {dtype}")
    rng = np.random.default_rng(N + K)
    off, E, M = _offsets(rows)
    x, w, d = normal(rng, 1, dtype, M, K), normal(rng, K ** -0.5, dtype, E, N, K), normal(rng, 1, dtype, M, N)
    shape = moe.LinearShape(M=M, N=N, K=K, E=E, dtype=dtype, out_dtype=out)
    dx = torch.full((M, K), MARK, dtype=TORCH[dtype], device="cuda")
    dw = torch.full((E, N, K), MARK, dtype=TORCH[out], device="cuda")
    assert moe.grouped_linear_backward(d, x, _gpu(off), w, shape, dx=dx, dw=dw) == (dx, dw)
    rx, ex, rw, ew = ref_backward(f64(d), f64(x), f64(w), off)
    close(dx, rx, round_tol(rx, dtype, ex), "dx")
    close(dw, rw, round_tol(rw, out, ew), "dw")
    _untouched(dx, off, E, M, "dx")
    # each gradient by itself is the same
    only_x, none = moe.grouped_linear_backward(d, None, _gpu(off), w, shape, dx=torch.full_like(dx, MARK), dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = moe.grouped_linear_backward(d, x, _gpu(off), None, shape, dx=False)
    assert none is None and torch.equal(only_w, dw)


ACTS = [("swiglu", 0.0), ("swiglu", 1.5), ("situ", 0.0)]


@pytest.mark.parametrize("rows", ["one", "sixteen", "blocks", "more", "none"])
@pytest.mark.parametrize("I,K", [(8, 8), (24, 40), (128, 264), (136, 1000)])
@pytest.mark.parametrize("kind,limit", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated(rows, I, K, kind, limit, dtype):
    say(f"[linear] gated {rows} {I} {K} {kind} {limit} {dtype}")
    rng = np.random.default_rng(I * K)
    off, E, M = _offsets(rows)
    x, w = normal(rng, 1, dtype, M, K), normal(rng, 1.5 * K ** -0.5, dtype, E, 2 * I, K)
    shape = moe.GatedShape(M=M, I=I, H=K, E=E, dtype=dtype, activation=kind, swiglu_limit=limit)
    h = torch.full((M, I), MARK, dtype=TORCH[dtype], device="cuda")
    gu = torch.full((M, 2 * I), MARK, dtype=TORCH[dtype], device="cuda")
    assert moe.gated_linear(x, _gpu(off), w, shape, out=h, gu=gu) is h
    ref, mag = ref_forward(f64(x), f64(w), off)
    err = sum_tol(K) * mag
    close(gu, ref, round_tol(ref, dtype, err), "gu")
    g, u = ref[:, :I], ref[:, I:]
    want, by_g, by_u = act(g, u, kind, limit)
    # the derivatives change by less than (2 + |u|) times the sums' errors over them
    e2 = (err[:, :I] * (np.abs(by_g) + (2 + np.abs(u)) * err[:, :I]) + err[:, I:] * (np.abs(by_u) + 2 * err[:, :I])
          + act_err(g, u, kind))
    if limit > 0:  # by_g and by_u drop to 0 at the border: the larger side counts there
        e2 = e2 + 2 * (1 + np.abs(u)) * err[:, :I] * (np.abs(g - limit) <= err[:, :I]) + 2 * (1 + np.abs(g)) * err[:, I:] * (
            np.abs(np.abs(u) - limit) <= err[:, I:])
    close(h, want, round_tol(want, dtype, e2), "h")
    _untouched(h, off, E, M, "h")
    _untouched(gu, off, E, M, "gu")
    alone = torch.full_like(h, MARK)
    moe.gated_linear(x, _gpu(off), w, shape, out=alone)
    assert torch.equal(alone, h)


@pytest.mark.parametrize("rows", ["one", "sixteen", "blocks", "tiles", "none"])
@pytest.mark.parametrize("I,K", [(8, 8), (24, 40), (136, 264)])
@pytest.mark.parametrize("kind,limit", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated_backward(rows, I, K, kind, limit, dtype):
    say(f"[linear] gated backward {rows} {I} {K} {kind} {limit} {dtype}")
    rng = np.random.default_rng(I + K)
    off, E, M = _offsets(rows)
    x, w = normal(rng, 1, dtype, M, K), normal(rng, K ** -0.5, dtype, E, 2 * I, K)
    gu, dh = normal(rng, 1.5, dtype, M, 2 * I), normal(rng, 1, dtype, M, I)
    gu[::3, 0] = 1.5  # on the border
    shape = moe.GatedShape(M=M, I=I, H=K, E=E, dtype=dtype, activation=kind, swiglu_limit=limit)
    dx = torch.full((M, K), MARK, dtype=TORCH[dtype], device="cuda")
    dgu = torch.full((M, 2 * I), MARK, dtype=TORCH[dtype], device="cuda")
    dx, dw = moe.gated_linear_backward(dh, x, _gpu(off), gu, w, shape, dx=dx, dgu=dgu)
    g, u = f64(gu)[:, :I], f64(gu)[:, I:]
    _, by_g, by_u = act(g, u, kind, limit)
    d = np.concatenate([by_g, by_u], 1) * np.tile(f64(dh), 2)
    err = np.tile(np.abs(f64(dh)) * act_err(g, u, kind), 2)
    slack = round_tol(d, dtype, err)
    close(dgu, np.where(np.all(f64(dgu) == MARK, 1)[:, None], np.nan, d), slack, "dgu")
    rx, ex, rw, ew = ref_backward(d, f64(x), f64(w), off, slack)
    close(dx, rx, round_tol(rx, dtype, ex), "dx")
    close(dw, rw, round_tol(rw, dtype, ew), "dw")
    _untouched(dx, off, E, M, "dx")
    _untouched(dgu, off, E, M, "dgu")


def test_one_matrix_without_offsets():
    rng = np.random.default_rng(5)
    for M in (1, 15, 16, 17, 300):
        x, w, d = normal(rng, 1, "bf16", M, 72), normal(rng, .1, "bf16", 80, 72), normal(rng, 1, "bf16", M, 80)
        s = moe.LinearShape(M=M, N=80, K=72)
        one, all_rows = w[None], _gpu([0, M])
        assert torch.equal(moe.grouped_linear(x, None, w, s), moe.grouped_linear(x, all_rows, one, s))
        a, b = moe.grouped_linear_backward(d, x, None, w, s), moe.grouped_linear_backward(d, x, all_rows, one, s)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        g = moe.GatedShape(M=M, I=40, H=72)
        assert torch.equal(moe.gated_linear(x, None, w, g), moe.gated_linear(x, all_rows, one, g))


def test_strided_rows():
    rng = np.random.default_rng(6)
    M, N, K = 70, 48, 40
    w = normal(rng, .1, "bf16", N, K)
    both = torch.full((M, 160), MARK, dtype=torch.bfloat16, device="cuda")
    both[:, 8:48] = normal(rng, 1, "bf16", M, K)
    x = both[:, 8:48].contiguous()
    s = moe.LinearShape(M=M, N=N, K=K)
    moe.grouped_linear(both[:, 8:48], None, w, s, out=both[:, 56:104])
    assert torch.equal(both[:, 56:104], moe.grouped_linear(x, None, w, s))
    moe.gated_linear(both[:, 8:48], None, w, moe.GatedShape(M=M, I=24, H=K), out=both[:, 128:152])
    assert torch.equal(both[:, 128:152], moe.gated_linear(x, None, w, moe.GatedShape(M=M, I=24, H=K)))
    rest = torch.cat([both[:, :8], both[:, 48:56], both[:, 104:128], both[:, 152:]], 1)
    assert torch.equal(both[:, 8:48], x) and bool((rest == MARK).all())


def test_values_that_are_no_numbers_stay_in_their_rows():
    # one expert's rows and matrix hold NaN and infinities: the others' results are the same
    rng = np.random.default_rng(7)
    off, E, M, N, K = [0, 20, 55, 70], 3, 75, 40, 72
    x, w, d = normal(rng, 1, "bf16", M, K), normal(rng, .1, "bf16", E, N, K), normal(rng, 1, "bf16", M, N)
    s = moe.LinearShape(M=M, N=N, K=K, E=E)
    run = lambda: (moe.grouped_linear(x, _gpu(off), w, s), *moe.grouped_linear_backward(d, x, _gpu(off), w, s))  # noqa: E731
    out, dx, dw = run()
    for t in (x, d):
        t[20:55] = float("nan")
        t[70:] = float("inf")
    w[1] = float("inf")
    out2, dx2, dw2 = run()
    for a, b in ((out, out2), (dx, dx2)):
        assert torch.equal(a[:20], b[:20]) and torch.equal(a[55:70], b[55:70]) and bool(b[20:55].isnan().all())
    assert torch.equal(dw[0], dw2[0]) and torch.equal(dw[2], dw2[2]) and bool(dw2[1].isnan().all())


def test_offsets_past_the_rows():
    # values past M count as M, as for the 4-bit products
    rng = np.random.default_rng(8)
    M, N, K = 40, 24, 32
    x, w, d = normal(rng, 1, "bf16", M, K), normal(rng, .1, "bf16", 3, N, K), normal(rng, 1, "bf16", M, N)
    s = moe.LinearShape(M=M, N=N, K=K, E=3)
    a, b = _gpu([0, 30, 64, 99]), _gpu([0, 30, 40, 40])
    assert torch.equal(moe.grouped_linear(x, a, w, s), moe.grouped_linear(x, b, w, s))
    for p, q in zip(moe.grouped_linear_backward(d, x, a, w, s), moe.grouped_linear_backward(d, x, b, w, s)):
        assert torch.equal(p, q)


def test_gradients_against_differences():
    # along a random direction, forward in 32-bit results: the sum of gradient times
    # step is the difference of the results' sums weighted by dh
    rng = np.random.default_rng(9)
    off, E, M, I, K = _gpu([0, 9, 9, 40]), 3, 40, 16, 64
    for kind, limit in ACTS:
        x, w, dh = normal(rng, 1, "fp16", M, K), normal(rng, .15, "fp16", E, 2 * I, K), normal(rng, 1, "fp16", M, I)
        s = moe.GatedShape(M=M, I=I, H=K, E=E, dtype="fp16", activation=kind, swiglu_limit=limit)
        gu = torch.empty(M, 2 * I, dtype=torch.float16, device="cuda")
        moe.gated_linear(x, off, w, s, gu=gu)
        dx, dw = moe.gated_linear_backward(dh, x, off, gu, w, s)

        def value(xx, ww):
            ref, _ = ref_forward(xx, ww, [0, 9, 9, 40])
            return float((act(ref[:, :I], ref[:, I:], kind, limit)[0] * f64(dh)).sum())

        for grad, at in ((dx, 0), (dw, 1)):
            base = [f64(x), f64(w)]
            step = rng.standard_normal(grad.shape)
            ends = []
            for sign in (1, -1):
                moved = list(base)
                moved[at] = base[at] + sign * 1e-6 * step
                ends.append(value(*moved))
            slope = (ends[0] - ends[1]) / 2e-6
            got = float((f64(grad) * step).sum())
            # each gradient is off by the roundings of fp16 (its own, and those of gu and
            # dgu in its sum); their signs are as good as random, so the sum's spread is
            # the norm of the terms, and six times it a bound that holds
            spread = np.sqrt(((f64(grad) * step) ** 2).sum())
            scale = np.linalg.norm(f64(grad)) / np.sqrt(grad.numel()) * np.linalg.norm(step)
            assert abs(got - slope) <= 6 * 4 * EPS["fp16"] * (spread + scale), (kind, limit, at, got, slope)
