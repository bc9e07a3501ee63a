"""The activation's limit on the GPU: NaN and infinities in the gated products of 16-bit
matrices and in the expert layer, values on the limit itself."""
import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe

from gpu_util import run, say, to_device
from linear_util import act, act_err, close, normal
from ops_util import TORCH, f64, round_tol
from workloads import LayerShape, make_inputs

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _gpu(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


# few rows (one a matrix, several an expert), tiles of 64, 128 and 256, short and long stages
SIZES = [(3, 1, 24, 40), (24, 3, 40, 72), (90, 3, 24, 40), (300, 12, 1024, 1024), (3000, 24, 648, 2312), (2500, 1, 2568, 4104),
         (9000, 40, 1024, 520)]


@pytest.mark.parametrize("M,E,I,K", SIZES)
@pytest.mark.parametrize("kind,limit", [("swiglu", 0.0), ("swiglu", 1.5), ("situ", 0.0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_no_number_becomes_one_forward(M, E, I, K, kind, limit, dtype):
    say(f"[limit] forward {M} {E} {I} {K} {kind} {limit} {dtype}")
    rng = np.random.default_rng(M + I)
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w = (torch.randn(*n, generator=g, device="cuda").mul_(s).to(TORCH[dtype]) for n, s in (((M, K), 1), ((E, 2 * I, K), 1.5 * K ** -0.5)))
    off = [M * e // E for e in range(E + 1)]
    shape = moe.GatedShape(M=M, I=I, H=K, E=E, dtype=dtype, activation=kind, swiglu_limit=limit)
    gu, gu2 = (torch.zeros(M, 2 * I, dtype=TORCH[dtype], device="cuda") for _ in range(2))
    h = moe.gated_linear(x, _gpu(off), w, shape, gu=gu)
    rows = [0, off[1] - 1]  # one of NaN, one whose products' infinities cancel (or meet zeros)
    x[rows[0], int(rng.integers(K))] = NAN
    x[rows[1], 0], x[rows[1], 1] = INF, -INF
    w[0, :, 0], w[0, :, 1] = w[0, :, 0].abs() + 0.25, w[0, :, 1].abs() + 0.25
    e, i, j = E - 1, 1, I - 2  # a gate row and an up row of the last expert
    w[e, i], w[e, I + j] = NAN, NAN
    h2 = moe.gated_linear(x, _gpu(off), w, shape, gu=gu2)
    assert bool(h2[rows].isnan().all()) and bool(gu2[rows].isnan().all())
    last = h2[off[e]:]
    assert bool(last[:, i].isnan().all()) and bool(last[:, j].isnan().all())
    keep = torch.ones(M, I, dtype=torch.bool, device="cuda")
    keep[:off[1]] = False  # expert 0 has other weights
    keep[off[e]:, [i, j]] = False
    assert torch.equal(h2[keep], h[keep])
    assert torch.equal(gu2[off[1]:off[e]], gu[off[1]:off[e]])


@pytest.mark.parametrize("kind,limit", [("swiglu", 0.0), ("swiglu", 1.5), ("situ", 0.0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_no_number_becomes_one_backward(kind, limit, dtype):
    rng = np.random.default_rng(3)
    off, E, M, I, K = [0, 30, 70], 2, 75, 24, 40
    x, w, dh = normal(rng, 1, dtype, M, K), normal(rng, K ** -0.5, dtype, E, 2 * I, K), normal(rng, 1, dtype, M, I)
    gu = normal(rng, 1, dtype, M, 2 * I)
    gu[5, I] = gu[6, 1] = gu[6, I + 1] = 0.5  # inside the limit
    shape = moe.GatedShape(M=M, I=I, H=K, E=E, dtype=dtype, activation=kind, swiglu_limit=limit)
    out = []
    for spoilt in (False, True):
        if spoilt:
            gu[5, 0], gu[6, I + 1], gu[70:] = NAN, NAN, NAN
        dgu = torch.zeros(M, 2 * I, dtype=TORCH[dtype], device="cuda")
        dx = torch.zeros(M, K, dtype=TORCH[dtype], device="cuda")
        dx, dw = moe.gated_linear_backward(dh, x, _gpu(off), gu, w, shape, dx=dx, dgu=dgu)
        out.append((dgu, dx, dw))
    (dgu, dx, dw), (dgu2, dx2, dw2) = out
    # NaN g: both gradients; NaN u: that of g (SiTU: of both), du is dh times the gate's half
    gone = torch.zeros(M, 2 * I, dtype=torch.bool, device="cuda")
    gone[5, 0] = gone[5, I] = gone[6, 1] = True
    gone[6, I + 1] = kind == "situ"
    assert torch.equal(dgu2.isnan(), gone) and torch.equal(dgu2[~gone], dgu[~gone])
    row = gone.any(1)
    assert bool(dx2[row].isnan().all()) and torch.equal(dx2[~row], dx[~row])
    col = gone.any(0)
    assert bool(dw2[0, col].isnan().all()) and torch.equal(dw2[0, ~col], dw[0, ~col]) and torch.equal(dw2[1], dw[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_infinities_are_cut_off(dtype):
    # g = inf counts as L, u = +-inf as +-L; their own gradients are 0
    rng = np.random.default_rng(4)
    M, I, K, L = 20, 16, 24, 2.0
    gu, dh = normal(rng, 1, dtype, M, 2 * I), normal(rng, 1, dtype, M, I)
    gu[3, 2], gu[4, I + 3], gu[5, I + 4] = INF, INF, -INF
    same = gu.clone()
    same[3, 2], same[4, I + 3], same[5, I + 4] = 2 * L, 3 * L, -2 * L
    x, w = normal(rng, 1, dtype, M, K), normal(rng, 0.2, dtype, 2 * I, K)
    shape = moe.GatedShape(M=M, I=I, H=K, dtype=dtype, swiglu_limit=L)
    got = []
    for pre in (gu, same):
        dgu = torch.empty(M, 2 * I, dtype=TORCH[dtype], device="cuda")
        got.append((dgu, *moe.gated_linear_backward(dh, x, None, pre, w, shape, dgu=dgu)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][0][3, 2] == 0 and got[0][0][4, I + 3] == 0 and got[0][0][5, I + 4] == 0


@pytest.mark.parametrize("M", [4, 40])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_values_on_the_limit(M, dtype):
    # pre-activations that are exact: one step below the limit, on it, one above, on both
    # sides. On it counts as inside.
    say(f"[limit] border {M} {dtype}")
    L, I = 1.5, 16
    step = 2.0 ** (-7 if dtype == "bf16" else -10)
    at = np.array([L - step, L, L + step, -L + step, -L, -L - step, 0.0, 4.0])
    pre = np.concatenate([np.tile(at, I // 8), np.repeat(at, 2)])  # [2 I]: every g with several u
    assert pre.shape == (2 * I,)
    w = torch.zeros(2 * I, 8, dtype=TORCH[dtype], device="cuda")
    w[:, 0] = torch.from_numpy(pre).to(TORCH[dtype])
    assert np.array_equal(f64(w[:, 0]), pre)
    x = torch.zeros(M, 8, dtype=TORCH[dtype], device="cuda")
    x[:, 0] = 1
    shape = moe.GatedShape(M=M, I=I, H=8, dtype=dtype, swiglu_limit=L)
    gu = torch.zeros(M, 2 * I, dtype=TORCH[dtype], device="cuda")
    h = moe.gated_linear(x, None, w, shape, gu=gu)
    assert np.array_equal(f64(gu), np.tile(pre, (M, 1)))
    g, u = np.tile(pre[:I], (M, 1)), np.tile(pre[I:], (M, 1))
    want, by_g, by_u = act(g, u, "swiglu", L)
    close(h, want, round_tol(want, dtype, act_err(g, u, "swiglu")), "h")
    rng = np.random.default_rng(M)
    dh = normal(rng, 1, dtype, M, I)
    dgu = torch.zeros(M, 2 * I, dtype=TORCH[dtype], device="cuda")
    moe.gated_linear_backward(dh, x, None, gu, w, shape, dgu=dgu)
    d = np.concatenate([by_g, by_u], 1) * np.tile(f64(dh), 2)
    err = np.tile(np.abs(f64(dh)) * act_err(g, u, "swiglu"), 2)
    close(dgu, d, round_tol(d, dtype, err), "dgu")
    cut = np.concatenate([g > L, np.abs(u) > L], 1)
    assert bool((f64(dgu)[cut] == 0).all()) and bool((f64(dgu)[:, :I][(g == L) & (u != 0)] != 0).all())


# decode and prefill, one row of a token block spoilt
@pytest.mark.parametrize("s", [LayerShape("limit_decode", T=24, E=8, E_g=8, topk=2, H=512, I=256, B=16, swiglu_limit=3.0),
                               LayerShape("limit_prefill", T=700, E=6, E_g=6, topk=2, H=512, I=128, B=128, swiglu_limit=3.0)],
                         ids=lambda s: s.name)
def test_no_number_becomes_one_in_the_layer(s):
    dev = to_device(s, make_inputs(s, 5))
    clean = run(s, dev)[0].clone()
    dev["x"][7, 11] = NAN
    out = run(s, dev)[0]
    torch.cuda.synchronize()
    rest = torch.arange(s.T, device="cuda") != 7
    assert torch.equal(out[rest], clean[rest]) and bool(out[7].isnan().all())
