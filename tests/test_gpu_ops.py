"""Dispatch, combine and the 4-bit products against 64-bit references, at the
sizes, maps and layouts where they can go wrong."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe
import oracle
from workloads import LayerShape, make_inputs

from gpu_util import check_out, out_np, say, to_device
from ops_util import (TORCH, f64, pack_rows, ref_combine, ref_combine_backward, ref_maps,
                      ref_weights, round_tol, sum_tol)

pytestmark = pytest.mark.gpu


def _ids(rng, T, topk, experts, mode="distinct"):
    if mode == "distinct":
        ids = np.argsort(rng.random((T, experts)), axis=1)[:, :topk]
    elif mode == "one":
        ids = np.full((T, topk), experts - 1)
    elif mode == "none":
        ids = rng.choice([-1, experts, experts + 7, 2 ** 31 - 1, -2 ** 31], size=(T, topk))
    else:  # any: repeats within a token, and ids that name nothing
        ids = rng.integers(-2, experts + 2, size=(T, topk))
        ids[rng.random((T, topk)) < 0.05] = -2 ** 31
    return np.ascontiguousarray(ids.astype(np.int32))


def _same(got: torch.Tensor, want: np.ndarray):
    return np.array_equal(got.cpu().numpy(), want)


def _close(got: torch.Tensor, ref: np.ndarray, tol: np.ndarray, what: str):
    err = np.abs(f64(got) - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / tol):.2f} tolerances"


def _filled(shape, dtype):
    """A buffer of a pattern that no operator writes, and its bits."""
    t = torch.full(shape, 777.0, dtype=dtype, device="cuda")
    return t, t.clone()


# T, E, experts, offset, topk, H, dtype, mode
ROUTES = [
    (1, 1, 1, 0, 1, 1, "bf16", "distinct"),
    (1, 8, 8, 0, 2, 512, "bf16", "distinct"),
    (3, 5, 9, 4, 3, 7, "fp16", "any"),
    (64, 896, 896, 0, 16, 3584, "bf16", "distinct"),
    (33, 30, 60, 30, 4, 1023, "fp32", "distinct"),
    (40, 16, 16, 0, 32, 130, "bf16", "any"),
    (65, 2048, 2048, 0, 5, 260, "fp16", "distinct"),
    (256, 448, 896, 448, 16, 264, "bf16", "distinct"),     # 4096 slots: the last one-launch size
    (241, 448, 896, 0, 17, 264, "bf16", "any"),            # 4097 slots: the range sort
    (1500, 2048, 2048, 0, 5, 33, "fp32", "distinct"),
    (1025, 3, 3, 0, 9, 65, "bf16", "any"),
    (2048, 64, 64, 0, 8, 96, "fp16", "one"),
    (1200, 7, 7, 0, 4, 40, "bf16", "none"),
    (20, 7, 7, 0, 4, 40, "bf16", "none"),
    (700, 1, 1, 0, 1, 4104, "bf16", "one"),
    (9000, 100, 100, 0, 1, 15, "fp16", "distinct"),
]


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(map(str, c)))
def test_dispatch_and_combine(case):
    T, E, experts, offset, topk, H, dtype, mode = case
    say(f"[ops] routing {case}")
    rng = np.random.default_rng(T * 100003 + H * 101 + topk)
    ids = _ids(rng, T, topk, experts, mode)
    off, row_slot, slot_row = ref_maps(ids, E, offset)
    R, S, dt = int(off[-1]), T * topk, TORCH[dtype]
    shape = moe.DispatchShape(T=T, E=E, topk=topk, H=H, dtype=dtype, expert_offset=offset)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dt).cuda()
    rows, rows0 = _filled((S, H), dt)
    rs = torch.full((S,), -77, dtype=torch.int32, device="cuda")
    got = moe.dispatch(x, torch.from_numpy(ids).cuda(), shape, out=rows, row_slot=rs)
    torch.cuda.synchronize()
    assert _same(got[1], off) and _same(got[3], slot_row)
    assert _same(got[2][:R], row_slot) and bool((got[2][R:] == -77).all())
    assert torch.equal(rows[:R], x[torch.from_numpy(row_slot // topk).cuda()])
    assert torch.equal(rows[R:], rows0[R:])

    # the gradient of dispatch, and combine, from rows with NaN behind the last
    # expert's and weights that are no numbers where there is no row
    y = torch.from_numpy(rng.standard_normal((S, H))).to(dt).cuda()
    y[R:] = float("nan")
    w = rng.standard_normal((T, topk)).astype(np.float32)
    w[slot_row < 0] = np.where(rng.random((slot_row < 0).sum()) < 0.5, np.nan, np.inf)
    wt = torch.from_numpy(w).cuda()
    for name, wts in (("dispatch_backward", np.ones_like(w)), ("combine", w)):
        out, _ = _filled((T, H), dt)
        if name == "combine":
            moe.combine(y, got[3], wt, shape, out=out)
        else:
            moe.dispatch_backward(y, got[3], shape, out=out)
        torch.cuda.synchronize()
        ref, mag = ref_combine(f64(y), slot_row, wts.astype(np.float64))
        # a term passes its product and at most topk additions
        _close(out, ref, round_tol(ref, dtype, (topk + 1) * 2.0 ** -24 * mag), name)
        assert not f64(out)[(slot_row < 0).all(1)].any()  # tokens without a row: zeros

    dout = torch.from_numpy(rng.standard_normal((T, H))).to(dt).cuda()
    dy, dy0 = _filled((S, H), dt)
    dy, dw = moe.combine_backward(dout, y, got[3], wt, shape, dy=dy)
    torch.cuda.synchronize()
    rdy, rdw, mag = ref_combine_backward(f64(dout), f64(y), slot_row, w.astype(np.float64))
    assert torch.equal(dy[R:], dy0[R:])
    _close(dy[:R], rdy[:R], round_tol(rdy[:R], dtype, np.abs(rdy[:R]) * 2.0 ** -24), "drows")
    # a product, then a lane's H / 64 + 8 additions and the six between lanes
    _close(dw, rdw, (H / 64 + 16) * 2.0 ** -24 * mag, "dtopk_w")
    assert not f64(dw)[slot_row < 0].any()


def test_dispatch_of_no_tokens_writes_offsets():
    shape = moe.DispatchShape(T=0, E=5, topk=2, H=16)
    offsets = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    x = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    rows, off, _, slot_row = moe.dispatch(x, ids, shape, offsets=offsets)
    assert off.tolist() == [0] * 6 and rows.shape == (0, 16)
    w = torch.empty((0, 2), device="cuda")
    assert moe.combine(rows, slot_row, w, shape).shape == (0, 16)
    assert moe.dispatch_backward(rows, slot_row, shape).shape == (0, 16)
    dy, dw = moe.combine_backward(x, rows, slot_row, w, shape)
    assert dy.shape == (0, 16) and dw.shape == (0, 2)


@pytest.mark.parametrize("H", [512, 513])
@pytest.mark.parametrize("T", [48, 700])
def test_rows_at_any_element_address(T, H):
    # tensors that start one element into their storage: no 4-byte alignment
    topk, E = 8, 12
    rng = np.random.default_rng(T * H)
    ids = _ids(rng, T, topk, E, "any")
    off, row_slot, slot_row = ref_maps(ids, E, 0)
    R, S = int(off[-1]), T * topk
    shape = moe.DispatchShape(T=T, E=E, topk=topk, H=H)

    def odd(n):
        return torch.randn(n * H + 1, device="cuda").to(torch.bfloat16)[1:].view(n, H)

    x, out, tok = odd(T), odd(S), odd(T)
    got = moe.dispatch(x, torch.from_numpy(ids).cuda(), shape, out=out)
    assert torch.equal(out[:R], x[torch.from_numpy(row_slot // topk).cuda()])
    w = torch.rand(T, topk, device="cuda")
    moe.combine(out, got[3], w, shape, out=tok)
    ref, mag = ref_combine(f64(out), slot_row, f64(w))
    _close(tok, ref, round_tol(ref, "bf16", (topk + 1) * 2.0 ** -24 * mag), "combine")
    dout, dy = odd(T), odd(S)
    _, dw = moe.combine_backward(dout, out, got[3], w, shape, dy=dy)
    rdy, rdw, mag = ref_combine_backward(f64(dout), f64(out), slot_row, f64(w))
    _close(dy[:R], rdy[:R], round_tol(rdy[:R], "bf16", np.abs(rdy[:R]) * 2.0 ** -24), "drows")
    _close(dw, rdw, (H / 64 + 16) * 2.0 ** -24 * mag, "dtopk_w")


def test_combine_ignores_rows_outside_the_array():
    T, topk, H = 5, 3, 72
    shape = moe.DispatchShape(T=T, E=4, topk=topk, H=H, dtype="fp32")
    rows = torch.randn(T * topk, H, device="cuda")
    good = np.arange(T * topk, dtype=np.int32).reshape(T, topk)
    bad = good.copy()
    bad[0, 1], bad[2, 0], bad[3, 2], bad[4] = T * topk, 2 ** 31 - 1, -2 ** 31, -5
    w = torch.rand(T, topk, device="cuda")
    kept = np.where((bad >= 0) & (bad < T * topk), bad, -1)
    ref, mag = ref_combine(f64(rows), kept, f64(w))
    m = torch.from_numpy(bad).cuda()
    _close(moe.combine(rows, m, w, shape), ref, round_tol(ref, "fp32", 4 * 2.0 ** -24 * mag), "combine")
    dout = torch.randn(T, H, device="cuda")
    dy, dy0 = _filled((T * topk, H), torch.float32)
    _, dw = moe.combine_backward(dout, rows, m, w, shape, dy=dy)
    rdy, rdw, mag = ref_combine_backward(f64(dout), f64(rows), kept, f64(w))
    gone = np.isnan(rdy)
    assert torch.equal(dy[torch.from_numpy(gone).cuda()], dy0[torch.from_numpy(gone).cuda()])
    _close(dw, rdw, (H / 64 + 16) * 2.0 ** -24 * mag, "dtopk_w")


def test_gradients_against_differences():
    """L = <g, combine(dispatch(x) * a, w)> is linear in x and in w: the
    difference L(+d) - L(-d) over 2 is the derivative along d, up to the 32-bit
    rounding of the operators."""
    T, topk, E, H = 37, 4, 10, 203
    rng = np.random.default_rng(5)
    ids = torch.from_numpy(_ids(rng, T, topk, E, "any")).cuda()
    shape = moe.DispatchShape(T=T, E=E, topk=topk, H=H, dtype="fp32")
    x, g, dx = (torch.randn(T, H, device="cuda") for _ in range(3))
    a = torch.randn(T * topk, H, device="cuda")
    w, dw = torch.randn(T, topk, device="cuda"), torch.randn(T, topk, device="cuda")
    rows = torch.zeros(T * topk, H, device="cuda")
    _, _, _, slot_row = moe.dispatch(x, ids, shape, out=rows)

    def loss(xx, ww):
        r = torch.zeros(T * topk, H, device="cuda")
        moe.dispatch(xx, ids, shape, out=r)
        out = moe.combine(r * a, slot_row, ww, shape)
        return float((out.double() * g.double()).sum()), float((out.abs().double() * g.abs().double()).sum())

    drows = torch.zeros(T * topk, H, device="cuda")
    _, grad_w = moe.combine_backward(g, rows * a, slot_row, w, shape, dy=drows)
    grad_x = moe.dispatch_backward(drows * a, slot_row, shape)
    for which, d in (("x", dx), ("w", dw)):
        lp, mp = loss(x + d, w) if which == "x" else loss(x, w + d)
        lm, mm = loss(x - d, w) if which == "x" else loss(x, w - d)
        grad = grad_x if which == "x" else grad_w
        want = (lp - lm) / 2
        got = float((grad.double() * d.double()).sum())
        # every value passes some (topk + 4) 32-bit roundings on either side, the
        # dot products H / 64 + 16 more; magnitudes bounded by those of the terms
        big = float((grad.abs().double() * d.abs().double()).sum()) + mp + mm
        mags = float((rows * a).abs().double().sum()) * float(g.abs().max()) * float(w.abs().max() + dw.abs().max())
        tol = (topk + 4 + H / 64 + 16) * 2.0 ** -24 * (big + mags)
        assert abs(got - want) <= tol, (which, got, want, tol)


# ------------------------------------------------------------------ products


def _matrix(rng, E, N, K, fmt, group, dtype, zeros, scales=None):
    codes = rng.integers(0, 16, size=(E, N, K)).astype(np.int64)
    if fmt == "mxfp4":
        s = rng.integers(118, 128, size=(E, N, K // 32)).astype(np.uint8) if scales is None else scales
        st, s64 = torch.from_numpy(s).cuda(), s
    else:
        s = rng.uniform(-0.02, 0.02, size=(E, N, K // group)) if scales is None else scales
        st = torch.from_numpy(s).to(TORCH[dtype]).cuda()
        s64 = f64(st)
    z = rng.integers(0, 16, size=(E, N, K // group)).astype(np.uint8) if zeros else None
    wt = moe.prepack(torch.from_numpy(pack_rows(codes)).cuda())
    return dict(w=wt, scales=st, zeros=None if z is None else torch.from_numpy(z).cuda()), \
        ref_weights(codes, s64, z, fmt, group)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,group,zeros", [("mxfp4", 32, False), ("int4", 32, True),
                                             ("int4", 64, True), ("int4", 128, True), ("int4", 32, False)])
def test_every_weight_comes_out_exactly(fmt, group, zeros, dtype):
    # x is the identity: out[k, n] is weight [n, k], exact in 32 bits (a scale of
    # 8 or 11 bits times codes and zero points of 4)
    K, N = 256, 50
    say(f"[ops] identity {fmt} {group} {dtype}")
    rng = np.random.default_rng(group)
    m, (W, _) = _matrix(rng, 1, N, K, fmt, group, dtype, zeros)
    shape = moe.W4Shape(M=K, N=N, K=K, format=fmt, group=group, dtype=dtype, out_dtype="fp32")
    x = torch.eye(K, device="cuda").to(TORCH[dtype])
    got = moe.w4_linear(x, m["w"], m["scales"], shape, zeros=m["zeros"])
    assert np.array_equal(f64(got), W[0].T)


# M, N, K, fmt, group, dtype, out dtype, zeros, bias
LINEAR = [
    (1, 1, 128, "mxfp4", 32, "bf16", "bf16", False, False),
    (1, 16, 128, "int4", 128, "fp16", "fp16", False, False),
    (1, 100, 384, "mxfp4", 32, "fp16", "fp32", False, True),
    (2, 17, 896, "int4", 32, "bf16", "bf16", True, True),
    (3, 130, 1024, "int4", 64, "bf16", "fp32", True, False),
    (15, 65, 1152, "mxfp4", 32, "bf16", "fp32", False, False),
    (16, 200, 2048, "int4", 128, "bf16", "fp16", True, True),
    (17, 33, 1024, "mxfp4", 32, "fp16", "fp16", False, True),
    (32, 48, 2176, "int4", 32, "fp16", "fp32", False, False),
    (33, 70, 1280, "mxfp4", 32, "bf16", "bf16", False, True),
    (63, 129, 640, "int4", 64, "fp16", "fp16", True, False),
    (64, 16, 8192, "int4", 128, "fp16", "fp32", True, False),
    (65, 300, 256, "mxfp4", 32, "bf16", "fp32", False, False),
    (130, 257, 1408, "int4", 64, "bf16", "bf16", False, True),
    (5, 1000, 8192, "mxfp4", 32, "bf16", "fp32", False, False),
    (7, 5000, 128, "mxfp4", 32, "bf16", "bf16", False, False),
    (1, 7168, 2048, "mxfp4", 32, "bf16", "bf16", False, False),
    # many weight groups: four to a wave, K split over the waves, or not (short K)
    (3, 32900, 1024, "mxfp4", 32, "bf16", "bf16", False, True),
    (16, 32770, 1152, "int4", 32, "bf16", "fp32", True, False),
    (6, 200000, 128, "int4", 64, "fp16", "fp16", True, False),
    (20, 40001, 256, "int4", 128, "bf16", "bf16", False, False),
    (50, 40001, 256, "mxfp4", 32, "fp16", "fp32", False, False),
    (70, 9000, 2048, "int4", 128, "fp16", "fp16", True, False),
    (49, 900, 1024, "int4", 32, "bf16", "fp32", True, True),
    # K over eight waves
    (9, 5000, 2176, "int4", 64, "bf16", "fp32", False, True),
    (12, 40, 7168, "int4", 32, "fp16", "fp32", True, False),
]


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(map(str, c)))
def test_w4_linear(case):
    M, N, K, fmt, group, dtype, odt, zeros, bias = case
    say(f"[ops] linear {case}")
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    m, (W, mag) = _matrix(rng, 1, N, K, fmt, group, dtype, zeros)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(TORCH[dtype]).cuda()
    b = torch.from_numpy(rng.standard_normal((1, N))).to(TORCH[dtype]).cuda() if bias else None
    shape = moe.W4Shape(M=M, N=N, K=K, format=fmt, group=group, dtype=dtype, out_dtype=odt)
    got = moe.w4_linear(x, m["w"], m["scales"], shape, zeros=m["zeros"], bias=b)
    again = moe.w4_linear(x, m["w"][0], m["scales"][0], shape,
                          zeros=None if m["zeros"] is None else m["zeros"][0],
                          bias=None if b is None else b[0])
    torch.cuda.synchronize()
    assert torch.equal(got, again)  # the same bits again; matrices without the leading 1
    ref = f64(x) @ W[0].T + (f64(b)[0] if bias else 0)
    size = np.abs(f64(x)) @ mag[0].T + (np.abs(f64(b)[0]) if bias else 0)
    _close(got, ref, round_tol(ref, odt, sum_tol(K) * size), "out")


def test_w4_linear_strided_rows():
    M, N, K = 19, 45, 1152
    rng = np.random.default_rng(3)
    m, (W, mag) = _matrix(rng, 1, N, K, "int4", 64, "bf16", True)
    wide = torch.from_numpy(rng.standard_normal((M, 3 * K))).to(torch.bfloat16).cuda()
    x = wide[:, K:2 * K]
    big, big0 = _filled((M, N + 11), torch.float32)
    shape = moe.W4Shape(M=M, N=N, K=K, format="int4", group=64, out_dtype="fp32")
    moe.w4_linear(x, m["w"], m["scales"], shape, zeros=m["zeros"], out=big[:, 3:3 + N])
    torch.cuda.synchronize()
    assert torch.equal(big[:, :3], big0[:, :3]) and torch.equal(big[:, 3 + N:], big0[:, 3 + N:])
    ref, size = f64(x) @ W[0].T, np.abs(f64(x)) @ mag[0].T
    _close(big[:, 3:3 + N], ref, round_tol(ref, "fp32", sum_tol(K) * size), "out")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_mxfp4_scale_bytes_at_their_ends(dtype):
    # one scale byte a weight row, tokens that keep the result in range
    K, bytes_ = 128, [0, 1, 2, 100, 127, 200, 252, 255]
    N = len(bytes_)
    rng = np.random.default_rng(1)
    scales = np.repeat(np.array(bytes_, np.uint8)[None, :, None], K // 32, 2)
    m, (W, mag) = _matrix(rng, 1, N, K, "mxfp4", 32, dtype, False, scales)
    x = torch.from_numpy(rng.standard_normal((4, K)) * 2.0 ** -6).to(TORCH[dtype]).cuda()
    shape = moe.W4Shape(M=4, N=N, K=K, dtype=dtype, out_dtype="fp32")
    got = f64(moe.w4_linear(x, m["w"], m["scales"], shape))
    assert np.isnan(got[:, -1]).all()
    ref, size = f64(x) @ W[0, :-1].T, np.abs(f64(x)) @ mag[0, :-1].T
    _close(torch.from_numpy(got[:, :-1]), ref, round_tol(ref, "fp32", sum_tol(K) * size) + 128 * 2.0 ** -149, "out")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scales_that_are_no_numbers_stay_in_their_weight_row(dtype):
    K, N = 1152, 40
    rng = np.random.default_rng(2)
    scales = rng.uniform(0.01, 0.02, size=(1, N, K // 128))
    scales[0, 3, 4], scales[0, 20, 0], scales[0, 39, 8], scales[0, 7] = np.nan, np.inf, -np.inf, 0.0
    m, (W, mag) = _matrix(rng, 1, N, K, "int4", 128, dtype, False, scales)
    x = torch.from_numpy(rng.standard_normal((3, K))).to(TORCH[dtype]).cuda()
    shape = moe.W4Shape(M=3, N=N, K=K, format="int4", group=128, dtype=dtype, out_dtype="fp32")
    got = f64(moe.w4_linear(x, m["w"], m["scales"], shape))
    odd = [3, 20, 39]
    assert not np.isfinite(got[:, odd]).any()
    rest = np.setdiff1d(np.arange(N), odd)
    ref, size = f64(x) @ W[0, rest].T, np.abs(f64(x)) @ mag[0, rest].T
    _close(torch.from_numpy(got[:, rest]), ref, round_tol(ref, "fp32", sum_tol(K) * size), "out")
    assert not got[:, 7].any()


@pytest.mark.parametrize("dtype,step", [("fp16", 2.0 ** -24), ("bf16", 2.0 ** -133)])
def test_subnormal_tokens_count(dtype, step):
    # tokens of 0 to 3 of the type's smallest steps: every sum is exact in 32 bits
    K, N, M = 256, 20, 5
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.integers(0, 4, size=(M, K)) * step).to(TORCH[dtype]).cuda()
    scale = 2.0 ** 10
    m, (W, _) = _matrix(rng, 1, N, K, "int4", 128, dtype, True, np.full((1, N, K // 128), scale))
    shape = moe.W4Shape(M=M, N=N, K=K, format="int4", group=128, dtype=dtype, out_dtype="fp32")
    got = moe.w4_linear(x, m["w"], m["scales"], shape, zeros=m["zeros"])
    assert np.array_equal(f64(got), f64(x) @ W[0].T)


def test_rows_of_x_do_not_meet():
    # a row of infinities and one of NaN: the others are as without them
    M, N, K = 20, 50, 1024
    rng = np.random.default_rng(4)
    for fmt, group in (("mxfp4", 32), ("int4", 32)):
        m, _ = _matrix(rng, 1, N, K, fmt, group, "bf16", fmt == "int4")
        x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16).cuda()
        shape = moe.W4Shape(M=M, N=N, K=K, format=fmt, group=group)
        want = moe.w4_linear(x, m["w"], m["scales"], shape, zeros=m["zeros"])
        x2 = x.clone()
        x2[5], x2[17, 3] = float("nan"), float("inf")
        got = moe.w4_linear(x2, m["w"], m["scales"], shape, zeros=m["zeros"])
        keep = [i for i in range(M) if i not in (5, 17)]
        assert torch.equal(got[keep], want[keep])
        assert bool(got[5].isnan().all()) and not bool(got[17].isfinite().any())


# rows of each expert, rows behind, N, K, fmt, group, dtype, out dtype, zeros, bias
GROUPED = [
    ([1], 0, 30, 128, "mxfp4", 32, "bf16", "bf16", False, False),
    ([0, 3, 0, 0, 20, 1, 16, 17, 0], 5, 70, 256, "mxfp4", 32, "bf16", "fp32", False, True),
    ([0, 0, 0, 40], 3, 33, 1024, "int4", 64, "fp16", "fp16", True, True),
    ([70, 0, 1, 130], 0, 50, 1152, "int4", 128, "bf16", "bf16", False, False),
    ([0, 0, 0], 4, 16, 128, "int4", 32, "bf16", "bf16", False, False),
    ([2] * 100, 700, 20, 384, "mxfp4", 32, "fp16", "fp32", False, False),
    ([33, 34, 31, 0, 90], 0, 100, 1536, "mxfp4", 32, "bf16", "bf16", False, False),
    ([5, 1, 0, 3], 100, 768, 3584, "mxfp4", 32, "bf16", "fp32", False, False),
    # many rows an expert: tiles of 64, their ragged ends
    ([400, 0, 17, 70, 33, 1, 5, 330], 200, 50, 1152, "mxfp4", 32, "fp16", "fp32", False, True),
    ([300, 40], 30, 600, 256, "int4", 64, "bf16", "bf16", True, False),
    ([300, 40], 30, 600, 256, "int4", 32, "bf16", "bf16", True, False),
    # one wave a weight group's K, and zero points and scales that would not fit LDS then
    ([1, 0, 3, 5, 9, 2] * 20, 3, 500, 384, "int4", 32, "bf16", "fp32", True, True),
    ([2, 1] * 8, 0, 4096, 8192, "int4", 32, "fp16", "fp32", True, False),
]


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "-".join(map(str, [len(c[0]), *c[1:]])))
def test_w4_grouped_linear(case):
    counts, behind, N, K, fmt, group, dtype, odt, zeros, bias = case
    say(f"[ops] grouped {case}")
    E, R = len(counts), sum(counts)
    M = R + behind
    rng = np.random.default_rng(R * 31 + K)
    m, (W, mag) = _matrix(rng, E, N, K, fmt, group, dtype, zeros)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(TORCH[dtype]).cuda()
    x[R:] = float("nan")
    b = torch.from_numpy(rng.standard_normal((E, N))).to(TORCH[dtype]).cuda() if bias else None
    shape = moe.W4Shape(M=M, N=N, K=K, E=E, format=fmt, group=group, dtype=dtype, out_dtype=odt)
    out, out0 = _filled((M, N), TORCH[odt])
    moe.w4_grouped_linear(x, torch.from_numpy(off).cuda(), m["w"], m["scales"], shape,
                          zeros=m["zeros"], bias=b, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[R:], out0[R:])
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        ref = f64(x[lo:hi]) @ W[e].T + (f64(b)[e] if bias else 0)
        size = np.abs(f64(x[lo:hi])) @ mag[e].T + (np.abs(f64(b)[e]) if bias else 0)
        _close(out[lo:hi], ref, round_tol(ref, odt, sum_tol(K) * size), f"expert {e}")


def test_w4_grouped_linear_clamps_offsets():
    # offsets past M count as M, decreasing ones own nothing; nothing outside is touched
    E, M, N, K = 5, 12, 40, 256
    rng = np.random.default_rng(11)
    m, (W, mag) = _matrix(rng, E, N, K, "mxfp4", 32, "bf16", False)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16).cuda()
    shape = moe.W4Shape(M=M, N=N, K=K, E=E, out_dtype="fp32")
    for off in ([0, 3, 3, 9, 50, 2 ** 31 - 1], [2, 1, 4, 4, 12, 3], [-7, 2, 5, -2 ** 31, 8, 8]):
        out, out0 = _filled((M, N), torch.float32)
        moe.w4_grouped_linear(x, torch.tensor(off, dtype=torch.int32, device="cuda"), m["w"],
                              m["scales"], shape, out=out)
        owner = np.full(M, -1)
        for e in range(E):
            owner[max(off[e], 0):max(min(off[e + 1], M), 0)] = e
        none = torch.from_numpy(owner < 0).cuda()
        if off[0] == 0 or off[0] == 2:
            assert torch.equal(out[none], out0[none])
        else:
            continue  # a row may have two owners: only its place in the buffer is promised
        for r in np.nonzero(owner >= 0)[0]:
            ref, size = W[owner[r]] @ f64(x[r]), mag[owner[r]] @ np.abs(f64(x[r]))
            _close(out[r], ref, round_tol(ref, "fp32", sum_tol(K) * size), f"row {r}")


def test_most_experts():
    E, N, K = 2048, 18, 128
    rng = np.random.default_rng(8)
    counts = rng.integers(0, 3, size=E)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1])
    m, (W, mag) = _matrix(rng, E, N, K, "mxfp4", 32, "bf16", False)
    x = torch.from_numpy(rng.standard_normal((R, K))).to(torch.bfloat16).cuda()
    shape = moe.W4Shape(M=R, N=N, K=K, E=E)
    got = moe.w4_grouped_linear(x, torch.from_numpy(off).cuda(), m["w"], m["scales"], shape)
    e = np.repeat(np.arange(E), counts)
    ref = np.einsum("rk,rnk->rn", f64(x), W[e])
    size = np.einsum("rk,rnk->rn", np.abs(f64(x)), mag[e])
    _close(got, ref, round_tol(ref, "bf16", sum_tol(K) * size), "out")


# ------------------------------------------------------------------ together


def _layer(dev, s, ids, w, shape, sw13, sw2):
    """The layer from the operators: dispatch, both products, combine."""
    rows, offsets, _, slot_row = moe.dispatch(dev["x"], ids, shape)
    h = moe.w4_grouped_linear(rows, offsets, dev["w13"], dev["s13"], sw13)
    g, u = h[:, :s.I], h[:, s.I:]
    act = (torch.nn.functional.silu(g) * u).to(torch.bfloat16)
    y = moe.w4_grouped_linear(act, offsets, dev["w2"], dev["s2"], sw2)
    return moe.combine(y, slot_row, w, shape)


@pytest.mark.parametrize("s", [
    LayerShape("ops_decode", T=64, E=48, E_g=96, topk=6, H=1024, I=256, B=16, expert_offset=48, mode="ids"),
    LayerShape("ops_prompt", T=600, E=16, E_g=16, topk=8, H=512, I=128, B=64, mode="ids"),
], ids=lambda s: s.name)
def test_the_operators_make_the_layer(s):
    """dispatch -> product -> SwiGLU -> product -> combine on the layer's own
    weights, against the layer's oracle, and with a graph that replays it over
    new inputs between eager calls."""
    say(f"[ops] layer {s.name}")
    sets = []
    dev = None
    for seed in (41, 42):
        inp = make_inputs(s, seed, weights=True)
        if dev is None:
            dev, first = to_device(s, inp), inp
        inp = {**inp, **{k: first[k] for k in ("w13", "s13", "w2", "s2")}}
        ids, w = torch.from_numpy(inp["topk_ids"]).cuda(), torch.from_numpy(inp["topk_w"]).cuda()
        x = torch.from_numpy(inp["x"].view(np.int16)).cuda().view(torch.bfloat16)
        sets.append((inp, x, ids, w))
    S = s.T * s.topk
    shape = moe.DispatchShape(T=s.T, E=s.E, topk=s.topk, H=s.H, expert_offset=s.expert_offset)
    sw13 = moe.W4Shape(M=S, N=2 * s.I, K=s.H, E=s.E, out_dtype="fp32")
    sw2 = moe.W4Shape(M=S, N=s.H, K=s.I, E=s.E)
    want = []
    for inp, x, ids, w in sets:
        dev["x"] = x
        out = _layer(dev, s, ids, w, shape, sw13, sw2)
        check_out(out_np(out), oracle.reference_forward(s, inp)["out"], s.name)
        want.append(out.clone())

    dev["x"], ids, w = sets[0][1].clone(), sets[0][2].clone(), sets[0][3].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):  # another stream than the default one, then captured on it
        assert torch.equal(_layer(dev, s, ids, w, shape, sw13, sw2), want[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = _layer(dev, s, ids, w, shape, sw13, sw2)
    torch.cuda.synchronize()
    for i in (0, 1, 1, 0, 1):
        dev["x"].copy_(sets[i][1])
        ids.copy_(sets[i][2])
        w.copy_(sets[i][3])
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), f"replay of set {i} differs"


def test_training_step_repeats_bit_for_bit():
    T, topk, E, H = 300, 8, 32, 520
    rng = np.random.default_rng(9)
    ids = torch.from_numpy(_ids(rng, T, topk, E)).cuda()
    shape = moe.DispatchShape(T=T, E=E, topk=topk, H=H)
    x, dout = (torch.randn(T, H, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.rand(T, topk, device="cuda")

    def step():
        rows, _, _, slot_row = moe.dispatch(x, ids, shape)
        out = moe.combine(rows, slot_row, w, shape)
        drows, dw = moe.combine_backward(dout, rows, slot_row, w, shape)
        return out, drows, dw, moe.dispatch_backward(drows, slot_row, shape)

    want = step()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        got = step()
    for i in range(4):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {i}"
        assert all(torch.equal(a, b) for a, b in zip(step(), want))


def test_stream_argument():
    """Calls on a stream given by its handle, which allocate their outputs, while
    the current stream is another: in order on theirs, and as on the default one."""
    T, topk, E, H, N = 700, 8, 16, 512, 640
    rng = np.random.default_rng(21)
    ids = torch.from_numpy(_ids(rng, T, topk, E)).cuda()
    shape = moe.DispatchShape(T=T, E=E, topk=topk, H=H)
    m, _ = _matrix(rng, E, N, H, "mxfp4", 32, "bf16", False)
    ws = moe.W4Shape(M=T * topk, N=N, K=H, E=E)
    back = moe.DispatchShape(T=T, E=E, topk=topk, H=N)
    x, w = torch.randn(T, H, device="cuda").to(torch.bfloat16), torch.rand(T, topk, device="cuda")

    def chain(**kw):
        rows, off, _, slot_row = moe.dispatch(x, ids, shape, **kw)
        return moe.combine(moe.w4_grouped_linear(rows, off, m["w"], m["scales"], ws, **kw), slot_row, w, back, **kw)

    want = chain()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = [chain(stream=s.cuda_stream) for s in side for _ in range(3)]  # three chains at once
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_first_call_inside_a_capture():
    # a process whose first call of every operator is captured
    code = """
import torch, mxfp4_weight_expert_amd as moe
x = torch.randn(6, 256, device="cuda").to(torch.bfloat16)
ids = torch.tensor([[0, 1]] * 6, dtype=torch.int32, device="cuda")
w = torch.ones(6, 2, device="cuda")
s = moe.DispatchShape(T=6, E=2, topk=2, H=256)
ws = moe.W4Shape(M=12, N=32, K=256, E=2, out_dtype="fp32")
c = torch.randint(0, 256, (2, 32, 128), dtype=torch.uint8, device="cuda")
sc = torch.full((2, 32, 8), 127, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
def run():
    rows, off, _, back = moe.dispatch(x, ids, s)
    y = moe.w4_grouped_linear(rows, off, c, sc, ws)
    out = moe.combine(rows, back, w, s)
    d, dw = moe.combine_backward(out, rows, back, w, s)
    return y, out, d, dw, moe.dispatch_backward(d, back, s)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
for _ in range(3):
    g.replay()
    want = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_rows_past_32_bit_offsets():
    # 655,360 rows of 8 KB: 5.4 GB of rows, with a twin of the last token's slots
    T, topk, E, H = 20480, 32, 40, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(topk, 1).indices.to(torch.int32)
    shape = moe.DispatchShape(T=T, E=E, topk=topk, H=H)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    rows, off, row_slot, slot_row = moe.dispatch(x, ids, shape)
    order = torch.sort(ids.view(-1).long() * (T * topk) + torch.arange(T * topk, device="cuda")).values % (T * topk)
    assert torch.equal(row_slot.long(), order) and int(off[-1]) == T * topk
    at = torch.cat([torch.arange(0, T * topk, 997, device="cuda"), torch.arange(T * topk - 64, T * topk, device="cuda")])
    assert torch.equal(rows[at], x[order[at] // topk])
    w = torch.ones(T, topk, device="cuda")
    out = moe.combine(rows, slot_row, w, shape)
    t = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    # topk equal terms: exact sums of up to 32 copies but for the last rounding
    assert torch.equal(out[t], (x[t].float() * topk).to(torch.bfloat16))
    drows, dw = moe.combine_backward(x, rows, slot_row, w, shape)
    assert torch.equal(drows[at], rows[at])
    ref = (f64(x[t]) ** 2).sum(1)[:, None].repeat(topk, 1)
    _close(dw[t], ref, (H / 64 + 16) * 2.0 ** -24 * ref, "dtopk_w")


def test_weights_past_32_bit_offsets():
    # 130 matrices of 8192 x 8192: 4.4 GB of codes; rows for the first and last
    E, N, K = 130, 8192, 8192
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sc = torch.randint(118, 128, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn(6, K, generator=g, device="cuda").to(torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:], off[-2], off[-1] = 2, 3, 6
    got = moe.w4_grouped_linear(x, off, w, sc, moe.W4Shape(M=6, N=N, K=K, E=E, out_dtype="fp32"))
    one = moe.W4Shape(M=6, N=N, K=K, out_dtype="fp32")
    for e, lo, hi in ((0, 0, 2), (E - 2, 2, 3), (E - 1, 3, 6)):
        alone = moe.w4_linear(x, w[e].clone(), sc[e].clone(), one)[lo:hi]
        codes = w[e].view(N // 16, K // 128, 16, 64).transpose(1, 2).reshape(N, K // 2)[-32:]
        codes = torch.stack([codes & 15, codes >> 4], -1).view(32, K).cpu().numpy()
        W, mag = ref_weights(codes, sc[e, -32:].cpu().numpy(), None, "mxfp4", 32)
        ref, size = f64(x[lo:hi]) @ W.T, np.abs(f64(x[lo:hi])) @ mag.T
        tol = round_tol(ref, "fp32", sum_tol(K) * size)
        _close(got[lo:hi, -32:], ref, tol, f"matrix {e}")
        _close(alone[:, -32:], ref, tol, f"matrix {e} alone")


def test_binding_refusals_on_the_gpu():
    shape = moe.DispatchShape(T=4, E=4, topk=2, H=16)
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="topk_ids is on cpu"):
        moe.dispatch(x, ids.cpu(), shape)
    with pytest.raises(moe.MoeError) as ei:
        moe.dispatch(x, ids, shape, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert ei.value.code == 3
    with pytest.raises(moe.MoeError) as ei:
        moe.dispatch(x, ids, moe.DispatchShape(T=4, E=4, topk=2, H=16, expert_offset=-1))
    assert ei.value.code == 1
    rows = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError) as ei:  # the sum over its own rows
        moe.combine(rows, ids, torch.zeros(4, 2, device="cuda"), shape, out=rows[2:6])
    assert ei.value.code == 1
