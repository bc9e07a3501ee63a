"""Dispatch, combine and the 4-bit products as a program meets them: tensors that
autograd follows, memory shared by several tensors, batches routed otherwise, and
values that are no numbers."""
import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe

from gpu_util import say
from ops_util import TORCH, f64, pack_rows, ref_combine, ref_combine_backward, ref_maps, ref_weights, round_tol, sum_tol

pytestmark = pytest.mark.gpu


def _close(got, ref, tol, what):
    err = np.abs(f64(got) - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / tol):.2f} tolerances"


def _matrices(rng, E, N, K, fmt="mxfp4", group=32, dtype="bf16", zeros=False):
    """(arrays on the GPU, weights and their magnitudes in 64 bits)."""
    codes = rng.integers(0, 16, size=(E, N, K)).astype(np.int64)
    if fmt == "mxfp4":
        s = rng.integers(118, 128, size=(E, N, K // 32)).astype(np.uint8)
        st = torch.from_numpy(s).cuda()
    else:
        st = torch.from_numpy(rng.uniform(-0.02, 0.02, size=(E, N, K // group))).to(TORCH[dtype]).cuda()
        s = f64(st)
    z = rng.integers(0, 16, size=s.shape).astype(np.uint8) if zeros else None
    arrays = dict(w=moe.prepack(torch.from_numpy(pack_rows(codes)).cuda()), scales=st,
                  zeros=None if z is None else torch.from_numpy(z).cuda())
    return arrays, ref_weights(codes, s, z, fmt, group)


def _grouped(m, x, off, shape, **kw):
    off = torch.as_tensor(off, dtype=torch.int32).cuda()
    return moe.w4_grouped_linear(x, off, m["w"], m["scales"], shape, zeros=m["zeros"], **kw)


# ------------------------------------------------------------------ batches


# a wave reads all of K, of few and many weight groups a matrix, or a part of it
@pytest.mark.parametrize("N,K,fmt,group", [(768, 3584, "mxfp4", 32), (400, 1024, "int4", 64), (96, 8192, "mxfp4", 32)])
def test_a_rows_bits_do_not_depend_on_other_experts_rows(N, K, fmt, group):
    E, mine, M = 64, 41, 400
    rng = np.random.default_rng(K)
    m, _ = _matrices(rng, E, N, K, fmt, group)
    shape = moe.W4Shape(M=M, N=N, K=K, E=E, format=fmt, group=group, out_dtype="fp32")
    own = torch.from_numpy(rng.standard_normal((3, K))).to(torch.bfloat16).cuda()
    seen = []
    for trial in range(4):
        say(f"[ops] batch {trial} of {N} {K} {fmt}")
        counts = rng.integers(0, 1 + 2 ** trial, size=E)
        counts[mine] = 3
        off = np.minimum(np.concatenate([[0], np.cumsum(counts)]), M)
        lo = int(off[mine])
        x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16).cuda()
        x[lo:lo + 3] = own
        seen.append(_grouped(m, x, off, shape)[lo:lo + 3].clone())
    assert all(torch.equal(s, seen[0]) for s in seen[1:])


@pytest.mark.parametrize("M,N,K,fmt,group", [(150, 4000, 2048, "mxfp4", 32), (70, 9000, 1152, "int4", 32)])
def test_a_rows_bits_do_not_depend_on_its_place(M, N, K, fmt, group):
    rng = np.random.default_rng(M)
    m, _ = _matrices(rng, 1, N, K, fmt, group)
    shape = moe.W4Shape(M=M, N=N, K=K, format=fmt, group=group, out_dtype="fp32")
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16).cuda()
    at = torch.from_numpy(rng.permutation(M)).cuda()
    want = moe.w4_linear(x, m["w"], m["scales"], shape)
    assert torch.equal(moe.w4_linear(x[at], m["w"], m["scales"], shape), want[at])


# ------------------------------------------------------------------ autograd


def _routed(T=6, topk=2, E=4, H=128, dtype=torch.bfloat16):
    shape = moe.DispatchShape(T=T, E=E, topk=topk, H=H)
    ids = torch.arange(T * topk, dtype=torch.int32, device="cuda").view(T, topk) % E
    x = torch.randn(T, H, device="cuda").to(dtype)
    rows, off, _, back = moe.dispatch(x, ids, shape)
    return shape, ids, x, rows, off, back, torch.rand(T, topk, device="cuda")


def test_tensors_that_require_gradients_are_refused():
    shape, ids, x, rows, off, back, w = _routed()
    s = moe.W4Shape(M=12, N=32, K=128, E=4)
    c = torch.zeros(4, 32, 64, dtype=torch.uint8, device="cuda")
    sc = torch.full((4, 32, 4), 127, dtype=torch.uint8, device="cuda")
    bias = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    one = moe.W4Shape(M=12, N=32, K=128)

    def want(t):
        return t.detach().clone().requires_grad_()

    calls = {
        "x": [lambda: moe.dispatch(want(x), ids, shape),
              lambda: moe.w4_linear(want(rows), c[:1], sc[:1], one),
              lambda: moe.w4_grouped_linear(want(rows), off, c, sc, s)],
        "rows": [lambda: moe.combine(want(rows), back, w, shape),
                 lambda: moe.combine_backward(x, want(rows), back, w, shape)],
        "topk_w": [lambda: moe.combine(rows, back, want(w), shape),
                   lambda: moe.combine_backward(x, rows, back, want(w), shape)],
        "dout": [lambda: moe.combine_backward(want(x), rows, back, w, shape)],
        "drows": [lambda: moe.dispatch_backward(want(rows), back, shape)],
        "bias": [lambda: moe.w4_grouped_linear(rows, off, c, sc, s, bias=want(bias))],
        "out": [lambda: moe.combine(rows, back, w, shape, out=want(x)),
                lambda: moe.w4_linear(rows, c[:1], sc[:1], one, out=want(bias.new_zeros(12, 32)))],
    }
    for name, fs in calls.items():
        for f in fs:
            with pytest.raises(ValueError, match=f"{name} requires a gradient"):
                f()
            with torch.no_grad():
                f()  # where nothing is recorded, nothing is lost


def test_operators_inside_an_autograd_function():
    # forward and backward of a function run without recording: the operators take
    # the tensors there, leaves that require gradients among the saved ones
    shape, ids, x, _, _, _, w = _routed()

    class Routed(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            rows, _, _, back = moe.dispatch(x, ids, shape)
            ctx.save_for_backward(rows, back, w)
            return moe.combine(rows, back, w, shape)

        @staticmethod
        def backward(ctx, dout):
            rows, back, w = ctx.saved_tensors
            drows, dw = moe.combine_backward(dout.contiguous(), rows, back, w, shape)
            return moe.dispatch_backward(drows, back, shape), dw

    xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
    Routed.apply(xl, wl).float().sum().backward()
    # dout is 1: dx = sum_k w, each w rounded in its row of drows and the sum once more;
    # dw is the sum of the token's row
    sw = f64(w).sum(1, keepdims=True)
    _close(xl.grad, np.broadcast_to(sw, x.shape), 2.01 * sw * 2.0 ** -8 + 2.0 ** -20, "dx")
    ref = np.repeat(f64(x).sum(1)[:, None], 2, 1)
    _close(wl.grad, ref, 20 * 2.0 ** -24 * np.abs(f64(x)).sum(1)[:, None], "dw")


def test_outputs_given_count_as_changed():
    # a tensor that a recorded product saved, then given as an output: its old values
    # are gone, and the gradient that needs them has to be refused
    shape, ids, x, rows, off, back, w = _routed()
    s, one = moe.W4Shape(M=12, N=128, K=128, E=4), moe.W4Shape(M=12, N=128, K=128)
    c = torch.zeros(4, 128, 64, dtype=torch.uint8, device="cuda")
    sc = torch.full((4, 128, 4), 127, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    maps = dict(offsets=torch.zeros(5, **i32), row_slot=torch.zeros(12, **i32), slot_row=torch.zeros(6, 2, **i32))
    before = [t._version for t in maps.values()]
    moe.dispatch(x, ids, shape, **maps)
    assert all(t._version > v for t, v in zip(maps.values(), before))
    calls = [
        (rows, lambda b: moe.dispatch(x, ids, shape, out=b)),
        (x, lambda b: moe.combine(rows, back, w, shape, out=b)),
        (x, lambda b: moe.dispatch_backward(rows, back, shape, out=b)),
        (rows, lambda b: moe.combine_backward(x, rows, back, w, shape, dy=b)),
        (w, lambda b: moe.combine_backward(x, rows, back, w, shape, dw=b)),
        (rows, lambda b: moe.w4_linear(rows, c[:1], sc[:1], one, out=b)),
        (rows, lambda b: moe.w4_grouped_linear(rows, off, c, sc, s, out=b)),
    ]
    for like, call in calls:
        buf = torch.ones_like(like)
        leaf = torch.ones_like(like).requires_grad_()
        y = (leaf * buf).sum()
        call(buf)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    with torch.inference_mode():  # tensors without a version
        moe.combine(rows, back, w, shape, out=torch.zeros_like(x))


# ------------------------------------------------------------------ memory


@pytest.mark.parametrize("odt", ["bf16", "fp32"])
def test_x_and_out_as_columns_of_one_matrix(odt):
    # the rows of the one lie between the rows of the other, on either side
    M, N, K = 37, 72, 256
    rng = np.random.default_rng(12)
    m, (W, mag) = _matrices(rng, 1, N, K)
    size = 2 if odt == "bf16" else 4
    width = K + N * size // 2 + 8
    shape = moe.W4Shape(M=M, N=N, K=K, out_dtype=odt)
    for xfirst in (True, False):
        wide = torch.from_numpy(rng.standard_normal((M, width))).to(torch.bfloat16).cuda()
        at = 0 if xfirst else N * size // 2
        x = wide[:, at:at + K]
        out = wide.view(TORCH[odt])[:, 2 * K // size:2 * K // size + N] if xfirst else wide.view(TORCH[odt])[:, :N]
        keep, x0 = wide[:, at + K:] if not xfirst else wide[:, K + N * size // 2:], x.clone()
        keep0 = keep.clone()
        for grouped in (False, True):
            if grouped:
                _grouped(m, x, [0, M], shape, out=out)
            else:
                moe.w4_linear(x, m["w"], m["scales"], shape, out=out)
            torch.cuda.synchronize()
            assert torch.equal(x, x0) and torch.equal(keep, keep0)
            ref, mags = f64(x) @ W[0].T, np.abs(f64(x)) @ mag[0].T
            _close(out, ref, round_tol(ref, odt, sum_tol(K) * mags), f"x first {xfirst}, grouped {grouped}")


def test_offsets_that_count_a_row_twice_write_nowhere_else():
    # [-7, 2, 5, -2**31, 8, 8]: experts 0, 1 own rows 0-1, 2-4, expert 3 rows 0-7; the
    # rows that two own are one of the two results, and nothing else is written
    E, M, N, K, G = 5, 12, 40, 256, 16
    rng = np.random.default_rng(13)
    m, (W, mag) = _matrices(rng, E, N, K)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16).cuda()
    buf = torch.full((M + 2 * G, N + 5), 777.0, device="cuda")
    out = buf[G:G + M, 2:2 + N]
    _grouped(m, x, [-7, 2, 5, -2 ** 31, 8, 8], moe.W4Shape(M=M, N=N, K=K, E=E, out_dtype="fp32"), out=out)
    torch.cuda.synchronize()
    owners = [[0, 3]] * 2 + [[1, 3]] * 3 + [[3]] * 3
    got = f64(out)
    for r, es in enumerate(owners):
        ok = np.zeros(N, bool)
        for e in es:
            ref, size = W[e] @ f64(x[r]), mag[e] @ np.abs(f64(x[r]))
            ok |= np.abs(got[r] - ref) <= round_tol(ref, "fp32", sum_tol(K) * size)
        assert ok.all(), r
    buf[G:G + 8, 2:2 + N] = 777.0
    assert bool((buf == 777.0).all())


# ------------------------------------------------------------------ values


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_no_numbers_in_rows_that_count(dtype):
    # NaN and infinities reach the sums they take part in, and no others
    T, topk, E, H = 50, 3, 6, 1031
    rng = np.random.default_rng(14)
    ids = rng.integers(-1, E, size=(T, topk)).astype(np.int32)
    off, row_slot, slot_row = ref_maps(ids, E, 0)
    shape = moe.DispatchShape(T=T, E=E, topk=topk, H=H, dtype=dtype)
    rows = torch.from_numpy(rng.standard_normal((T * topk, H))).to(TORCH[dtype]).cuda()
    R = int(off[-1])
    rows[2, 5], rows[7, 1030], rows[R - 1, 512], rows[R:] = float("nan"), float("inf"), -float("inf"), float("nan")
    x = torch.from_numpy(rng.standard_normal((T, H))).to(TORCH[dtype]).cuda()
    dout = x.clone()
    dout[11, 8], dout[13, 1030] = float("inf"), float("nan")
    w = rng.standard_normal((T, topk)).astype(np.float32)
    w[20, 1] = 0.0
    wt, back = torch.from_numpy(w).cuda(), torch.from_numpy(slot_row.astype(np.int32)).cuda()

    def same(got, ref, err, what, dt):
        g, nan = f64(got), np.isnan(ref)
        assert np.array_equal(np.isnan(g), nan), what
        inf = np.isinf(ref)
        assert np.array_equal(g[inf], ref[inf]), what
        fin = ~(nan | inf)
        assert (np.abs(g - ref)[fin] <= (round_tol(ref[fin], dt, err[fin]) if dt else err[fin])).all(), what

    with np.errstate(invalid="ignore"):
        ref, mag = ref_combine(f64(rows), slot_row, w.astype(np.float64))
        same(moe.combine(rows, back, wt, shape), ref, (topk + 1) * 2.0 ** -24 * mag, "combine", dtype)
        ref, mag = ref_combine(f64(rows), slot_row, np.ones_like(w, dtype=np.float64))
        same(moe.dispatch_backward(rows, back, shape), ref, (topk + 1) * 2.0 ** -24 * mag, "dispatch_backward", dtype)
        dy, dw = moe.combine_backward(dout, rows, back, wt, shape)
        rdy, rdw, mag = ref_combine_backward(f64(dout), f64(rows), slot_row, w.astype(np.float64))
        same(dy[:R], rdy[:R], np.abs(rdy[:R]) * 2.0 ** -24, "drows", dtype)
        same(dw, rdw, (H / 64 + 16) * 2.0 ** -24 * mag, "dtopk_w", None)


def test_long_ranges_of_many_experts():
    # past 2^18 slots the maps come from ranges of 1024: 2000 experts, a last range that
    # is ragged, ids elsewhere, a token that names an expert twice
    T, topk, E, offset, H = 52501, 5, 2000, 48, 3
    rng = np.random.default_rng(15)
    ids = rng.integers(0, E + 96, size=(T, topk)).astype(np.int32)
    ids[:, 4] = np.where(rng.random(T) < 0.2, ids[:, 0], ids[:, 4])
    flat = ids.reshape(-1).astype(np.int64) - offset
    here = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(here, flat, E), kind="stable")[:here.sum()]
    slot_row = np.full(T * topk, -1, np.int64)
    slot_row[order] = np.arange(len(order))
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[here], minlength=E))])
    shape = moe.DispatchShape(T=T, E=E, topk=topk, H=H, expert_offset=offset)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    rows, o, rs, sr = moe.dispatch(x, torch.from_numpy(ids).cuda(), shape)
    R = len(order)
    assert np.array_equal(o.cpu().numpy(), off) and np.array_equal(sr.cpu().numpy().reshape(-1), slot_row)
    assert np.array_equal(rs[:R].cpu().numpy(), order)
    assert torch.equal(rows[:R], x[torch.from_numpy(order // topk).cuda()])


# ------------------------------------------------------------------ tiles of 32 and 64 rows


# M, N, K, fmt, group, dtype, zeros: many weight groups, a wave all of K or a fourth
@pytest.mark.parametrize("case", [
    (20, 129279, 1024, "mxfp4", 32, "bf16", False),
    (29, 129277, 512, "int4", 64, "fp16", True),
    (50, 129279, 1024, "mxfp4", 32, "fp16", False),
    (61, 129270, 256, "int4", 64, "bf16", True),
    (50, 70001, 4096, "int4", 128, "bf16", True),
    (100, 100003, 256, "int4", 32, "fp16", True),
], ids=lambda c: "-".join(map(str, c)))
def test_w4_linear_of_many_rows_and_weight_groups(case):
    M, N, K, fmt, group, dtype, zeros = case
    say(f"[ops] linear {case}")
    rng = np.random.default_rng(N + K)
    g = torch.Generator(device="cuda").manual_seed(K)
    Np = (N + 15) // 16 * 16
    w = torch.randint(0, 256, (Np, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "mxfp4":
        sc = torch.randint(118, 128, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    else:
        sc = (0.02 * torch.rand(N, K // group, generator=g, device="cuda")).to(TORCH[dtype])
    z = torch.randint(0, 16, (N, K // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    x = torch.from_numpy(rng.standard_normal((M, K))).to(TORCH[dtype]).cuda()
    shape = moe.W4Shape(M=M, N=N, K=K, format=fmt, group=group, dtype=dtype, out_dtype="fp32")
    buf = torch.full((M + 2, N + 3), 777.0, device="cuda")
    moe.w4_linear(x, w, sc, shape, zeros=z, out=buf[1:M + 1, 1:N + 1])
    torch.cuda.synchronize()
    got = f64(buf)
    buf[1:M + 1, 1:N + 1] = 777.0
    assert bool((buf == 777.0).all())
    # whole 16-row groups of weights: the first, some between, the last with its ragged end
    groups = np.unique(np.concatenate([[0, Np // 16 - 2, Np // 16 - 1], rng.integers(0, Np // 16, 60)]))
    for i in groups:
        n1 = min(N, 16 * i + 16)
        codes = w[16 * i:16 * i + 16].reshape(K // 128, 16, 64).transpose(0, 1).reshape(16, K // 2).cpu().numpy()
        codes = np.stack([codes & 15, codes >> 4], -1).reshape(16, K)[:n1 - 16 * i].astype(np.int64)
        s = sc[16 * i:n1]
        W, mag = ref_weights(codes, s.cpu().numpy() if fmt == "mxfp4" else f64(s),
                             None if z is None else z[16 * i:n1].cpu().numpy(), fmt, group)
        ref, size = f64(x) @ W.T, np.abs(f64(x)) @ mag.T
        err = np.abs(got[1:M + 1, 16 * i + 1:n1 + 1] - ref)
        assert (err <= round_tol(ref, "fp32", sum_tol(K) * size)).all(), (i, err.max())


# rows of each expert, rows behind, N, K, fmt, group, dtype, zeros: tiles of 64 rows
# (more than 128 rows an expert), two weight groups a wave; K split over the waves, or
# (the last two) not
@pytest.mark.parametrize("case", [
    ([200, 0, 1, 63, 64, 65, 129, 40], 700, 1040, 640, "mxfp4", 32, "bf16", False),
    ([150, 33, 17, 0, 300, 16, 5, 130], 500, 1030, 384, "int4", 64, "fp16", True),
    ([130, 64, 0, 7] * 16, 5100, 520, 128, "mxfp4", 32, "bf16", False),
    ([1, 200, 33, 31] * 16, 4500, 515, 256, "int4", 64, "bf16", True),
], ids=lambda c: "-".join(map(str, [len(c[0]), *c[1:]])))
def test_w4_grouped_linear_of_many_rows_and_weight_groups(case):
    counts, behind, N, K, fmt, group, dtype, zeros = case
    say(f"[ops] grouped {case}")
    E, R = len(counts), sum(counts)
    M = R + behind
    assert M // E > 128
    rng = np.random.default_rng(N + K)
    m, (W, mag) = _matrices(rng, E, N, K, fmt, group, dtype, zeros)
    off = np.concatenate([[0], np.cumsum(counts)])
    x = torch.from_numpy(rng.standard_normal((M, K))).to(TORCH[dtype]).cuda()
    x[R:] = float("nan")
    out = torch.full((M, N), 777.0, device="cuda")
    _grouped(m, x, off, moe.W4Shape(M=M, N=N, K=K, E=E, format=fmt, group=group, dtype=dtype, out_dtype="fp32"), out=out)
    torch.cuda.synchronize()
    assert bool((out[R:] == 777.0).all())
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        ref, size = f64(x[lo:hi]) @ W[e].T, np.abs(f64(x[lo:hi])) @ mag[e].T
        _close(out[lo:hi], ref, round_tol(ref, "fp32", sum_tol(K) * size), f"expert {e}")
