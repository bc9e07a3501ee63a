"""The 16-bit products and adapters as a program meets them: a routed layer that trains,
adapters beside frozen 4-bit projections, streams, captured graphs, memory that several
tensors share."""
import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe

from linear_util import close, normal, ref_forward
from ops_util import f64, pack_rows, ref_weights, round_tol, sum_tol

pytestmark = pytest.mark.gpu


class Routed(torch.autograd.Function):
    """Tokens by expert, gated product, down projection, back to tokens."""

    @staticmethod
    def forward(ctx, x, ids, topk_w, w13, w2, act):
        T, H = x.shape
        E, two_i, _ = w13.shape
        route = moe.DispatchShape(T=T, E=E, topk=ids.shape[1], H=H, dtype="fp16")
        up = moe.GatedShape(M=T * ids.shape[1], I=two_i // 2, H=H, E=E, dtype="fp16", activation=act)
        down = moe.LinearShape(M=up.M, N=H, K=up.I, E=E, dtype="fp16")
        rows, off, _, back = moe.dispatch(x, ids, route)
        gu = torch.empty(up.M, two_i, dtype=x.dtype, device=x.device)
        h = moe.gated_linear(rows, off, w13, up, gu=gu)
        y = moe.grouped_linear(h, off, w2, down)
        ctx.save_for_backward(rows, off, back, topk_w, gu, h, y, w13, w2)
        ctx.shapes = route, up, down
        return moe.combine(y, back, topk_w, route)

    @staticmethod
    def backward(ctx, dout):
        rows, off, back, topk_w, gu, h, y, w13, w2 = ctx.saved_tensors
        route, up, down = ctx.shapes
        dy, dw = moe.combine_backward(dout.contiguous(), y, back, topk_w, route)
        dh, dw2 = moe.grouped_linear_backward(dy, h, off, w2, down)
        drows, dw13 = moe.gated_linear_backward(dh, rows, off, gu, w13, up)
        return moe.dispatch_backward(drows, back, route), None, dw, dw13, dw2, None


def _reference(x, ids, topk_w, w13, w2, act):
    """The layer in 64 bits, token by token and column by column."""
    I = w13.shape[1] // 2
    out = []
    for t in range(x.shape[0]):
        row = torch.zeros_like(x[t])
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            if 0 <= e < w13.shape[0]:
                g, u = w13[e, :I] @ x[t], w13[e, I:] @ x[t]
                a = g * torch.sigmoid(g) * u if act == "swiglu" else (
                    4 * torch.tanh(g / 4) * torch.sigmoid(g) * 25 * torch.tanh(u / 25))
                row = row + topk_w[t, k] * (w2[e] @ a)
        out.append(row)
    return torch.stack(out)


@pytest.mark.parametrize("act", ["swiglu", "situ"])
def test_a_routed_layer_that_trains(act):
    rng = np.random.default_rng(21)
    T, H, I, E, k = 50, 64, 40, 5, 2
    ids = torch.from_numpy(rng.integers(-1, E, size=(T, k)).astype(np.int32)).cuda()
    ids[ids == 3] = 2  # an expert without rows
    leaves = [normal(rng, 1, "fp16", T, H), torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda(),
              normal(rng, H ** -0.5, "fp16", E, 2 * I, H), normal(rng, I ** -0.5, "fp16", E, H, I)]
    leaves = [t.requires_grad_() for t in leaves]
    dout = normal(rng, 1, "fp16", T, H)
    out = Routed.apply(leaves[0], ids, *leaves[1:], act)
    out.backward(dout)
    exact = [t.detach().double().cpu().requires_grad_() for t in leaves]
    ref = _reference(exact[0], ids.cpu(), *exact[1:], act)
    ref.backward(dout.double().cpu())
    # Rounded to half steps of 2^-11 on the way: forward h, y and the result (and gu, for
    # the backward pass), backward dy, dh, dgu, drows and the result: at most eight, each
    # carried on by products whose spread is that of their terms. Eight roundings add up
    # to at most 8 * 2^-11 of the norm, with as much again for what act's derivative does
    # to gu's (its slope changes by at most about as much as its argument).
    for got, want, what in ((out, ref, "out"), *((l.grad, e.grad, n) for l, e, n in zip(leaves, exact, ("x", "topk_w", "w13", "w2")))):
        err = np.linalg.norm(f64(got) - want.detach().numpy()) / np.linalg.norm(want.detach().numpy())
        assert err <= 16 * 2.0 ** -11, (what, err)
    assert bool((leaves[2].grad[3] == 0).all()) and bool((leaves[3].grad[3] == 0).all())


def test_adapters_beside_a_4_bit_projection():
    # a decode batch: the frozen projection, then each row's adapter in place
    rng = np.random.default_rng(22)
    M, N, K, R, A = 24, 80, 256, 16, 6
    codes = rng.integers(0, 16, size=(1, N, K)).astype(np.int64)
    scales = rng.integers(120, 126, size=(1, N, K // 32)).astype(np.uint8)
    w = moe.prepack(torch.from_numpy(pack_rows(codes)).cuda())
    W, mag = ref_weights(codes, scales, None, "mxfp4", 32)
    x = normal(rng, 1, "bf16", M, K)
    ids = rng.integers(-1, A, size=M)
    a, b = normal(rng, K ** -0.5, "bf16", A, R, K), normal(rng, R ** -0.5, "bf16", A, N, R)
    scale = torch.from_numpy(rng.uniform(0.5, 2, A).astype(np.float32)).cuda()
    out = moe.w4_linear(x, w, torch.from_numpy(scales).cuda(), moe.W4Shape(M=M, N=N, K=K, out_dtype="fp32"))
    s = moe.AdapterShape(M=M, N=N, K=K, R=R, A=A, out_dtype="fp32")
    moe.adapter_linear(x, *moe.adapter_maps(torch.from_numpy(ids.astype(np.int32)).cuda(), s), a, b, scale, s, base=out, out=out)
    ref, tol = f64(x) @ W[0].T, sum_tol(K) * (np.abs(f64(x)) @ mag[0].T)
    tol = tol + 2.0 ** -23 * np.abs(ref)
    for m in np.nonzero(ids >= 0)[0]:
        t = f64(a[ids[m]]) @ f64(x[m])
        et = sum_tol(K) * (np.abs(f64(a[ids[m]])) @ np.abs(f64(x[m]))) + 2.0 ** -16 * np.abs(t)
        f, B = f64(scale)[ids[m]], f64(b[ids[m]])
        ref[m] += f * (B @ t)
        tol[m] += f * (np.abs(B) @ et + (sum_tol(3 * R) + 2.0 ** -22) * (np.abs(B) @ np.abs(t)))
    close(out, ref, round_tol(ref, "fp32", tol), "out")


def _work(rng):
    """Calls of every operator on tensors of their own: (call, its outputs)."""
    M, E, I, H = 70, 4, 40, 72
    off = torch.tensor([0, 20, 20, 55, 66], dtype=torch.int32, device="cuda")
    x, w13, w2 = normal(rng, 1, "bf16", M, H), normal(rng, .1, "bf16", E, 2 * I, H), normal(rng, .1, "bf16", E, H, I)
    up, down = moe.GatedShape(M=M, I=I, H=H, E=E), moe.LinearShape(M=M, N=H, K=I, E=E, out_dtype="fp32")
    lora = moe.AdapterShape(M=M, N=H, K=H, R=8, A=3)
    z = lambda *n, dt=torch.bfloat16: torch.zeros(*n, dtype=dt, device="cuda")  # noqa: E731
    o = dict(h=z(M, I), gu=z(M, 2 * I), y=z(M, H, dt=torch.float32), dx=z(M, H), dw=z(E, 2 * I, H), dgu=z(M, 2 * I), dh=z(M, I),
             dw2=z(E, H, I, dt=torch.float32), ad=z(M, H), off=z(4, dt=torch.int32), rs=z(M, dt=torch.int32),
             sr=z(M, dt=torch.int32))
    a, b = normal(rng, .1, "bf16", 3, 8, H), normal(rng, .3, "bf16", 3, H, 8)
    ids = torch.from_numpy(rng.integers(-1, 3, size=M).astype(np.int32)).cuda()
    ws = torch.empty(moe.adapter_query(lora), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        moe.gated_linear(x, off, w13, up, out=o["h"], gu=o["gu"], stream=stream)
        moe.grouped_linear(o["h"], off, w2, down, out=o["y"], stream=stream)
        moe.grouped_linear_backward(x, o["h"], off, w2, down, dx=o["dh"], dw=o["dw2"], stream=stream)
        moe.gated_linear_backward(o["dh"], x, off, o["gu"], w13, up, dx=o["dx"], dw=o["dw"], dgu=o["dgu"], stream=stream)
        maps = moe.adapter_maps(ids, lora, offsets=o["off"], row_slot=o["rs"], slot_row=o["sr"], workspace=ws, stream=stream)
        moe.adapter_linear(x, *maps, a, b, None, lora, base=x, out=o["ad"], workspace=ws, stream=stream)
    return call, o, x


def test_on_another_stream():
    rng = np.random.default_rng(23)
    call, outs, _ = _work(rng)
    call()
    want = {n: t.clone() for n, t in outs.items()}
    for t in outs.values():
        t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(t, want[n]) for n, t in outs.items())
    with torch.cuda.stream(side):
        for t in outs.values():
            t.zero_()
        call()
    side.synchronize()
    assert all(torch.equal(t, want[n]) for n, t in outs.items())


def test_captured_graphs():
    # two graphs of the same calls on tensors of their own, replayed in turn with eager
    # work and new inputs between the replays
    rng = np.random.default_rng(24)
    works = [_work(rng) for _ in range(2)]
    graphs = []
    for call, _, _ in works:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for turn in range(4):
        for g, (call, outs, x) in zip(graphs, works):
            x.copy_(normal(rng, 1 + turn, "bf16", *x.shape))
            for t in outs.values():
                t.fill_(turn)
            g.replay()
            torch.cuda.synchronize()
            got = {n: t.clone() for n, t in outs.items()}
            for t in outs.values():
                t.fill_(turn)
            call()
            torch.cuda.synchronize()
            assert all(torch.equal(t, got[n]) for n, t in outs.items()), turn


def test_outputs_count_as_changed():
    rng = np.random.default_rng(25)
    call, outs, _ = _work(rng)
    before = {n: t._version for n, t in outs.items()}
    call()
    assert all(t._version > before[n] for n, t in outs.items())


def test_workspace_too_small():
    s = moe.AdapterShape(M=64, N=8, K=4096, R=128, A=2)
    z = lambda *n, dt=torch.bfloat16: torch.zeros(*n, dtype=dt, device="cuda")  # noqa: E731
    maps = moe.adapter_maps(z(64, dt=torch.int32), s)
    with pytest.raises(moe.MoeError) as e:
        moe.adapter_linear(z(64, 4096), *maps, z(2, 128, 4096), z(2, 8, 128), None, s, workspace=z(256, dt=torch.uint8))
    assert e.value.code == 3


def test_no_rows():
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    e = lambda *n: torch.empty(*n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    s, g = moe.LinearShape(M=0, N=16, K=24, E=2), moe.GatedShape(M=0, I=8, H=24, E=2)
    assert moe.grouped_linear(e(0, 24), off, e(2, 16, 24), s).shape == (0, 16)
    dx, dw = moe.grouped_linear_backward(e(0, 16), e(0, 24), off, e(2, 16, 24), s)
    assert dx.shape == (0, 24) and bool((dw == 0).all())
    assert moe.gated_linear(e(0, 24), off, e(2, 16, 24), g).shape == (0, 8)
    dx, dw = moe.gated_linear_backward(e(0, 8), e(0, 24), off, e(0, 16), e(2, 16, 24), g)
    assert dx.shape == (0, 24) and bool((dw == 0).all())
    a = moe.AdapterShape(M=0, N=16, K=24, R=8, A=2)
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    maps = moe.adapter_maps(ids, a)
    assert maps[0].tolist() == [0, 0, 0]
    assert moe.adapter_linear(e(0, 24), *maps, e(2, 8, 24), e(2, 16, 8), None, a).shape == (0, 16)


def test_rows_past_four_gigabytes():
    # the last rows of x, out and the adapters' arrays lie beyond 32-bit byte offsets
    M, H, N = 300_000, 8192, 64
    x = torch.zeros(M, H, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(26)
    last = normal(rng, 1, "bf16", 40, H)
    x[-40:] = last
    w = normal(rng, H ** -0.5, "bf16", N, H)
    off = torch.tensor([M - 40, M], dtype=torch.int32, device="cuda")
    s = moe.LinearShape(M=M, N=N, K=H)
    want, mag = ref_forward(f64(last), f64(w)[None], None)
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    moe.grouped_linear(x, off, w, s, out=out)
    close(out[-40:], want, round_tol(want, "bf16", sum_tol(H) * mag), "out")
    # dout as wide as x: its last rows' gradient
    d = moe.LinearShape(M=M, N=H, K=N)
    wt = w.t().contiguous()
    dx = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    moe.grouped_linear_backward(x, None, off, wt, d, dx=dx, dw=False)
    close(dx[-40:], want, round_tol(want, "bf16", sum_tol(H) * mag), "dx")
    assert bool((out[:-40] == 0).all()) and bool((dx[:-40] == 0).all())
    a = moe.AdapterShape(M=M, N=N, K=H, R=8, A=1)
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[-40:] = 0
    eye = torch.eye(8, dtype=torch.bfloat16, device="cuda").repeat(8, 1)[None].contiguous()
    got = moe.adapter_linear(x, *moe.adapter_maps(ids, a), w[None, :8].contiguous(), eye, None, a)
    ref = np.tile(want[:, :8], 8)
    close(got[-40:], ref, round_tol(ref, "bf16", sum_tol(H) * np.tile(mag[:, :8], 8) + 2.0 ** -15 * np.abs(ref)), "adapter")
    assert bool((got[:-40] == 0).all())
