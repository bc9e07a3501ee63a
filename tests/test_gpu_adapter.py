"""Low-rank adapters on the GPU, against their definition in 64 bits."""
import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe

from gpu_util import say
from linear_util import close, normal
from ops_util import TORCH, f64, ref_maps, round_tol, sum_tol

pytestmark = pytest.mark.gpu

MARK = -3.0


def _ref(x, ids, a, b, scale, base):
    """(result, bound on its 32-bit value)."""
    out, tol = base.copy(), 2.0 ** -23 * np.abs(base)
    for i in range(a.shape[0]):
        m = np.nonzero(ids == i)[0]
        if not len(m):
            continue
        t, tm = x[m] @ a[i].T, np.abs(x[m]) @ np.abs(a[i]).T
        # t's own sum, its two halves (2^-16 of it in bf16; of the row's largest 2^-22
        # in fp16, which is less), the second sum, the scale and the addition
        et = sum_tol(x.shape[1]) * tm + 2.0 ** -16 * np.abs(t) + 2.0 ** -22 * np.abs(t).max(1, keepdims=True)
        up = np.abs(t) @ np.abs(b[i]).T
        out[m] += scale[i] * (t @ b[i].T)
        tol[m] += np.abs(scale[i]) * (et @ np.abs(b[i]).T + (sum_tol(2 * b.shape[2]) + 2.0 ** -22) * up)
    return out, tol


def _case(rng, M, N, K, R, A, dtype="bf16", out=None, none=0.2):
    out = out or dtype
    ids = rng.integers(0, A, size=M)
    ids[rng.random(M) < none] = -1
    t = dict(x=normal(rng, 1, dtype, M, K), a=normal(rng, K ** -0.5, dtype, A, R, K), b=normal(rng, R ** -0.5, dtype, A, N, R),
             scale=torch.from_numpy(rng.uniform(-2, 2, A).astype(np.float32)).cuda(), base=normal(rng, 1, out, M, N))
    return ids, t, moe.AdapterShape(M=M, N=N, K=K, R=R, A=A, dtype=dtype, out_dtype=out)


def _maps(ids, shape):
    return moe.adapter_maps(torch.as_tensor(ids, dtype=torch.int32).cuda(), shape)


def _run(ids, t, shape, **kw):
    return moe.adapter_linear(t["x"], *_maps(ids, shape), t["a"], t["b"], kw.pop("scale", t["scale"]), shape,
                              base=kw.pop("base", t["base"]), **kw)


def _want(ids, t, scale=True, base=True):
    s = f64(t["scale"]) if scale else np.ones(t["a"].shape[0])
    return _ref(f64(t["x"]), ids, f64(t["a"]), f64(t["b"]), s, f64(t["base"]) * (1 if base else 0))


@pytest.mark.parametrize("M,A", [(1, 1), (1, 7), (5, 3), (17, 300), (64, 5), (70, 2048)])
def test_maps(M, A):
    rng = np.random.default_rng(M)
    ids = rng.integers(-2, A + 2, size=M)
    off, row_slot, slot_row = (f64(v).astype(int) for v in _maps(ids, moe.AdapterShape(M=M, N=8, K=8, R=8, A=A)))
    ro, rr, rs = ref_maps(ids[:, None], A, 0)
    assert np.array_equal(off, ro) and np.array_equal(row_slot[:ro[-1]], rr) and np.array_equal(slot_row, rs[:, 0])


def test_maps_of_many_rows():
    rng = np.random.default_rng(1)
    for M in (4096, 4097, 30000):
        ids = rng.integers(-1, 50, size=M)
        off, row_slot, slot_row = (f64(v).astype(int) for v in _maps(ids, moe.AdapterShape(M=M, N=8, K=8, R=8, A=50)))
        ro, rr, rs = ref_maps(ids[:, None], 50, 0)
        assert np.array_equal(off, ro) and np.array_equal(row_slot[:ro[-1]], rr) and np.array_equal(slot_row, rs[:, 0])


# few rows of many adapters; tiles with full, partial and following ones; more adapters
# than a block has threads
ROWS = [(1, 1), (3, 40), (50, 4), (90, 300), (33, 1), (70, 2), (400, 3)]


@pytest.mark.parametrize("M,A", ROWS)
@pytest.mark.parametrize("N,K,R", [(1, 8, 8), (16, 40, 16), (63, 264, 24), (200, 1032, 32), (257, 136, 64), (130, 2056, 72), (320, 96, 128)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")])
def test_adapters(M, A, N, K, R, dtype, out):
    say(f"[adapter] {M} {A} {N} {K} {R} {dtype} {out}")
    rng = np.random.default_rng(M * N)
    ids, t, shape = _case(rng, M, N, K, R, A, dtype, out)
    ref, tol = _want(ids, t)
    got = _run(ids, t, shape)
    close(got, ref, round_tol(ref, out, tol), "out")
    assert torch.equal(got[ids < 0], t["base"][ids < 0])
    # in place
    own = t["base"].clone()
    assert _run(ids, t, shape, base=own, out=own) is own and torch.equal(own, got)


# tiles of 32 rows, an adapter's last one partial; spans of N of several pieces, a short last one
@pytest.mark.parametrize("M,A,N,K,R", [(4300, 3, 70, 264, 24), (3300, 100, 1030, 72, 32), (1601, 50, 2057, 520, 64),
                                       (1601, 1, 513, 1032, 72), (1025, 7, 1100, 2056, 128), (9001, 9, 776, 40, 128)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16")])
def test_adapters_of_many_rows(M, A, N, K, R, dtype, out):
    say(f"[adapter] {M} {A} {N} {K} {R} {dtype} {out}")
    rng = np.random.default_rng(M + N)
    ids, t, shape = _case(rng, M, N, K, R, A, dtype, out, none=0.1)
    ref, tol = _want(ids, t)
    got = _run(ids, t, shape)
    close(got, ref, round_tol(ref, out, tol), "out")
    assert torch.equal(got[ids < 0], t["base"][ids < 0])
    own = t["base"].clone()
    assert _run(ids, t, shape, base=own, out=own) is own and torch.equal(own, got)


def test_without_base_and_scale():
    rng = np.random.default_rng(3)
    ids, t, shape = _case(rng, 45, 70, 80, 16, 4)
    ref, tol = _want(ids, t, scale=False, base=False)
    out = torch.full((45, 70), MARK, dtype=torch.bfloat16, device="cuda")
    close(_run(ids, t, shape, scale=None, base=None, out=out), ref, round_tol(ref, "bf16", tol), "out")
    assert bool((out[ids < 0] == 0).all())


def test_no_row_has_an_adapter():
    rng = np.random.default_rng(4)
    ids, t, shape = _case(rng, 40, 70, 80, 16, 4, none=2.0)
    assert torch.equal(_run(ids, t, shape), t["base"])


def test_strided_rows():
    rng = np.random.default_rng(5)
    for out_type in ("bf16", "fp32"):
        ids, t, shape = _case(rng, 50, 45, 40, 8, 3, out=out_type)
        want = _run(ids, t, shape)
        x = torch.zeros(50, 56, dtype=torch.bfloat16, device="cuda")[:, 8:48]
        x.copy_(t["x"])
        wide = torch.full((50, 107), MARK, dtype=TORCH[out_type], device="cuda")
        wide[:, 3:48] = t["base"]
        s = dict(t, x=x, base=wide[:, 3:48])
        assert torch.equal(_run(ids, s, shape, out=wide[:, 55:100]), want)
        assert torch.equal(wide[:, 3:48], t["base"])
        own = wide[:, 3:48]
        assert torch.equal(_run(ids, s, shape, base=own, out=own), want)
        rest = torch.cat([wide[:, :3], wide[:, 48:55], wide[:, 100:]], 1)
        assert bool((rest == MARK).all())


def test_halves_past_the_type_s_range():
    # t far past 65504 and far below its smallest number, results in range
    rng = np.random.default_rng(6)
    for size in (2.0 ** 14, 2.0 ** -14):
        ids, t, shape = _case(rng, 40, 50, 256, 16, 3, "fp16", "fp32", none=0.0)
        t["x"], t["a"] = (t["x"] * size).clamp(-6e4, 6e4), t["a"] * min(size, 8.0)
        t["base"].zero_()
        ref, tol = _want(ids, t)
        close(_run(ids, t, shape), ref, round_tol(ref, "fp32", tol), f"out at {size}")


def test_values_that_are_no_numbers_stay_in_their_rows():
    rng = np.random.default_rng(7)
    ids, t, shape = _case(rng, 40, 50, 64, 24, 3, none=0.1)
    ids[:3], ids[10] = 0, 1
    want = _run(ids, t, shape)
    t["x"][10] = float("nan")
    t["a"][2], t["b"][2] = float("inf"), float("nan")
    t["x"][ids < 0] = float("nan")
    got = _run(ids, t, shape)
    same = (ids != 2) & (np.arange(40) != 10)
    assert torch.equal(got[same], want[same]) and bool(got[10].isnan().all()) and bool(got[ids == 2].isnan().all())


def test_bits_do_not_depend_on_other_rows():
    # for one shape a row's result goes by the row and its adapter alone
    rng = np.random.default_rng(8)
    ids, t, shape = _case(rng, 64, 300, 512, 16, 20, none=0.0)
    want = _run(ids, t, shape)
    other = ids.copy()
    other[1::2] = rng.integers(0, 20, size=32)
    got = _run(other, t, shape)
    assert torch.equal(got[::2], want[::2])
