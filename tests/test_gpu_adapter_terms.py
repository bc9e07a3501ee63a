"""What the adapters keep of t = x A^T between their two products, by sums that are exact:
a term less, or one bit of the last term, changes the result."""
import numpy as np
import pytest
import torch

import mxfp4_weight_expert_amd as moe

from gpu_util import say
from ops_util import TORCH, f64

# bits of t behind the point that the terms hold beside the seven before it: two values of
# bf16 hold 16 bits, three hold 24; two of fp16 hold 22, of which the smallest type step in a
# row divided to below 2 leaves 21 here
KEPT = {("bf16", "bf16"): 8, ("bf16", "fp32"): 16, ("fp16", "fp16"): 13, ("fp16", "fp32"): 13}
AT = (3, 40, 77)  # places of K of the three parts of t, in different steps of the MFMA


def _parts(dtype, out):
    """Scales of the parts, whole numbers of up to seven or eight bits each, and their ranges."""
    kept = KEPT[dtype, out]
    return [(1.0, 120), (2.0 ** -8, 255)] + ([(2.0 ** -kept, 2 ** (kept - 8) - 1)] if kept > 8 else [])


def _case(M, N, R, A, dtype, out, seed):
    """x, a, b in 64 bits, all exact in dtype, and t [M, A, R], exact in 32 bits."""
    rng = np.random.default_rng(seed)
    parts = _parts(dtype, out)
    x = np.zeros((M, 80))
    a = np.zeros((A, R, 80))
    for at, (scale, most) in zip(AT, parts):
        x[:, at] = rng.integers(-most, most + 1, size=M)
        # the first part is common to all of a row's t; the others have signs, some are left out
        a[:, :, at] = scale * (1 if at == AT[0] else rng.integers(-1, 2, size=(A, R)))
    # differences of two t, where the common part cancels, and single ones
    b = np.zeros((A, N, R))
    for i in range(A):
        for n in range(N):
            p, q = rng.choice(R, size=2, replace=False)
            b[i, n, p] = 1
            if n % 3:
                b[i, n, q] = -1
    return x, a, b, np.einsum("mk,ark->mar", x, a)


def _terms(t, dtype, count):
    """Sum of `count` values of dtype that t is held as."""
    kept, left = np.zeros_like(t), t
    for _ in range(count):
        v = torch.from_numpy(left).float().to(TORCH[dtype]).double().numpy()
        kept, left = kept + v, left - v
    return kept


@pytest.mark.parametrize("dtype,out", KEPT)
def test_the_sums_tell_a_term_less(dtype, out):
    # on the CPU: with one term less many of the expected results would be others
    x, a, b, t = _case(64, 30, 16, 2, dtype, out, 1)
    count = 3 if (dtype, out) == ("bf16", "fp32") else 2
    scale = 2.0 ** -6  # as the kernel divides a row of fp16: to below 2
    assert np.array_equal(_terms(t * scale, dtype, count), t * scale)
    less = _terms(t * scale, dtype, count - 1) / scale
    want, got = (np.einsum("mr,nr->mn", v[:, 0], b[0]) for v in (t, less))
    assert (want != got).mean() > 0.2


# one tile and several, of 16 rows and of 32, few and many parts of K's sum
@pytest.mark.gpu
@pytest.mark.parametrize("M,A,N,R", [(1, 1, 7, 8), (40, 3, 50, 16), (300, 4, 130, 24), (3300, 2, 300, 32), (4100, 3, 70, 72),
                                     (1601, 1, 257, 128)])
@pytest.mark.parametrize("dtype,out", KEPT)
def test_nothing_is_lost_between_the_products(M, A, N, R, dtype, out):
    say(f"[adapter terms] {M} {A} {N} {R} {dtype} {out}")
    x, a, b, t = _case(M, N, R, A, dtype, out, M + R)
    ids = np.random.default_rng(M).integers(0, A, size=M)
    to = lambda v: torch.from_numpy(v).to(TORCH[dtype]).cuda()  # noqa: E731
    X, a_, b_ = to(x), to(a), to(b)
    assert np.array_equal(f64(X), x) and np.array_equal(f64(a_), a) and np.array_equal(f64(b_), b)
    scale = 2.0 ** np.random.default_rng(R).integers(-3, 4, size=A)
    s = moe.AdapterShape(M=M, N=N, K=80, R=R, A=A, dtype=dtype, out_dtype=out)
    maps = moe.adapter_maps(torch.from_numpy(ids.astype(np.int32)).cuda(), s)
    got = moe.adapter_linear(X, *maps, a_, b_, torch.from_numpy(scale.astype(np.float32)).cuda(), s)
    want = np.stack([scale[i] * (b[i] @ t[m, i]) for m, i in enumerate(ids)])
    assert np.array_equal(want.astype(np.float32), want)  # exact in 32 bits, so rounded once
    rounded = torch.from_numpy(want.astype(np.float32)).to(TORCH[out])
    assert torch.equal(got.cpu(), rounded)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["fp16", "fp32"])
def test_small_values_beside_large_ones_in_halves(out):
    # fp16: a row is divided by a power of two before it is rounded, so what is lost goes by
    # the value (2^-22 of it: half a step twice) or by the row's largest, which lies between
    # 1 and 2 then (2^-25: half the type's smallest number)
    rng = np.random.default_rng(7)
    M, R = 48, 16
    size = 2.0 ** rng.integers(-30, 1, size=R)
    x = np.zeros((M, 16))
    x[:, 0] = rng.integers(1024, 2048, size=M)
    x[:, 1] = rng.integers(0, 2048, size=M)
    a = np.zeros((1, R, 16))
    # t up to 2^14 and down to 2^-20, of 22 bits
    a[0, :, 0], a[0, :, 1] = size * 8, size * 8 * 2.0 ** -11
    a = np.where(np.abs(a) < 2.0 ** -24, 0, a)  # what the type holds
    b = np.eye(R)[None]
    to = lambda v: torch.from_numpy(v).half().cuda()  # noqa: E731
    A_ = to(a)
    t = x @ f64(A_)[0].T
    s = moe.AdapterShape(M=M, N=R, K=16, R=R, A=1, dtype="fp16", out_dtype=out)
    maps = moe.adapter_maps(torch.zeros(M, dtype=torch.int32, device="cuda"), s)
    got = f64(moe.adapter_linear(to(x), *maps, A_, to(b), None, s))
    most = np.abs(t).max(1, keepdims=True)
    bound = 2.0 ** -23 * np.abs(t) + 2.0 ** -22 * np.abs(t) + 2.0 ** -25 * most  # t's own sum first
    if out == "fp16":
        bound = bound + (np.abs(t) + bound) * 2.0 ** -11 + 2.0 ** -25
    assert (np.abs(got - t) <= bound).all(), float((np.abs(got - t) / bound).max())
