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
