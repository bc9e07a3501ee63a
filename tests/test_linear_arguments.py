"""Arguments of the 16-bit products' binding that a gradient needs (no GPU needed)."""
import ctypes

import pytest
import torch

import mxfp4_weight_expert_amd as moe
from mxfp4_weight_expert_amd import linear

BF = torch.bfloat16


@pytest.mark.parametrize("E", [1, 2])
def test_an_operand_that_a_gradient_reads_is_asked_for(E):
    z = lambda *n: torch.zeros(*n, dtype=BF)  # noqa: E731
    off = torch.zeros(E + 1, dtype=torch.int32)
    x, y, w, w13, gu = z(6, 16), z(6, 8), z(E, 8, 16), z(E, 16, 16), z(6, 16)
    s, g = moe.LinearShape(M=6, N=8, K=16, E=E), moe.GatedShape(M=6, I=8, H=16, E=E)
    for call, what in (
            (lambda **k: moe.grouped_linear_backward(y, None, off, w, s, **k), "x is needed for dw"),
            (lambda **k: moe.grouped_linear_backward(y, x, off, None, s, **k), "w is needed for dx"),
            (lambda **k: moe.gated_linear_backward(y, None, off, gu, w13, g, **k), "x is needed for dw"),
            (lambda **k: moe.gated_linear_backward(y, x, off, gu, None, g, **k), "w13 is needed for dx")):
        with pytest.raises(ValueError, match=what):
            call()
        # not wanted: nothing but the GPU is missing
        with pytest.raises(ValueError, match="on the GPU"):
            call(**{what[-2:]: False})


INVALID, HIP = 1, 4  # HIP: past every check, and no GPU to launch on
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="fabricated device addresses: run only where no GPU is visible")


def _p(v):
    return ctypes.c_void_p(v << 36) if v else None


@no_gpu
def test_terms_of_the_pre_activations_gradient():
    M, I = 64, 48
    shape = lambda n: moe.GatedShape(M=M, I=I, H=128, E=4, dgu_terms=n)  # noqa: E731
    forward = lambda n: linear._entry("gated")(_p(1), _p(2), _p(3), shape(n)._c, _p(4), _p(5), None)  # noqa: E731
    back = lambda n, dx=7: linear._entry("gated_backward")(_p(1), _p(2), _p(3), _p(4), _p(5), shape(n)._c, _p(6),  # noqa: E731
                                                           ctypes.c_void_p(dx if dx > 64 else dx << 36), _p(8), None)
    for n in (0, 1, 2):  # 0 stands for 1
        assert forward(n) == HIP and back(n) == HIP
    for n in (-1, 3):
        assert forward(n) == INVALID and back(n) == INVALID
    behind = (6 << 36) + M * 2 * I * 2  # behind the first array
    assert back(1, behind) == HIP and back(2, behind) == INVALID and back(2, behind + M * 2 * I * 2) == HIP


def test_array_of_terms_is_checked():
    z = lambda *n: torch.zeros(*n, dtype=BF)  # noqa: E731
    x, y, w13, gu = z(6, 16), z(6, 8), z(16, 16), z(6, 16)
    run = lambda n, dgu: moe.gated_linear_backward(y, x, None, gu, w13, moe.GatedShape(M=6, I=8, H=16, dgu_terms=n), dgu=dgu)  # noqa: E731
    for n, wrong in ((1, z(2, 6, 16)), (2, z(6, 16)), (2, z(6, 2, 16))):
        with pytest.raises(ValueError, match="dgu must"):
            run(n, wrong)
    for n, right in ((1, z(6, 16)), (2, z(2, 6, 16)), (2, None)):
        with pytest.raises(ValueError, match="on the GPU"):
            run(n, right)
    with pytest.raises(ValueError, match="dgu_terms"):
        moe.GatedShape(M=6, I=8, H=16, dgu_terms=1 << 32).to_c()
