"""Arguments of the 16-bit products' binding that a gradient needs (no GPU needed)."""
import pytest
import torch

import mxfp4_weight_expert_amd as moe

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
