"""Host-side checks of the operators' arguments (no GPU needed)."""
import pytest
import torch

import mxfp4_weight_expert_amd as moe


def test_tensors_that_require_gradients_are_refused():
    # the calls record nothing: a gradient would be lost without a word
    s = moe.DispatchShape(T=2, E=4, topk=2, H=8)
    x, rows = (torch.zeros(n, 8, dtype=torch.bfloat16) for n in (2, 4))
    maps, w = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    p = moe.W4Shape(M=2, N=16, K=128)
    xp, c = torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(16, 64, dtype=torch.uint8)
    sc = torch.zeros(16, 4, dtype=torch.uint8)
    calls = {"x": [lambda t: moe.dispatch(t(x), maps, s), lambda t: moe.w4_linear(t(xp), c, sc, p),
                   lambda t: moe.w4_linear(t(torch.zeros(2, 136, dtype=torch.bfloat16))[:, :128], c, sc, p)],
             "rows": [lambda t: moe.combine(t(rows), maps, w, s), lambda t: moe.combine_backward(x, t(rows), maps, w, s)],
             "topk_w": [lambda t: moe.combine(rows, maps, t(w), s)],
             "dout": [lambda t: moe.combine_backward(t(x), rows, maps, w, s)],
             "drows": [lambda t: moe.dispatch_backward(t(rows), maps, s)],
             "bias": [lambda t: moe.w4_linear(xp, c, sc, p, bias=t(torch.zeros(16, dtype=torch.bfloat16)))]}
    for name, fs in calls.items():
        for f in fs:
            with pytest.raises(ValueError, match=f"{name} requires a gradient"):
                f(lambda t: t.clone().requires_grad_())
            with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
                f(lambda t: t.clone().requires_grad_())  # goes on to the next check
