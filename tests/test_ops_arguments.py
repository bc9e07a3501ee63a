"""Host-side checks of the operators' arguments (no GPU needed)."""
import ctypes

import pytest
import torch

import mxfp4_weight_expert_amd as moe
from mxfp4_weight_expert_amd import ops

# Fabricated addresses: never where a kernel could start.
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="fabricated device addresses: run only where no GPU is visible")
GB = 1 << 30
HIP = 4  # MOE_ERR_HIP: past every check, and no GPU to launch on


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


def _w4(x, out, M=5, N=48, K=128, ldx=0, ldo=0, out_dtype="bf16"):
    c = moe.W4Shape(M=M, N=N, K=K, out_dtype=out_dtype).to_c(ldx, ldo)
    p = [ctypes.c_void_p(v) if v else None for v in (x, 8 * GB, 9 * GB, 0, 0)]
    return ops._entry("w4_linear")(*p, ctypes.byref(c), ctypes.c_void_p(out), None)


@no_gpu
def test_rows_of_out_between_rows_of_x():
    x, ld = GB, 128 + 48 + 16  # elements of two bytes
    for out in (x + 2 * 128, x + 2 * (128 + 16)):  # right behind a row of x, right before the next
        assert _w4(x, out, ldx=ld, ldo=ld) == HIP
    for out in (x + 2 * 127, x + 2 * (128 + 17), x, x - 2 * 47, x - 2 * 48 + 2):  # one element into a row
        assert _w4(x, out, ldx=ld, ldo=ld) == 1
    assert _w4(x, x - 2 * 48, ldx=ld, ldo=ld) == HIP  # before the first row, and between the others
    assert _w4(x, x - 2 * (ld + 48), ldx=ld, ldo=ld) == HIP
    # 32-bit results: the same bytes from row to row are half the elements
    assert _w4(x, x + 2 * 128, N=24, ldx=ld, ldo=ld // 2, out_dtype="fp32") == HIP
    assert _w4(x, x + 2 * 126, N=24, ldx=ld, ldo=ld // 2, out_dtype="fp32") == 1
    # rows that drift against each other: refused, also where they should miss
    assert _w4(x, x + 2 * 128, ldx=ld, ldo=ld + 8) == 1
    assert _w4(x, x + 2 * (4 * ld + 128), ldx=ld, ldo=ld + 8) == HIP  # behind the last row
    assert _w4(x, x + 2 * 128, M=1, ldx=ld, ldo=48) == HIP  # one row has no next


@no_gpu
def test_workspace_of_dispatch_on_its_own():
    at = {n: (i + 1) * GB for i, n in enumerate(("x", "ids", "rows", "offsets", "row_slot", "slot_row", "ws"))}

    def run(shape, **kw):
        a = {n: ctypes.c_void_p(v) for n, v in {**at, **kw}.items()}
        return ops._entry("dispatch")(a["x"], a["ids"], shape._c, a["rows"], a["offsets"], a["row_slot"],
                                      a["slot_row"], a["ws"], GB, None)

    for T in (64, 4000):  # one launch; maps that use the workspace
        s = moe.DispatchShape(T=T, E=896, topk=16, H=512)
        assert run(s) == HIP
        need = moe.dispatch_query(s)
        for n in ("x", "ids", "rows", "offsets", "row_slot", "slot_row"):
            assert run(s, ws=at[n]) == 1, n
            assert run(s, ws=at[n] - need + 256) == 1, n
            assert run(s, ws=at[n] - need) == HIP, n
    s = moe.DispatchShape(T=0, E=896, topk=16, H=512)
    assert run(s, ws=at["offsets"]) == 1


def test_sizes_past_32_bits_are_refused():
    # not cut off to the C structs' 32 bits, where they would name another shape
    big = 1 << 32
    for kw in (dict(T=big + 4), dict(E=big + 4), dict(topk=big + 2), dict(H=big + 16), dict(expert_offset=big),
               dict(expert_offset=-big), dict(T=1 << 31)):
        s = moe.DispatchShape(**{**dict(T=4, E=4, topk=2, H=16), **kw})
        with pytest.raises(ValueError, match=next(iter(kw))):
            s.to_c()
        with pytest.raises(ValueError, match=next(iter(kw))):
            moe.dispatch_query(s)
    for kw in (dict(M=big + 4), dict(N=big + 32), dict(K=big + 128), dict(E=big + 1), dict(group=big + 32)):
        s = moe.W4Shape(**{**dict(M=4, N=32, K=128), **kw})
        with pytest.raises(ValueError, match=next(iter(kw))):
            s.to_c()
