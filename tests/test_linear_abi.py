"""Host-side checks of the 16-bit products' C ABI and binding (no GPU needed): the library
exports what the header declares, structs agree, and bad arguments are refused before
anything is launched."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import mxfp4_weight_expert_amd as moe
from mxfp4_weight_expert_amd import linear

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_linear.h")
GB = 1 << 30
OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = range(5)  # HIP: past every check, and no GPU to launch on

# Fabricated addresses: never where a kernel could start.
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="fabricated device addresses: run only where no GPU is visible")


def test_library_exports_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_linear_\w+)\s*\(", text))
    nm = subprocess.run(["nm", "-D", "--defined-only", moe.lib_path], capture_output=True, text=True)
    assert names == set(re.findall(r"\bT (moe_linear_\w+)", nm.stdout)) and len(names) == 7


@pytest.mark.parametrize("lang", ["c99", "c++"])
def test_structs_match_header(tmp_path, lang):
    pairs = [("moe_linear_shape", linear._LinearShape), ("moe_gated_shape", linear._GatedShape),
             ("moe_adapter_shape", linear._AdapterShape)]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe_linear.h"', "int main(void){"]
    want = []
    for name, cls in pairs:
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f[0]}));')
            want.append(getattr(cls, f[0]).offset)
    src = tmp_path / ("probe.c" if lang == "c99" else "probe.cc")
    src.write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "probe"
    cc = ["gcc", "-std=c99"] if lang == "c99" else ["g++"]
    subprocess.run([*cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == want


A = {n: (i + 1) * 64 * GB for i, n in enumerate(["x", "off", "w", "out", "gu", "dout", "dx", "dw", "dgu", "a", "b", "scale",
                                                 "base", "rs", "sr", "ws", "ids"])}


def _p(v):
    return ctypes.c_void_p(v) if v else None


def _forward(shape, ldx=0, ldo=0, gated=False, **kw):
    a = {**A, **kw}
    c = ctypes.byref(shape.to_c(ldx, ldo))
    if gated:
        return linear._entry("gated")(_p(a["x"]), _p(a["off"]), _p(a["w"]), c, _p(a["out"]), _p(a["gu"]), None)
    return linear._entry("grouped")(_p(a["x"]), _p(a["off"]), _p(a["w"]), c, _p(a["out"]), None)


def _backward(shape, ldx=0, ldo=0, gated=False, **kw):
    a = {**A, **kw}
    c = ctypes.byref(shape.to_c(ldx, ldo))
    if gated:
        return linear._entry("gated_backward")(_p(a["dout"]), _p(a["x"]), _p(a["off"]), _p(a["gu"]), _p(a["w"]), c,
                                               _p(a["dgu"]), _p(a["dx"]), _p(a["dw"]), None)
    return linear._entry("grouped_backward")(_p(a["dout"]), _p(a["x"]), _p(a["off"]), _p(a["w"]), c, _p(a["dx"]),
                                             _p(a["dw"]), None)


def _ls(**kw):
    return moe.LinearShape(**{**dict(M=64, N=48, K=128, E=4), **kw})


def _gs(**kw):
    return moe.GatedShape(**{**dict(M=64, I=48, H=128, E=4), **kw})


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(E=0), INVALID), (dict(N=44), INVALID),
    (dict(K=132), INVALID), (dict(M=(1 << 23) + 1), UNSUPPORTED), (dict(N=(1 << 20) + 8), UNSUPPORTED),
    (dict(K=(1 << 20) + 8), UNSUPPORTED), (dict(E=2049), UNSUPPORTED), (dict(N=1 << 16, K=(1 << 14) + 8), UNSUPPORTED),
    (dict(dtype="fp32"), UNSUPPORTED), (dict(dtype="fp16", out_dtype="bf16"), UNSUPPORTED),
    (dict(M=1 << 23, N=1 << 16, K=8), UNSUPPORTED), (dict(), HIP), (dict(out_dtype="fp32"), HIP), (dict(M=0), OK),
])
def test_shapes(kw, code):
    assert _forward(_ls(**kw)) == code
    if kw != dict(M=0):  # without rows the matrices' gradient is zeros
        assert _backward(_ls(**kw)) == code


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(I=0), INVALID), (dict(I=44), INVALID), (dict(H=20), INVALID), (dict(swiglu_limit=float("nan")), INVALID),
    (dict(activation="situ", act_beta=0.0), INVALID), (dict(activation="situ", act_linear_beta=float("inf")), INVALID),
    (dict(dtype="fp32"), UNSUPPORTED), (dict(I=1 << 15, H=1 << 15), UNSUPPORTED), (dict(act_beta=0.0), HIP),
    (dict(activation="situ"), HIP), (dict(I=1 << 14, H=1 << 15, M=8, E=1), HIP),
])
def test_gated_shapes(kw, code):
    assert _forward(_gs(**kw), gated=True) == code
    assert _backward(_gs(**kw), gated=True) == code


@no_gpu
def test_pointers():
    for call, shape, gated, need in ((_forward, _ls(), False, ("x", "w", "out")), (_forward, _gs(), True, ("x", "w", "out")),
                                     (_backward, _ls(), False, ("dout", "x", "w")),
                                     (_backward, _gs(), True, ("dout", "x", "w", "gu", "dgu"))):
        assert call(shape, gated=gated) == HIP
        for n in need:
            assert call(shape, gated=gated, **{n: 0}) == INVALID, n
            assert call(shape, gated=gated, **{n: A[n] + 8}) == INVALID, n
        assert call(shape, gated=gated, off=0) == INVALID  # several matrices
        assert call(shape, gated=gated, off=A["off"] + 2) == INVALID
    assert _forward(_gs(), gated=True, gu=0) == HIP
    one = _ls(E=1)
    assert _forward(one, off=0) == HIP and _backward(one, off=0) == HIP
    # a gradient that is not wanted needs less
    assert _backward(_ls(), dx=0, w=0) == HIP and _backward(_ls(), dw=0, x=0) == HIP
    assert _backward(_ls(), dx=0, dw=0) == OK


@no_gpu
def test_strides():
    s = _ls()
    assert _forward(s, ldx=136, ldo=56) == HIP
    for ldx, ldo in ((120, 0), (132, 0), (0, 40), (0, 52)):
        assert _forward(s, ldx, ldo) == INVALID and _forward(_gs(), ldx, ldo, gated=True) == INVALID
    assert _forward(s, (1 << 20) + 8, 0) == UNSUPPORTED
    # rows' gradient: as many tiles as the forward product of K columns
    wide = _ls(M=1 << 23, N=8, K=1 << 15)
    far = dict(x=1 << 42, dx=1 << 43)
    assert _forward(wide, **far) == HIP and _backward(wide, **far) == UNSUPPORTED and _backward(wide, dx=0, x=1 << 42) == UNSUPPORTED
    assert _backward(_ls(M=1 << 23, N=8, K=1 << 14), **far) == HIP
    assert _backward(s, ldx=128) == INVALID and _backward(_gs(), ldo=48, gated=True) == INVALID


@no_gpu
def test_overlaps():
    s, x = _ls(), A["x"]
    assert _forward(s, out=x + 64 * 128 * 2) == HIP  # right behind x
    assert _forward(s, out=x + 64 * 128 * 2 - 16) == INVALID and _forward(s, out=A["w"]) == INVALID
    assert _forward(s, out=A["off"]) == INVALID
    assert _forward(s, 192, 192, out=x + 2 * 128) == HIP  # columns of one matrix
    assert _forward(s, 192, 192, out=x + 2 * 120) == INVALID
    g = _gs()
    assert _forward(g, gated=True, gu=A["out"]) == INVALID and _forward(g, gated=True, gu=x) == INVALID
    for n, on in (("dx", "dout"), ("dx", "x"), ("dx", "w"), ("dw", "w"), ("dw", "dx"), ("dw", "off"), ("dx", "off")):
        assert _backward(s, **{n: A[on]}) == INVALID, (n, on)
        assert _backward(g, gated=True, **{n: A[on]}) == INVALID, (n, on)
    assert _backward(g, gated=True, dgu=A["gu"]) == INVALID and _backward(g, gated=True, dgu=A["dout"]) == INVALID
    # arrays that are not read may lie anywhere
    assert _backward(s, dw=0, dx=A["x"]) == HIP and _backward(s, dx=0, dw=A["w"]) == HIP


def _as(**kw):
    return moe.AdapterShape(**{**dict(M=64, N=50, K=128, R=16, A=4), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(R=0), INVALID), (dict(A=0), INVALID),
    (dict(K=20), INVALID), (dict(R=12), INVALID), (dict(R=136), UNSUPPORTED), (dict(A=2049), UNSUPPORTED),
    (dict(M=(1 << 23) + 1), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=(1 << 20) + 8), UNSUPPORTED),
    (dict(dtype="fp32"), UNSUPPORTED), (dict(out_dtype="fp16"), UNSUPPORTED),
])
def test_adapter_query_refuses(kw, code):
    with pytest.raises(moe.MoeError) as e:
        moe.adapter_query(_as(**kw))
    assert e.value.code == code


def test_adapter_query_sizes():
    for kw in (dict(), dict(M=0), dict(M=1), dict(M=50000, A=2048)):
        n = moe.adapter_query(_as(**kw))
        assert n >= 256 and n % 256 == 0 and n >= _as(**kw).M * 16 * 4
    n = ctypes.c_uint64()
    query = linear._entry("adapter_query")
    assert query(None, ctypes.byref(n)) == INVALID and query(_as()._c, None) == INVALID


def _adapter(shape, ld=(0, 0, 0), wsb=GB, **kw):
    a = {**A, **kw}
    return linear._entry("adapter")(*(_p(a[n]) for n in ("x", "off", "rs", "sr", "a", "b", "scale")),
                                    ctypes.byref(shape.to_c(*ld)), _p(a["base"]), _p(a["out"]), _p(a["ws"]), wsb, None)


@no_gpu
def test_adapter_arguments():
    s = _as()
    assert _adapter(s) == HIP and _adapter(s, scale=0) == HIP and _adapter(s, base=0) == HIP
    assert _adapter(s, out=A["base"]) == HIP  # in place
    assert _adapter(_as(M=0), x=0, out=0, ws=0) == OK
    for n in ("x", "off", "rs", "sr", "a", "b", "out"):
        assert _adapter(s, **{n: 0}) == INVALID, n
    for n in ("x", "a", "b"):
        assert _adapter(s, **{n: A[n] + 8}) == INVALID, n
    for n in ("off", "rs", "sr", "scale"):
        assert _adapter(s, **{n: A[n] + 2}) == INVALID, n
    assert _adapter(s, base=A["base"] + 1) == INVALID and _adapter(s, out=A["out"] + 2) == HIP
    assert _adapter(_as(out_dtype="fp32"), out=A["out"] + 2) == INVALID
    assert _adapter(s, ws=0) == WORKSPACE and _adapter(s, ws=A["ws"] + 64) == WORKSPACE and _adapter(s, wsb=64) == WORKSPACE
    for n in ("x", "off", "rs", "sr", "a", "b", "scale"):
        assert _adapter(s, out=A[n]) == INVALID and _adapter(s, ws=A[n]) == INVALID, n
    assert _adapter(s, ws=A["base"]) == INVALID and _adapter(s, ws=A["out"]) == INVALID
    assert _adapter(s, out=A["base"] + 2) == INVALID  # neither in place nor apart
    assert _adapter(s, (0, 100, 104), out=A["base"]) == INVALID and _adapter(s, (0, 100, 100), out=A["base"]) == HIP
    assert _adapter(s, (0, 100, 100), out=A["base"] + 100) == HIP  # columns of one matrix
    for ld in ((120, 0, 0), (132, 0, 0), (0, 49, 0), (0, 0, 49)):
        assert _adapter(s, ld) == INVALID


@no_gpu
def test_adapter_maps_arguments():
    def run(shape, wsb=GB, **kw):
        a = {**A, **kw}
        return linear._entry("adapter_maps")(_p(a["ids"]), shape._c, _p(a["off"]), _p(a["rs"]), _p(a["sr"]), _p(a["ws"]),
                                             wsb, None)
    for M in (64, 9000):
        s = _as(M=M)
        assert run(s) == HIP and run(s, wsb=64) == WORKSPACE and run(s, ws=0) == WORKSPACE
        for n in ("ids", "off", "rs", "sr"):
            assert run(s, **{n: 0}) == INVALID and run(s, **{n: A[n] + 2}) == INVALID and run(s, ws=A[n]) == INVALID, n
        assert run(s, rs=A["sr"]) == INVALID and run(s, off=A["ids"]) == INVALID


def test_sizes_past_32_bits_are_refused():
    big = 1 << 32
    for shape, sizes in ((_ls, "MNKE"), (_gs, "MIHE"), (_as, "MNKRA")):
        for n in sizes:
            with pytest.raises(ValueError, match=n):
                shape(**{n: big + 8}).to_c()


def test_arrays_are_checked():
    bf = torch.bfloat16
    x, w, off = torch.zeros(6, 16, dtype=bf), torch.zeros(2, 8, 16, dtype=bf), torch.zeros(3, dtype=torch.int32)
    s, g = moe.LinearShape(M=6, N=8, K=16, E=2), moe.GatedShape(M=6, I=4, H=16, E=2)
    a = moe.AdapterShape(M=6, N=8, K=16, R=8, A=2)
    down, up, row = torch.zeros(2, 8, 16, dtype=bf), torch.zeros(2, 8, 8, dtype=bf), torch.zeros(6, dtype=torch.int32)
    out, gu = torch.zeros(6, 8, dtype=bf), torch.zeros(6, 8, dtype=bf)
    for call, what in (
            (lambda: moe.grouped_linear(x[:5], off, w, s), "x must"), (lambda: moe.grouped_linear(x, off[:2], w, s), "offsets must"),
            (lambda: moe.grouped_linear(x, off, w[0], s), "w must"), (lambda: moe.grouped_linear(x, off, w.float(), s), "w must"),
            (lambda: moe.grouped_linear(x, None, w, s), "offsets are needed"),
            (lambda: moe.grouped_linear(x, off, w, s, out=out[:, :7]), "out must"),
            (lambda: moe.grouped_linear_backward(out, x.t().contiguous().t(), off, w, s), "x must be contiguous"),
            (lambda: moe.grouped_linear_backward(x, x, off, w, s), "dout must"),
            (lambda: moe.gated_linear(x, off, w, g, gu=gu[:5]), "gu must"), (lambda: moe.gated_linear(x, off, w[:, :7], g), "w13 must"),
            (lambda: moe.gated_linear_backward(out[:, :4], x, off, gu, w, g), "dh must be contiguous"),
            (lambda: moe.adapter_linear(x, off, row, row, up, up, None, a), "a must"),
            (lambda: moe.adapter_linear(x, off, row, row, down, up, torch.ones(3), a), "scale must"),
            (lambda: moe.adapter_linear(x, off, row[:5], row, down, up, None, a), "row_slot must"),
            (lambda: moe.adapter_linear(x, off, row, row, down, up, None, a, base=out.float()), "base must"),
            (lambda: moe.adapter_maps(row.long(), a), "ids must")):
        with pytest.raises(ValueError, match=what):
            call()
    # everything in order: the first call that would need the GPU says so
    for call in (lambda: moe.grouped_linear(x, off, w, s), lambda: moe.gated_linear(x, off, w, g, gu=gu),
                 lambda: moe.adapter_linear(x, off, row, row, down, up, None, a), lambda: moe.adapter_maps(row, a)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_tensors_that_require_gradients_are_refused():
    bf = torch.bfloat16
    s, g, a = moe.LinearShape(M=6, N=8, K=16), moe.GatedShape(M=6, I=8, H=16), moe.AdapterShape(M=6, N=8, K=16, R=8, A=2)
    x, w, w13, gu, y = (torch.zeros(n, dtype=bf) for n in ((6, 16), (8, 16), (16, 16), (6, 16), (6, 8)))
    off, row = torch.zeros(3, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)
    down, up, scale = torch.zeros(2, 8, 16, dtype=bf), torch.zeros(2, 8, 8, dtype=bf), torch.ones(2)
    calls = {"x": [lambda t: moe.grouped_linear(t(x), None, w, s), lambda t: moe.gated_linear(t(x), None, w13, g),
                   lambda t: moe.adapter_linear(t(x), off, row, row, down, up, scale, a)],
             "w": [lambda t: moe.grouped_linear(x, None, t(w), s)], "w13": [lambda t: moe.gated_linear(x, None, t(w13), g)],
             "dout": [lambda t: moe.grouped_linear_backward(t(y), x, None, w, s)],
             "dh": [lambda t: moe.gated_linear_backward(t(y), x, None, gu, w13, g)],
             "gu": [lambda t: moe.gated_linear_backward(y, x, None, t(gu), w13, g)],
             "scale": [lambda t: moe.adapter_linear(x, off, row, row, down, up, t(scale), a)],
             "base": [lambda t: moe.adapter_linear(x, off, row, row, down, up, scale, a, base=t(y))]}
    for name, fs in calls.items():
        for f in fs:
            with pytest.raises(ValueError, match=f"{name} requires a gradient"):
                f(lambda t: t.clone().requires_grad_())
