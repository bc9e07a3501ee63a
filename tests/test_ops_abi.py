"""Host-side checks of the operators' C ABI and binding (no GPU needed): the
library exports what the header declares, structs agree, and bad arguments are
refused before anything is launched."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import mxfp4_weight_expert_amd as moe
from mxfp4_weight_expert_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_ops.h")

# The refusals below pass fabricated addresses: never where a kernel could start.
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="fabricated device addresses: run only where no GPU is visible")


def test_library_exports_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_ops_\w+)\s*\(", text))
    nm = subprocess.run(["nm", "-D", "--defined-only", moe.lib_path], capture_output=True, text=True)
    assert names == set(re.findall(r"\bT (moe_ops_\w+)", nm.stdout)) and len(names) == 7


@pytest.mark.parametrize("lang", ["c99", "c++"])
def test_structs_match_header(tmp_path, lang):
    pairs = [("moe_ops_dispatch_shape", ops._DispatchShape), ("moe_ops_w4_shape", ops._W4Shape)]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe_ops.h"', "int main(void){"]
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


def _ds(**kw):
    return moe.DispatchShape(**{**dict(T=64, E=896, topk=16, H=512), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(topk=0), 1), (dict(H=0), 1), (dict(expert_offset=-1), 1),
    (dict(topk=33), 2), (dict(E=2049), 2), (dict(H=(1 << 24) + 1), 2), (dict(T=(1 << 19) + 1), 2),
    (dict(T=1 << 15, topk=1, H=1 << 24), 2), (dict(T=1 << 20, topk=1, H=(1 << 13) + 1), 2),
])
def test_dispatch_query_refuses(kw, code):
    with pytest.raises(moe.MoeError) as ei:
        moe.dispatch_query(_ds(**kw))
    assert ei.value.code == code


def test_dispatch_query_sizes():
    assert moe.dispatch_query(_ds()) >= 256
    assert moe.dispatch_query(_ds(T=0)) >= 256
    big = moe.dispatch_query(_ds(T=32768))
    assert big >= 512 * 896 * 4 + 896 * 4 and big % 256 == 0
    bad = _ds().to_c()
    bad.dtype = 3
    n = ctypes.c_uint64()
    query = ops._entry("dispatch_query")
    assert query(ctypes.byref(bad), ctypes.byref(n)) == 2
    assert query(None, ctypes.byref(n)) == 1
    assert query(ctypes.byref(_ds().to_c()), None) == 1


MB = 1 << 20
# addresses a MB times 256 apart, so that no two arrays of these shapes touch
A = {n: (i + 1) * 256 * MB for i, n in enumerate(
    ["x", "ids", "rows", "offsets", "row_slot", "slot_row", "ws", "w", "out", "dw", "scales", "zeros", "bias"])}


def _p(v):
    return ctypes.c_void_p(v) if v else None


def _dispatch(shape, wsb=1 << 30, **kw):
    a = {**A, **kw}
    return ops._entry("dispatch")(_p(a["x"]), _p(a["ids"]), ctypes.byref(shape.to_c()),
                                       _p(a["rows"]), _p(a["offsets"]), _p(a["row_slot"]),
                                       _p(a["slot_row"]), _p(a["ws"]), wsb, None)


@no_gpu
def test_dispatch_refuses_before_launch():
    s = _ds()
    for n in ("x", "ids", "rows", "offsets", "row_slot", "slot_row"):
        assert _dispatch(s, **{n: 0}) == 1, n
    for n in ("ids", "offsets", "row_slot", "slot_row"):
        assert _dispatch(s, **{n: A[n] + 2}) == 1, n
    assert _dispatch(s, x=A["x"] + 1) == 1
    f = _ds(dtype="fp32")
    assert _dispatch(f, x=A["x"] + 2) == 1 and _dispatch(f, rows=A["rows"] + 2) == 1
    assert _dispatch(s, ws=0) == 3 and _dispatch(s, ws=A["ws"] + 64) == 3 and _dispatch(s, wsb=64) == 3
    assert _dispatch(_ds(T=8192), wsb=4096) == 3
    # overlaps: rows on x, offsets on the ids, row_slot inside slot_row
    assert _dispatch(s, rows=A["x"] + 64 * 512 * 2 - 2) == 1
    assert _dispatch(s, rows=A["x"] + 64 * 512 * 2, wsb=0) == 3  # side by side is fine
    assert _dispatch(s, offsets=A["ids"] + 64 * 16 * 4 - 4) == 1
    assert _dispatch(s, row_slot=A["slot_row"] + 4) == 1


def _combine(name, shape, **kw):
    a = {**A, **kw}
    sh = ctypes.byref(shape.to_c())
    if name == "dispatch_backward":
        return ops._entry("dispatch_backward")(_p(a["rows"]), _p(a["slot_row"]), sh, _p(a["out"]), None)
    if name == "combine":
        return ops._entry("combine")(_p(a["rows"]), _p(a["slot_row"]), _p(a["w"]), sh, _p(a["out"]), None)
    return ops._entry("combine_backward")(_p(a["x"]), _p(a["rows"]), _p(a["slot_row"]), _p(a["w"]), sh,
                                        _p(a["out"]), _p(a["dw"]), None)


@no_gpu
@pytest.mark.parametrize("name,args", [
    ("dispatch_backward", ("rows", "slot_row", "out")), ("combine", ("rows", "slot_row", "w", "out")),
    ("combine_backward", ("x", "rows", "slot_row", "w", "out", "dw"))])
def test_combine_refuses_before_launch(name, args):
    s = _ds()
    for n in args:
        assert _combine(name, s, **{n: 0}) == 1, n
        assert _combine(name, s, **{n: A[n] + 1}) == 1, n
        assert _combine(name, _ds(T=0), **{n: 0}) == 0, n  # nothing to do, nothing looked at
        assert _combine(name, _ds(topk=33), **{n: 0}) == 2, n
    assert _combine(name, s, out=A["rows"] + 2) == 1
    assert _combine(name, s, out=A["slot_row"]) == 1


def _ws(**kw):
    return moe.W4Shape(**{**dict(M=4, N=100, K=256), **kw})


def _w4(shape, grouped=False, ldx=0, ldo=0, **kw):
    a = {**A, "zeros": 0, "bias": 0, **kw}
    sh = ctypes.byref(shape.to_c(ldx, ldo))
    if grouped:
        return ops._entry("w4_grouped_linear")(_p(a["x"]), _p(a["offsets"]), _p(a["w"]), _p(a["scales"]),
                                             _p(a["zeros"]), _p(a["bias"]), sh, _p(a["out"]), None)
    return ops._entry("w4_linear")(_p(a["x"]), _p(a["w"]), _p(a["scales"]), _p(a["zeros"]),
                                 _p(a["bias"]), sh, _p(a["out"]), None)


@no_gpu
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(E=0), 1), (dict(K=192), 2),
    (dict(K=8192 + 128), 2), (dict(N=(1 << 24) + 1), 2), (dict(M=(1 << 23) + 1), 2), (dict(E=2049), 2),
    (dict(group=64), 2), (dict(format="int4", group=256), 2), (dict(format="int4", group=16), 2),
    (dict(dtype="fp32"), 2), (dict(M=1 << 23, N=1 << 24), 2),
    (dict(M=1 << 20, N=1 << 18), 2),
])
def test_w4_refuses_shapes(kw, code):
    assert _w4(_ws(**kw), grouped=True) == code


@no_gpu
def test_w4_refuses_before_launch():
    assert _w4(_ws(E=2)) == 1  # one matrix
    for n in ("x", "w", "scales", "out"):
        assert _w4(_ws(), **{n: 0}) == 1, n
        assert _w4(_ws(), **{n: A[n] + 1}) == 1, n
    assert _w4(_ws(), x=A["x"] + 8) == 1 and _w4(_ws(), w=A["w"] + 8) == 1
    assert _w4(_ws(), scales=A["scales"] + 2) == 1 and _w4(_ws(), bias=A["bias"] + 1) == 1
    assert _w4(_ws(out_dtype="fp32"), out=A["out"] + 2) == 1
    assert _w4(_ws(), zeros=A["zeros"]) == 1  # zero points belong to int4
    assert _w4(_ws(format="int4"), zeros=A["zeros"] + 2) == 1
    assert _w4(_ws(), grouped=True, offsets=0) == 1
    assert _w4(_ws(), grouped=True, offsets=A["offsets"] + 2) == 1
    assert _w4(_ws(), ldx=248) == 1 and _w4(_ws(), ldx=260) == 1 and _w4(_ws(), ldo=99) == 1
    assert _w4(_ws(), ldx=(1 << 24) + 8) == 2 and _w4(_ws(), ldo=(1 << 24) + 8) == 2
    assert _w4(_ws(), ldx=-8) == 1 and _w4(_ws(), ldo=-1) == 1
    assert _w4(_ws(), out=A["x"] + 256) == 1 and _w4(_ws(), out=A["w"] + 16) == 1
    assert _w4(_ws(M=0), x=0, out=0) == 0
    for field, v in (("format", 2), ("dtype", 3), ("out_dtype", 3), ("out_dtype", -1)):
        c = _ws().to_c()
        setattr(c, field, v)
        assert ops._entry("w4_linear")(_p(A["x"]), _p(A["w"]), _p(A["scales"]), None, None,
                                            ctypes.byref(c), _p(A["out"]), None) == 2, field
    assert ops._entry("w4_linear")(None, None, None, None, None, None, None, None) == 1


def test_shapes_copy_and_pickle_after_use():
    import copy
    import pickle

    d, w = _ds(T=3), _ws(format="int4", group=64)
    moe.dispatch_query(d)
    assert w._c is not None and w._arrays  # what a call keeps on the shape
    for s in (d, w):
        for t in (copy.deepcopy(s), pickle.loads(pickle.dumps(s))):
            assert t == s and hash(t) == hash(s)


def test_binding_refuses_host_tensors_and_wrong_layouts():
    s = _ds(T=2, E=4, topk=2, H=8)
    x, ids = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    for kw in ({}, {"stream": 0}):
        with pytest.raises(ValueError, match="GPU"):
            moe.dispatch(x, ids, s, **kw)
        with pytest.raises(ValueError, match="GPU"):
            moe.dispatch(x=x, topk_ids=ids, shape=s, **kw)
    with pytest.raises(ValueError, match="topk_ids"):
        moe.dispatch(x, ids.long(), s)
    with pytest.raises(ValueError, match="contiguous"):
        moe.dispatch(torch.zeros(8, 2, dtype=torch.bfloat16).t(), ids, s)
    with pytest.raises(ValueError, match="x must be"):
        moe.dispatch(x[:1], ids, s)
    with pytest.raises(ValueError, match="slot_row"):
        moe.combine(torch.zeros(4, 8, dtype=torch.bfloat16), ids[:1], torch.zeros(2, 2), s)
    with pytest.raises(ValueError, match="dout"):
        moe.combine_backward(x.float(), torch.zeros(4, 8, dtype=torch.bfloat16), ids, torch.zeros(2, 2), s)
    w = moe.W4Shape(M=2, N=20, K=128)
    xw, ww = torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.uint8)
    sc = torch.zeros(20, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        moe.w4_linear(xw, ww, sc, w)
    with pytest.raises(ValueError, match="w must be"):
        moe.w4_linear(xw, ww[:20], sc, w)
    with pytest.raises(ValueError, match="scales"):
        moe.w4_linear(xw, ww, sc.float(), w)
    with pytest.raises(ValueError, match="overlap"):
        moe.w4_linear(xw[:1].expand(2, 128), ww, sc, w)
    with pytest.raises(ValueError, match="contiguous rows"):
        moe.w4_linear(torch.zeros(128, 2, dtype=torch.bfloat16).t(), ww, sc, w)
