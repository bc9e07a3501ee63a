"""Python binding of the 16-bit products in include/moe_linear.h: rows times their
expert's matrix, the gated product of a feed-forward block, both with their
gradients, and low-rank adapters of many requests.

Argument checks and marshalling only, in the manner of ops.py: every step runs in
the library's HIP kernels, on the current stream of the tensors' device or on
`stream` (a raw stream handle of that device), which has to be ordered after the
inputs' writers. Outputs and workspaces are allocated, for that stream, when not
given. Nothing is recorded for autograd: the *_backward functions are the
gradients, for a torch.autograd.Function whose forward and backward make these
calls.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

from . import ACTIVATION, MOE_OK, MoeError, load_library, ops
from .ops import DTYPE, _check, _Kept, _on_stream, _row_stride, _torch_dtype, _whole

__all__ = ["LinearShape", "GatedShape", "AdapterShape", "adapter_query", "adapter_maps", "adapter_linear", "grouped_linear", "grouped_linear_backward", "gated_linear",
           "gated_linear_backward"]


class _LinearShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "E", "dtype", "out_dtype")] + [
        ("ldx", ctypes.c_int64), ("ldo", ctypes.c_int64)]


class _GatedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "I", "H", "E", "dtype", "activation")] + [
        (n, ctypes.c_float) for n in ("swiglu_limit", "act_beta", "act_linear_beta")] + [
        ("dgu_terms", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldo", ctypes.c_int64)]


class _AdapterShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "R", "A", "dtype", "out_dtype")] + [
        (n, ctypes.c_int64) for n in ("ldx", "ldb", "ldo")]


@dataclass(frozen=True)
class LinearShape(_Kept):
    """Shape of the grouped product (fields as in moe_linear_shape; the row strides
    come from the tensors). out_dtype None: dtype."""

    M: int
    N: int
    K: int
    E: int = 1
    dtype: str = "bf16"
    out_dtype: str = None
    _sizes = ("M", "N", "K", "E")

    def to_c(self, ldx: int = 0, ldo: int = 0) -> _LinearShape:
        self._fits
        return _LinearShape(self.M, self.N, self.K, self.E, DTYPE[self.dtype],
                            DTYPE[self.out_dtype or self.dtype], ldx, ldo)

    @functools.cached_property
    def _c(self):
        return ctypes.byref(self.to_c())

    @functools.cached_property
    def _torch(self):
        return _torch_dtype(self.dtype), _torch_dtype(self.out_dtype or self.dtype)

    @functools.cached_property
    def _arrays(self):
        """Shapes of x, out and the matrices."""
        return (self.M, self.K), (self.M, self.N), (self.E, self.N, self.K)


@dataclass(frozen=True)
class GatedShape(_Kept):
    """Shape of the gated product (fields as in moe_gated_shape; the row strides
    come from the tensors)."""

    M: int
    I: int
    H: int
    E: int = 1
    dtype: str = "bf16"
    activation: str = "swiglu"  # or "situ"
    swiglu_limit: float = 0.0
    act_beta: float = 4.0  # SiTU caps (read only for "situ")
    act_linear_beta: float = 25.0
    dgu_terms: int = 1  # 2: the backward pass keeps what rounding dgu leaves
    _sizes = ("M", "I", "H", "E", "dgu_terms")

    def to_c(self, ldx: int = 0, ldo: int = 0) -> _GatedShape:
        self._fits
        return _GatedShape(self.M, self.I, self.H, self.E, DTYPE[self.dtype], ACTIVATION[self.activation],
                           float(self.swiglu_limit), float(self.act_beta), float(self.act_linear_beta), self.dgu_terms, ldx, ldo)

    @functools.cached_property
    def _c(self):
        return ctypes.byref(self.to_c())

    @functools.cached_property
    def _torch(self):
        return _torch_dtype(self.dtype)

    @functools.cached_property
    def _arrays(self):
        """Shapes of x, h, the pre-activations and the matrices."""
        return (self.M, self.H), (self.M, self.I), (self.M, 2 * self.I), (self.E, 2 * self.I, self.H)

    @functools.cached_property
    def _dgu(self):
        return (self.M, 2 * self.I) if self.dgu_terms <= 1 else (self.dgu_terms, self.M, 2 * self.I)


@dataclass(frozen=True)
class AdapterShape(_Kept):
    """Shape of the adapters' product (fields as in moe_adapter_shape; the row
    strides come from the tensors). out_dtype None: dtype."""

    M: int
    N: int
    K: int
    R: int
    A: int
    dtype: str = "bf16"
    out_dtype: str = None
    _sizes = ("M", "N", "K", "R", "A")

    def to_c(self, ldx: int = 0, ldb: int = 0, ldo: int = 0) -> _AdapterShape:
        self._fits
        return _AdapterShape(self.M, self.N, self.K, self.R, self.A, DTYPE[self.dtype],
                             DTYPE[self.out_dtype or self.dtype], ldx, ldb, ldo)

    @functools.cached_property
    def _c(self):
        return ctypes.byref(self.to_c())

    @functools.cached_property
    def _torch(self):
        return _torch_dtype(self.dtype), _torch_dtype(self.out_dtype or self.dtype)

    @functools.cached_property
    def _arrays(self):
        """Shapes of x, out, a, b and the maps."""
        return ((self.M, self.K), (self.M, self.N), (self.A, self.R, self.K), (self.A, self.N, self.R),
                (self.A + 1,), (self.M,), (self.A,))

    @functools.cached_property
    def _workspace(self) -> int:
        return adapter_query(self)


@functools.lru_cache(maxsize=None)
def _entry(name: str):
    vp = ctypes.c_void_p
    ls, gs, ads = (ctypes.POINTER(c) for c in (_LinearShape, _GatedShape, _AdapterShape))
    u64 = ctypes.c_uint64
    fn = getattr(load_library(), "moe_linear_" + name)
    fn.argtypes = {
        "grouped": [vp, vp, vp, ls, vp, vp],
        "grouped_backward": [vp, vp, vp, vp, ls, vp, vp, vp],
        "gated": [vp, vp, vp, gs, vp, vp, vp],
        "gated_backward": [vp, vp, vp, vp, vp, gs, vp, vp, vp, vp],
        "adapter_query": [ads, ctypes.POINTER(u64)],
        "adapter_maps": [vp, ads, vp, vp, vp, vp, u64, vp],
        "adapter": [vp, vp, vp, vp, vp, vp, vp, ads, vp, vp, vp, u64, vp]}[name]
    fn.restype = ctypes.c_int
    return fn


def _run(name: str, index: int, *args):
    ops._call(_entry(name), "moe_linear_" + name, index, args)


def _offsets(offsets, E: int, gpu: int):
    if offsets is None:
        if E != 1:
            raise ValueError("offsets are needed where there are several matrices")
        return None
    return _whole(offsets, "offsets", (E + 1,), ops.torch.int32, gpu)


def _matrices(w, what: str, shape: tuple, dtype, gpu: int) -> int:
    """Address of the matrices; a single one may come without its leading 1."""
    return _check(w, what, shape[1:] if shape[0] == 1 and w.dim() == 2 else shape, dtype, gpu)


def grouped_linear(x, offsets, w, shape: LinearShape, *, out=None, stream=None):
    """Rows [offsets[e], offsets[e + 1]) of x times matrix e: out[m] = w[e] @ x[m].

    x [M, K] in shape.dtype (rows may be strided, multiples of 8 elements);
    offsets int32 [E + 1] (as dispatch returns them), or None with one matrix: all
    rows; w [E, N, K] (a single matrix may come as [N, K]). out [M, N] in
    shape.out_dtype (rows may be strided); rows that no expert owns stay as they
    were.
    """
    dt, odt = shape._torch
    if stream is not None:
        with _on_stream(stream, x):
            return grouped_linear(x, offsets, w, shape, out=out)
    rows, result, matrices = shape._arrays
    gpu = x.get_device()
    ldx, ldo = _row_stride(x, "x", rows, dt, gpu), 0
    if out is None:
        out = ops.torch.empty(result, dtype=odt, device=x.device)
    else:
        ldo = _row_stride(out, "out", result, odt, gpu)
    _run("grouped", gpu, x.data_ptr(), _offsets(offsets, shape.E, gpu), _matrices(w, "w", matrices, dt, gpu),
         ctypes.byref(shape.to_c(ldx, ldo)) if ldx or ldo else shape._c, out.data_ptr())
    ops._changed((out,))
    return out


def _gradient(t, shape: tuple, dtype, like):
    """The tensor for a gradient: given, to be made (None), or not wanted (False)."""
    if t is False:
        return None
    return ops.torch.empty(shape, dtype=dtype, device=like.device) if t is None else t


def _given(t, what: str, gradient, name: str) -> bool:
    """Whether an operand is there; the one that a wanted gradient reads has to be."""
    if t is None and gradient is not False:
        raise ValueError(f"{what} is needed for {name}")
    return t is not None


def grouped_linear_backward(dout, x, offsets, w, shape: LinearShape, *, dx=None, dw=None, stream=None):
    """Gradients of grouped_linear from dout [M, N] in shape.dtype: (dx [M, K],
    dw [E, N, K] in shape.out_dtype). Rows of dx that no expert owns stay as they
    were; an expert without rows gets zeros in dw. dx or dw False: not computed,
    None in its place (x, or w, may then be None). All arrays are contiguous.
    """
    dt, odt = shape._torch
    if stream is not None:
        with _on_stream(stream, dout):
            return grouped_linear_backward(dout, x, offsets, w, shape, dx=dx, dw=dw)
    rows, result, matrices = shape._arrays
    gpu = dout.get_device()
    pd, po = _check(dout, "dout", result, dt, gpu), _offsets(offsets, shape.E, gpu)
    px = _check(x, "x", rows, dt, gpu) if _given(x, "x", dw, "dw") else None
    pw = _matrices(w, "w", matrices, dt, gpu) if _given(w, "w", dx, "dx") else None
    dx, dw = _gradient(dx, rows, dt, dout), _gradient(dw, matrices, odt, dout)
    _run("grouped_backward", gpu, pd, px, po, pw, shape._c, None if dx is None else _check(dx, "dx", rows, dt, gpu),
         None if dw is None else _matrices(dw, "dw", matrices, odt, gpu))
    ops._changed(tuple(t for t in (dx, dw) if t is not None))
    return dx, dw


def gated_linear(x, offsets, w13, shape: GatedShape, *, out=None, gu=None, stream=None):
    """h = act(g, u) with g and u the products of x's rows and their expert's gate
    and up matrices; returns h [M, I].

    x [M, H] (rows may be strided, multiples of 8 elements); offsets as for
    grouped_linear; w13 [E, 2 I, H], gate rows first. out [M, I] (rows may be
    strided). gu: a tensor [M, 2 I] that takes the pre-activations for
    gated_linear_backward. Rows that no expert owns stay as they were in both.
    """
    dt = shape._torch
    if stream is not None:
        with _on_stream(stream, x):
            return gated_linear(x, offsets, w13, shape, out=out, gu=gu)
    rows, result, pre, matrices = shape._arrays
    gpu = x.get_device()
    ldx, ldo = _row_stride(x, "x", rows, dt, gpu), 0
    if out is None:
        out = ops.torch.empty(result, dtype=dt, device=x.device)
    else:
        ldo = _row_stride(out, "out", result, dt, gpu)
    _run("gated", gpu, x.data_ptr(), _offsets(offsets, shape.E, gpu), _matrices(w13, "w13", matrices, dt, gpu),
         ctypes.byref(shape.to_c(ldx, ldo)) if ldx or ldo else shape._c, out.data_ptr(),
         None if gu is None else _check(gu, "gu", pre, dt, gpu))
    ops._changed((out,) if gu is None else (out, gu))
    return out


def gated_linear_backward(dh, x, offsets, gu, w13, shape: GatedShape, *, dx=None, dw=None, dgu=None, stream=None):
    """Gradients of gated_linear from dh [M, I] at the pre-activations gu [M, 2 I]:
    (dx [M, H], dw [E, 2 I, H]). dgu [M, 2 I] takes the gradient of the
    pre-activations in the rows that experts own (made here when None), rounded to
    shape.dtype before the products that take it; with shape.dgu_terms 2 it is
    [2, M, 2 I], a sum of two such values, and dx and dw are off by their own
    rounding alone, in one and a half to two times the time. dx or dw False: not
    computed, None in its place. All arrays are contiguous.
    """
    dt = shape._torch
    if stream is not None:
        with _on_stream(stream, dh):
            return gated_linear_backward(dh, x, offsets, gu, w13, shape, dx=dx, dw=dw, dgu=dgu)
    rows, result, pre, matrices = shape._arrays
    gpu = dh.get_device()
    pd, po, pg = _check(dh, "dh", result, dt, gpu), _offsets(offsets, shape.E, gpu), _check(gu, "gu", pre, dt, gpu)
    px = _check(x, "x", rows, dt, gpu) if _given(x, "x", dw, "dw") else None
    pw = _matrices(w13, "w13", matrices, dt, gpu) if _given(w13, "w13", dx, "dx") else None
    if dgu is None:
        dgu = ops.torch.empty(shape._dgu, dtype=dt, device=dh.device)
    dx, dw = _gradient(dx, rows, dt, dh), _gradient(dw, matrices, dt, dh)
    _run("gated_backward", gpu, pd, px, po, pg, pw, shape._c, _check(dgu, "dgu", shape._dgu, dt, gpu),
         None if dx is None else _check(dx, "dx", rows, dt, gpu), None if dw is None else _matrices(dw, "dw", matrices, dt, gpu))
    ops._changed(tuple(t for t in (dgu, dx, dw) if t is not None))
    return dx, dw


def adapter_query(shape: AdapterShape) -> int:
    """Workspace bytes of adapter_maps and adapter_linear for a shape (raises MoeError
    if unsupported)."""
    n = ctypes.c_uint64()
    rc = _entry("adapter_query")(shape._c, ctypes.byref(n))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_linear_adapter_query")
    return int(n.value)


def _workspace(workspace, nbytes: int, like):
    if workspace is None:
        workspace = ops.torch.empty(nbytes, dtype=ops.torch.uint8, device=like.device)
    return workspace, _whole(workspace, "workspace", workspace.shape, ops.torch.uint8, like.get_device())


def adapter_maps(ids, shape: AdapterShape, *, offsets=None, row_slot=None, slot_row=None, workspace=None, stream=None):
    """Rows sorted by adapter; returns (offsets, row_slot, slot_row) for every
    adapter_linear with the same ids.

    ids int32 [M]: a row's adapter, any value outside [0, A) for none. offsets
    int32 [A + 1], row_slot (sorted row -> row) and slot_row (row -> sorted row,
    or -1) int32 [M]. workspace: uint8, at least adapter_query(shape) bytes.
    """
    nbytes = shape._workspace
    if stream is not None:
        with _on_stream(stream, ids):
            return adapter_maps(ids, shape, offsets=offsets, row_slot=row_slot, slot_row=slot_row, workspace=workspace)
    shape._torch  # imports torch
    *_, bounds, rows, _ = shape._arrays
    gpu, i32 = ids.get_device(), ops.torch.int32
    pi = _whole(ids, "ids", rows, i32, gpu)
    made = [ops.torch.empty(s, dtype=i32, device=ids.device) if t is None else t
            for t, s in ((offsets, bounds), (row_slot, rows), (slot_row, rows))]
    workspace, pw = _workspace(workspace, nbytes, ids)
    _run("adapter_maps", gpu, pi, shape._c, _whole(made[0], "offsets", bounds, i32, gpu),
         _whole(made[1], "row_slot", rows, i32, gpu), _whole(made[2], "slot_row", rows, i32, gpu), pw, workspace.numel())
    ops._changed(tuple(made))
    return tuple(made)


def adapter_linear(x, offsets, row_slot, slot_row, a, b, scale, shape: AdapterShape, *, base=None, out=None, workspace=None,
                   stream=None):
    """out[m] = base[m] + scale[i] * b[i] @ (a[i] @ x[m]), i the adapter of row m;
    rows without one get base[m].

    x [M, K] in shape.dtype (rows may be strided, multiples of 8 elements); the
    maps as adapter_maps returns them; a [A, R, K], b [A, N, R]; scale float32 [A]
    or None: 1. base [M, N] in shape.out_dtype, or None: 0; out [M, N] may be base
    itself (rows of both may be strided). workspace: uint8, at least
    adapter_query(shape) bytes.
    """
    (dt, odt), nbytes = shape._torch, shape._workspace
    if stream is not None:
        with _on_stream(stream, x):
            return adapter_linear(x, offsets, row_slot, slot_row, a, b, scale, shape, base=base, out=out, workspace=workspace)
    rows, result, down, up, bounds, maps, scales = shape._arrays
    gpu, i32 = x.get_device(), ops.torch.int32
    ldx, ldb = _row_stride(x, "x", rows, dt, gpu), 0
    if base is not None:
        ldb = _row_stride(base, "base", result, odt, gpu)
    if out is None:
        out, ldo = ops.torch.empty(result, dtype=odt, device=x.device), 0
    else:
        ldo = ldb if out is base else _row_stride(out, "out", result, odt, gpu)
    workspace, pw = _workspace(workspace, nbytes, x)
    _run("adapter", gpu, x.data_ptr(), _whole(offsets, "offsets", bounds, i32, gpu),
         _whole(row_slot, "row_slot", maps, i32, gpu), _whole(slot_row, "slot_row", maps, i32, gpu),
         _check(a, "a", down, dt, gpu), _check(b, "b", up, dt, gpu),
         None if scale is None else _check(scale, "scale", scales, ops.torch.float32, gpu),
         ctypes.byref(shape.to_c(ldx, ldb, ldo)) if ldx or ldb or ldo else shape._c,
         None if base is None else base.data_ptr(), out.data_ptr(), pw, workspace.numel())
    ops._changed((out,))
    return out
