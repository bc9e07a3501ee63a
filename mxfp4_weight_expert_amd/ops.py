"""Python binding of the operators in include/moe_ops.h: dispatch and combine of
tokens by expert with their gradients, and few-row products with 4-bit weights.

Argument checks and marshalling only; every step runs in the library's HIP
kernels, on the current stream of the tensors' device or on `stream` (a raw
stream handle of that device), which has to be ordered after the inputs' writers.
Outputs and the workspace are allocated, for that stream, when not given.

Nothing is recorded for autograd: a tensor that requires a gradient is refused
where gradients are being recorded. The *_backward functions are the gradients,
for a torch.autograd.Function whose forward and backward make these calls. What a
call writes counts as changed, so that autograd refuses values it had saved of it.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass, fields

from . import MOE_OK, MoeError, load_library

__all__ = ["DispatchShape", "W4Shape", "dispatch_query", "dispatch", "dispatch_backward", "combine",
           "combine_backward", "w4_linear", "w4_grouped_linear", "DTYPE", "W4_FORMAT"]

DTYPE = {"bf16": 0, "fp16": 1, "fp32": 2}
W4_FORMAT = {"mxfp4": 0, "int4": 1}
_TORCH_NAME = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


class _DispatchShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "E", "topk", "H", "expert_offset", "dtype")]


class _W4Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "E", "format", "group", "dtype",
                                              "out_dtype")] + [("ldx", ctypes.c_int64),
                                                               ("ldo", ctypes.c_int64)]


# imported by the first call: the binding itself needs none
torch = _changed = None


def _torch_dtype(name: str):
    global torch, _changed
    import torch

    _changed = torch._C._increment_version  # torch.autograd.graph.increment_version, of tuples
    return getattr(torch, _TORCH_NAME[name])


class _Kept:
    """A shape is copied and pickled by its fields, without what it keeps."""

    def __reduce__(self):
        return type(self), tuple(getattr(self, f.name) for f in fields(self))

    @functools.cached_property
    def _fits(self) -> bool:
        """ctypes cuts a number off to 32 bits, where it would name another shape."""
        for n in self._sizes:
            if not -2 ** 31 <= getattr(self, n) < 2 ** 31:
                raise ValueError(f"{n} = {getattr(self, n)} is out of range")
        return True


# A shape's C struct, torch types and array shapes are worked out at its first
# call and kept on it: a decode step's calls are shorter than making them anew.


@dataclass(frozen=True)
class DispatchShape(_Kept):
    """Shape of dispatch and combine (fields as in moe_ops_dispatch_shape)."""

    T: int
    E: int
    topk: int
    H: int
    dtype: str = "bf16"
    expert_offset: int = 0
    _sizes = ("T", "E", "topk", "H", "expert_offset")

    def to_c(self) -> _DispatchShape:
        self._fits
        return _DispatchShape(self.T, self.E, self.topk, self.H, self.expert_offset,
                              DTYPE[self.dtype])

    @functools.cached_property
    def _c(self):
        return ctypes.byref(self.to_c())

    @functools.cached_property
    def _torch(self):
        return _torch_dtype(self.dtype)

    @functools.cached_property
    def _arrays(self):
        """Shapes of tokens, rows and maps."""
        return (self.T, self.H), (self.T * self.topk, self.H), (self.T, self.topk)

    @functools.cached_property
    def _workspace(self) -> int:
        return dispatch_query(self)


@dataclass(frozen=True)
class W4Shape(_Kept):
    """Shape of the 4-bit products (fields as in moe_ops_w4_shape; the row
    strides come from the tensors). out_dtype None: dtype."""

    M: int
    N: int
    K: int
    E: int = 1
    format: str = "mxfp4"
    group: int = 32
    dtype: str = "bf16"
    out_dtype: str = None
    _sizes = ("M", "N", "K", "E", "group")

    def to_c(self, ldx: int = 0, ldo: int = 0) -> _W4Shape:
        self._fits
        return _W4Shape(self.M, self.N, self.K, self.E, W4_FORMAT[self.format], self.group,
                        DTYPE[self.dtype], DTYPE[self.out_dtype or self.dtype], ldx, ldo)

    @functools.cached_property
    def _c(self):
        return ctypes.byref(self.to_c())

    @functools.cached_property
    def _torch(self):
        """Types of x, the scales and out."""
        dt = _torch_dtype(self.dtype)
        return dt, torch.uint8 if self.format == "mxfp4" else dt, _torch_dtype(self.out_dtype or self.dtype)

    @functools.cached_property
    def _arrays(self):
        """Shapes of the codes, group values and bias of one matrix, and of all."""
        if min(self.M, self.N - 1, self.K - 1, self.E - 1) < 0 or self.group < 1:
            raise ValueError(f"sizes out of range: {self}")
        one = ((self.N + 15) // 16 * 16, self.K // 2), (self.N, self.K // self.group), (self.N,)
        return one, tuple((self.E, *s) for s in one)


@functools.lru_cache(maxsize=None)
def _entry(name: str):
    vp, u64 = ctypes.c_void_p, ctypes.c_uint64
    ds, ws = ctypes.POINTER(_DispatchShape), ctypes.POINTER(_W4Shape)
    fn = getattr(load_library(), "moe_ops_" + name)
    fn.argtypes = {
        "dispatch_query": [ds, ctypes.POINTER(u64)],
        "dispatch": [vp, vp, ds, vp, vp, vp, vp, vp, u64, vp],
        "dispatch_backward": [vp, vp, ds, vp, vp],
        "combine": [vp, vp, vp, ds, vp, vp],
        "combine_backward": [vp, vp, vp, vp, ds, vp, vp, vp],
        "w4_linear": [vp, vp, vp, vp, vp, ws, vp, vp],
        "w4_grouped_linear": [vp, vp, vp, vp, vp, vp, ws, vp, vp]}[name]
    fn.restype = ctypes.c_int
    return fn


def _refuse(t, what: str, shape: tuple, dtype, index: int, layout: str):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != index:
        first = f"GPU {index}" if index >= 0 else "the CPU"
        raise ValueError(f"{what} is on {t.device}, the first tensor on {first}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient, and this call would record none: make it under "
                         "torch.no_grad() or in a torch.autograd.Function")
    raise ValueError(f"{what} must {layout}")


def _check(t, what: str, shape: tuple, dtype, index: int) -> int:
    """A contiguous tensor's address. index: the GPU of the call's first tensor."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous() and not (t.requires_grad and torch.is_grad_enabled())):
        return t.data_ptr()
    _refuse(t, what, shape, dtype, index, "be contiguous")


def _whole(t, what: str, shape: tuple, dtype, index: int) -> int:
    """_check for whole numbers, which never require a gradient."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, what, shape, dtype, index, "be contiguous")


def _row_stride(t, what: str, shape: tuple, dtype, index: int) -> int:
    """Elements between the rows of a matrix whose rows are contiguous; 0 where
    the rows follow each other."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == index
            and not (t.requires_grad and torch.is_grad_enabled())):
        if t.is_contiguous():
            return 0
        if (shape[1] <= 1 or t.stride(1) == 1) and (shape[0] <= 1 or t.stride(0) >= shape[1]):
            return t.stride(0) if shape[0] > 1 else 0
    _refuse(t, what, shape, dtype, index, "have contiguous rows that do not overlap")


def _on_stream(stream: int, t):
    """`stream` as the current one, so that what a call allocates belongs to it."""
    import torch

    if not t.is_cuda:
        raise ValueError(f"tensors must be on the GPU, got {t.device}")
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=t.device))


def _run(name: str, index: int, *args):
    """Call an entry point on the GPU's current stream, with that GPU current (the
    library launches there)."""
    if index < 0:
        raise ValueError("tensors must be on the GPU")
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        rc = _entry(name)(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = _entry(name)(*args, stream)
    if rc != MOE_OK:
        raise MoeError(rc, "moe_ops_" + name)


def dispatch_query(shape: DispatchShape) -> int:
    """Workspace bytes of dispatch for a shape (raises MoeError if unsupported)."""
    n = ctypes.c_uint64()
    rc = _entry("dispatch_query")(shape._c, ctypes.byref(n))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_ops_dispatch_query")
    return int(n.value)


def dispatch(x, topk_ids, shape: DispatchShape, *, out=None, offsets=None, row_slot=None,
             slot_row=None, workspace=None, stream=None):
    """Token rows into expert order; returns (rows, offsets, row_slot, slot_row).

    x [T, H]; topk_ids int32 [T, topk] global ids, those outside
    [expert_offset, expert_offset + E) without a row. rows [T * topk, H] and
    row_slot int32 [T * topk] hold offsets[E] rows, what lies behind stays as
    it was; offsets int32 [E + 1]; slot_row int32 [T, topk], -1 without a row.
    workspace: uint8, at least dispatch_query(shape) bytes.
    """
    dt, nbytes = shape._torch, shape._workspace
    if stream is not None:
        with _on_stream(stream, x):
            return dispatch(x, topk_ids, shape, out=out, offsets=offsets, row_slot=row_slot,
                            slot_row=slot_row, workspace=workspace)
    tokens, sorted_rows, maps = shape._arrays
    gpu, i32 = x.get_device(), torch.int32
    px, pi = _check(x, "x", tokens, dt, gpu), _whole(topk_ids, "topk_ids", maps, i32, gpu)
    dev = x.device
    if out is None:
        out = torch.empty(sorted_rows, dtype=dt, device=dev)
    if offsets is None:
        offsets = torch.empty(shape.E + 1, dtype=i32, device=dev)
    if row_slot is None:
        row_slot = torch.empty(sorted_rows[0], dtype=i32, device=dev)
    if slot_row is None:
        slot_row = torch.empty(maps, dtype=i32, device=dev)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _run("dispatch", gpu, px, pi, shape._c, _check(out, "out", sorted_rows, dt, gpu),
         _whole(offsets, "offsets", (shape.E + 1,), i32, gpu),
         _whole(row_slot, "row_slot", sorted_rows[:1], i32, gpu),
         _whole(slot_row, "slot_row", maps, i32, gpu),
         _whole(workspace, "workspace", workspace.shape, torch.uint8, gpu), workspace.numel())
    _changed((out, offsets, row_slot, slot_row))
    return out, offsets, row_slot, slot_row


def dispatch_backward(drows, slot_row, shape: DispatchShape, *, out=None, stream=None):
    """Gradient of dispatch with respect to x: drows [T * topk, H] -> [T, H]."""
    dt = shape._torch
    if stream is not None:
        with _on_stream(stream, drows):
            return dispatch_backward(drows, slot_row, shape, out=out)
    tokens, sorted_rows, maps = shape._arrays
    gpu = drows.get_device()
    pd, ps = _check(drows, "drows", sorted_rows, dt, gpu), _whole(slot_row, "slot_row", maps, torch.int32, gpu)
    if out is None:
        out = torch.empty(tokens, dtype=dt, device=drows.device)
    _run("dispatch_backward", gpu, pd, ps, shape._c, _check(out, "out", tokens, dt, gpu))
    _changed((out,))
    return out


def combine(rows, slot_row, topk_w, shape: DispatchShape, *, out=None, stream=None):
    """Rows back to token order: out[t] = sum_k topk_w[t, k] * rows[slot_row[t, k]].

    rows [T * topk, H]; slot_row as dispatch gives it; topk_w float32 [T, topk].
    """
    dt = shape._torch
    if stream is not None:
        with _on_stream(stream, rows):
            return combine(rows, slot_row, topk_w, shape, out=out)
    tokens, sorted_rows, maps = shape._arrays
    gpu = rows.get_device()
    pr, ps = _check(rows, "rows", sorted_rows, dt, gpu), _whole(slot_row, "slot_row", maps, torch.int32, gpu)
    pw = _check(topk_w, "topk_w", maps, torch.float32, gpu)
    if out is None:
        out = torch.empty(tokens, dtype=dt, device=rows.device)
    _run("combine", gpu, pr, ps, pw, shape._c, _check(out, "out", tokens, dt, gpu))
    _changed((out,))
    return out


def combine_backward(dout, rows, slot_row, topk_w, shape: DispatchShape, *, dy=None, dw=None,
                     stream=None):
    """Gradients of combine from dout [T, H]: (drows [T * topk, H], dtopk_w
    float32 [T, topk]). Rows that no slot names stay as they were in `dy`;
    weights without a row get 0."""
    dt = shape._torch
    if stream is not None:
        with _on_stream(stream, dout):
            return combine_backward(dout, rows, slot_row, topk_w, shape, dy=dy, dw=dw)
    tokens, sorted_rows, maps = shape._arrays
    gpu, f32 = dout.get_device(), torch.float32
    pd, pr = _check(dout, "dout", tokens, dt, gpu), _check(rows, "rows", sorted_rows, dt, gpu)
    ps, pw = _whole(slot_row, "slot_row", maps, torch.int32, gpu), _check(topk_w, "topk_w", maps, f32, gpu)
    if dy is None:
        dy = torch.empty(sorted_rows, dtype=dt, device=dout.device)
    if dw is None:
        dw = torch.empty(maps, dtype=f32, device=dout.device)
    _run("combine_backward", gpu, pd, pr, ps, pw, shape._c, _check(dy, "dy", sorted_rows, dt, gpu),
         _check(dw, "dw", maps, f32, gpu))
    _changed((dy, dw))
    return dy, dw


def _matrix(t, what: str, bare: tuple, shape: tuple, dtype, gpu: int, grouped: bool):
    """Address of a matrix array; a single matrix may come without its leading 1."""
    check = _whole if dtype is torch.uint8 else _check
    return check(t, what, shape if grouped or t.dim() == len(shape) else bare, dtype, gpu)


def _w4(name, x, offsets, w, scales, shape, zeros, bias, out):
    dt, sdt, odt = shape._torch
    one, every = shape._arrays
    gpu, grouped = x.get_device(), offsets is not None
    ldx, ldo = _row_stride(x, "x", (shape.M, shape.K), dt, gpu), 0
    if out is None:
        out = torch.empty((shape.M, shape.N), dtype=odt, device=x.device)
    else:
        ldo = _row_stride(out, "out", (shape.M, shape.N), odt, gpu)
    cshape = ctypes.byref(shape.to_c(ldx, ldo)) if ldx or ldo else shape._c
    args = (_matrix(w, "w", one[0], every[0], torch.uint8, gpu, grouped),
            _matrix(scales, "scales", one[1], every[1], sdt, gpu, grouped),
            None if zeros is None else _matrix(zeros, "zeros", one[1], every[1], torch.uint8, gpu, grouped),
            None if bias is None else _matrix(bias, "bias", one[2], every[2], dt, gpu, grouped),
            cshape, out.data_ptr())
    if grouped:
        args = (_whole(offsets, "offsets", (shape.E + 1,), torch.int32, gpu), *args)
    _run(name, gpu, x.data_ptr(), *args)
    _changed((out,))
    return out


def w4_linear(x, w, scales, shape: W4Shape, *, zeros=None, bias=None, out=None, stream=None):
    """out = x @ weight.T (+ bias) for a few rows of x and one 4-bit matrix.

    x [M, K] in shape.dtype (rows may be strided, multiples of 8 elements);
    w uint8 [Np, K / 2] as prepack returns it, Np = N rounded up to 16;
    scales uint8 [N, K / 32] E8M0 (mxfp4) or shape.dtype [N, K / group] (int4);
    zeros uint8 [N, K / group] (int4; None: 8); bias [N]. The matrix arrays may
    carry a leading 1. out [M, N] in shape.out_dtype (rows may be strided).
    """
    if stream is not None:
        with _on_stream(stream, x):
            return _w4("w4_linear", x, None, w, scales, shape, zeros, bias, out)
    return _w4("w4_linear", x, None, w, scales, shape, zeros, bias, out)


def w4_grouped_linear(x, offsets, w, scales, shape: W4Shape, *, zeros=None, bias=None, out=None,
                      stream=None):
    """Rows [offsets[e], offsets[e + 1]) of x times matrix e, as w4_linear.

    offsets int32 [E + 1] (as dispatch returns them); w [E, Np, K / 2]; scales
    and zeros [E, N, K / group]; bias [E, N]. Rows of out that no expert owns
    stay as they were.
    """
    if offsets is None:
        raise ValueError("offsets are needed")
    if stream is not None:
        with _on_stream(stream, x):
            return _w4("w4_grouped_linear", x, offsets, w, scales, shape, zeros, bias, out)
    return _w4("w4_grouped_linear", x, offsets, w, scales, shape, zeros, bias, out)
