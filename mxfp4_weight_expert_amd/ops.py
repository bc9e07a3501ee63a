"""Python binding of the operators in include/moe_ops.h: dispatch and combine of
tokens by expert with their gradients, and few-row products with 4-bit weights.

Argument checks and marshalling only; every step runs in the library's HIP
kernels, on the current stream of the tensors' device or on `stream` (a raw
stream handle of that device), which has to be ordered after the inputs' writers.
Outputs and the workspace are allocated, for that stream, when not given.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from dataclasses import dataclass

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


def _torch_dtype(name: str):
    import torch

    return getattr(torch, _TORCH_NAME[name])


# A shape's C struct, torch types and array shapes are worked out at its first
# call and kept on it: a decode step's calls are shorter than making them anew.


@dataclass(frozen=True)
class DispatchShape:
    """Shape of dispatch and combine (fields as in moe_ops_dispatch_shape)."""

    T: int
    E: int
    topk: int
    H: int
    dtype: str = "bf16"
    expert_offset: int = 0

    def to_c(self) -> _DispatchShape:
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
class W4Shape:
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

    def to_c(self, ldx: int = 0, ldo: int = 0) -> _W4Shape:
        return _W4Shape(self.M, self.N, self.K, self.E, W4_FORMAT[self.format], self.group,
                        DTYPE[self.dtype], DTYPE[self.out_dtype or self.dtype], ldx, ldo)

    @functools.cached_property
    def _c(self):
        return ctypes.byref(self.to_c())

    @functools.cached_property
    def _torch(self):
        """Types of x, the scales and out."""
        import torch

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


def _check(t, what: str, shape: tuple, dtype, device):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the first tensor on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _row_stride(t, what: str, shape: tuple, dtype, device) -> int:
    """Elements between the rows of a matrix whose rows are contiguous; 0 where
    the rows follow each other."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the first tensor on {device}")
    if t.is_contiguous():
        return 0
    if (shape[1] > 1 and t.stride(1) != 1) or (shape[0] > 1 and t.stride(0) < shape[1]):
        raise ValueError(f"{what} must have contiguous rows that do not overlap")
    return t.stride(0) if shape[0] > 1 else 0


def _result(t, what: str, shape: tuple, dtype, device):
    """The caller's output, checked, or a new one."""
    if t is None:
        import torch

        return torch.empty(shape, dtype=dtype, device=device)
    _check(t, what, shape, dtype, device)
    return t


def _with_stream(fn):
    """Gives an operator its `stream` argument: that stream is the current one
    during the call, so that what the call allocates belongs to it."""

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch

        device = (args[0] if args else next(iter(kw.values()))).device
        if device.type != "cuda":
            raise ValueError(f"tensors must be on the GPU, got {device}")
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
            return fn(*args, **kw)

    sig = inspect.signature(fn)
    call.__signature__ = sig.replace(parameters=[
        *sig.parameters.values(),
        inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def _run(name: str, device, *args):
    """Call an entry point on the device's current stream, with `device` current
    (the library launches there)."""
    import torch

    if device.type != "cuda":
        raise ValueError(f"tensors must be on the GPU, got {device}")
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch._C._cuda_getDevice():
        rc = _entry(name)(*args, stream)
    else:
        with torch.cuda.device(device):
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


@_with_stream
def dispatch(x, topk_ids, shape: DispatchShape, *, out=None, offsets=None, row_slot=None,
             slot_row=None, workspace=None):
    """Token rows into expert order; returns (rows, offsets, row_slot, slot_row).

    x [T, H]; topk_ids int32 [T, topk] global ids, those outside
    [expert_offset, expert_offset + E) without a row. rows [T * topk, H] and
    row_slot int32 [T * topk] hold offsets[E] rows, what lies behind stays as
    it was; offsets int32 [E + 1]; slot_row int32 [T, topk], -1 without a row.
    workspace: uint8, at least dispatch_query(shape) bytes.
    """
    import torch

    dev, dt, i32 = x.device, shape._torch, torch.int32
    nbytes = shape._workspace
    tokens, sorted_rows, maps = shape._arrays
    _check(x, "x", tokens, dt, dev)
    _check(topk_ids, "topk_ids", maps, i32, dev)
    out = _result(out, "out", sorted_rows, dt, dev)
    offsets = _result(offsets, "offsets", (shape.E + 1,), i32, dev)
    row_slot = _result(row_slot, "row_slot", sorted_rows[:1], i32, dev)
    slot_row = _result(slot_row, "slot_row", maps, i32, dev)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        _check(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    _run("dispatch", dev, x.data_ptr(), topk_ids.data_ptr(), shape._c, out.data_ptr(),
         offsets.data_ptr(), row_slot.data_ptr(), slot_row.data_ptr(), workspace.data_ptr(),
         workspace.numel())
    return out, offsets, row_slot, slot_row


@_with_stream
def dispatch_backward(drows, slot_row, shape: DispatchShape, *, out=None):
    """Gradient of dispatch with respect to x: drows [T * topk, H] -> [T, H]."""
    import torch

    dev, dt = drows.device, shape._torch
    tokens, sorted_rows, maps = shape._arrays
    _check(drows, "drows", sorted_rows, dt, dev)
    _check(slot_row, "slot_row", maps, torch.int32, dev)
    out = _result(out, "out", tokens, dt, dev)
    _run("dispatch_backward", dev, drows.data_ptr(), slot_row.data_ptr(), shape._c,
         out.data_ptr())
    return out


@_with_stream
def combine(rows, slot_row, topk_w, shape: DispatchShape, *, out=None):
    """Rows back to token order: out[t] = sum_k topk_w[t, k] * rows[slot_row[t, k]].

    rows [T * topk, H]; slot_row as dispatch gives it; topk_w float32 [T, topk].
    """
    import torch

    dev, dt = rows.device, shape._torch
    tokens, sorted_rows, maps = shape._arrays
    _check(rows, "rows", sorted_rows, dt, dev)
    _check(slot_row, "slot_row", maps, torch.int32, dev)
    _check(topk_w, "topk_w", maps, torch.float32, dev)
    out = _result(out, "out", tokens, dt, dev)
    _run("combine", dev, rows.data_ptr(), slot_row.data_ptr(), topk_w.data_ptr(), shape._c,
         out.data_ptr())
    return out


@_with_stream
def combine_backward(dout, rows, slot_row, topk_w, shape: DispatchShape, *, dy=None, dw=None):
    """Gradients of combine from dout [T, H]: (drows [T * topk, H], dtopk_w
    float32 [T, topk]). Rows that no slot names stay as they were in `dy`;
    weights without a row get 0."""
    import torch

    dev, dt = dout.device, shape._torch
    tokens, sorted_rows, maps = shape._arrays
    _check(dout, "dout", tokens, dt, dev)
    _check(rows, "rows", sorted_rows, dt, dev)
    _check(slot_row, "slot_row", maps, torch.int32, dev)
    _check(topk_w, "topk_w", maps, torch.float32, dev)
    dy = _result(dy, "dy", sorted_rows, dt, dev)
    dw = _result(dw, "dw", maps, torch.float32, dev)
    _run("combine_backward", dev, dout.data_ptr(), rows.data_ptr(), slot_row.data_ptr(),
         topk_w.data_ptr(), shape._c, dy.data_ptr(), dw.data_ptr())
    return dy, dw


def _w4(name, x, offsets, w, scales, shape, zeros, bias, out):
    import torch

    dev = x.device
    dt, sdt, odt = shape._torch
    one, every = shape._arrays

    def matrix(t, what, i, dtype):
        if t is None:
            return None
        bare = offsets is None and t.dim() == len(one[i])  # one matrix, without its leading 1
        _check(t, what, one[i] if bare else every[i], dtype, dev)
        return t.data_ptr()

    ldx, ldo = _row_stride(x, "x", (shape.M, shape.K), dt, dev), 0
    if out is None:
        out = torch.empty((shape.M, shape.N), dtype=odt, device=dev)
    else:
        ldo = _row_stride(out, "out", (shape.M, shape.N), odt, dev)
    cshape = ctypes.byref(shape.to_c(ldx, ldo)) if ldx or ldo else shape._c
    args = [matrix(w, "w", 0, torch.uint8), matrix(scales, "scales", 1, sdt),
            matrix(zeros, "zeros", 1, torch.uint8), matrix(bias, "bias", 2, dt), cshape, out.data_ptr()]
    if offsets is not None:
        _check(offsets, "offsets", (shape.E + 1,), torch.int32, dev)
        args.insert(0, offsets.data_ptr())
    _run(name, dev, x.data_ptr(), *args)
    return out


@_with_stream
def w4_linear(x, w, scales, shape: W4Shape, *, zeros=None, bias=None, out=None):
    """out = x @ weight.T (+ bias) for a few rows of x and one 4-bit matrix.

    x [M, K] in shape.dtype (rows may be strided, multiples of 8 elements);
    w uint8 [Np, K / 2] as prepack returns it, Np = N rounded up to 16;
    scales uint8 [N, K / 32] E8M0 (mxfp4) or shape.dtype [N, K / group] (int4);
    zeros uint8 [N, K / group] (int4; None: 8); bias [N]. The matrix arrays may
    carry a leading 1. out [M, N] in shape.out_dtype (rows may be strided).
    """
    return _w4("w4_linear", x, None, w, scales, shape, zeros, bias, out)


@_with_stream
def w4_grouped_linear(x, offsets, w, scales, shape: W4Shape, *, zeros=None, bias=None, out=None):
    """Rows [offsets[e], offsets[e + 1]) of x times matrix e, as w4_linear.

    offsets int32 [E + 1] (as dispatch returns them); w [E, Np, K / 2]; scales
    and zeros [E, N, K / group]; bias [E, N]. Rows of out that no expert owns
    stay as they were.
    """
    return _w4("w4_grouped_linear", x, offsets, w, scales, shape, zeros, bias, out)
