"""Python binding of the operators in include/moe_ops.h: dispatch and combine of
tokens by expert with their gradients, and few-row products with 4-bit weights.

Argument checks and marshalling only; every step runs in the library's HIP
kernels, on the current stream of the tensors' device unless `stream` (a raw
stream handle of that device) is given. Outputs are allocated when not given.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

from . import MOE_OK, MoeError, _ptr, load_library

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


@functools.lru_cache(maxsize=None)
def _lib():
    lib = load_library()
    vp, u64 = ctypes.c_void_p, ctypes.c_uint64
    ds, ws = ctypes.POINTER(_DispatchShape), ctypes.POINTER(_W4Shape)
    for name, args in (
            ("dispatch_query", [ds, ctypes.POINTER(u64)]),
            ("dispatch", [vp, vp, ds, vp, vp, vp, vp, vp, u64, vp]),
            ("dispatch_backward", [vp, vp, ds, vp, vp]),
            ("combine", [vp, vp, vp, ds, vp, vp]),
            ("combine_backward", [vp, vp, vp, vp, ds, vp, vp, vp]),
            ("w4_linear", [vp, vp, vp, vp, vp, ws, vp, vp]),
            ("w4_grouped_linear", [vp, vp, vp, vp, vp, vp, ws, vp, vp])):
        fn = getattr(lib, "moe_ops_" + name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    return lib


@functools.lru_cache(maxsize=256)
def _c_shape(shape, *strides):
    return ctypes.byref(shape.to_c(*strides))


def _torch_dtype(name: str):
    import torch

    return getattr(torch, _TORCH_NAME[name])


def _check(t, what: str, shape: tuple, dtype, device):
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the first tensor on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _rows_stride(t, what: str, shape: tuple, dtype, device) -> int:
    """Elements between the rows of a matrix whose rows are contiguous."""
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, the first tensor on {device}")
    if shape[0] <= 1:
        if shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{what} must have contiguous rows")
        return 0
    if (shape[1] > 1 and t.stride(1) != 1) or t.stride(0) < shape[1]:
        raise ValueError(f"{what} must have contiguous rows that do not overlap")
    return t.stride(0)


def _run(name: str, device, stream, *args):
    """Call an entry point with `device` current (the library launches there)."""
    import torch

    if device.type != "cuda":
        raise ValueError(f"tensors must be on the GPU, got {device}")
    fn = getattr(_lib(), "moe_ops_" + name)
    if stream is None:
        stream = torch.cuda.current_stream(device).cuda_stream
    if device.index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != MOE_OK:
        raise MoeError(rc, "moe_ops_" + name)


def dispatch_query(shape: DispatchShape) -> int:
    """Workspace bytes of dispatch for a shape (raises MoeError if unsupported)."""
    n = ctypes.c_uint64()
    rc = _lib().moe_ops_dispatch_query(_c_shape(shape), ctypes.byref(n))
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
    import torch

    T, K, H, dev = shape.T, shape.topk, shape.H, x.device
    dt, i32 = _torch_dtype(shape.dtype), torch.int32
    nbytes = dispatch_query(shape)
    _check(x, "x", (T, H), dt, dev)
    _check(topk_ids, "topk_ids", (T, K), i32, dev)
    if out is None:
        out = torch.empty((T * K, H), dtype=dt, device=dev)
    else:
        _check(out, "out", (T * K, H), dt, dev)
    if offsets is None:
        offsets = torch.empty(shape.E + 1, dtype=i32, device=dev)
    else:
        _check(offsets, "offsets", (shape.E + 1,), i32, dev)
    if row_slot is None:
        row_slot = torch.empty(T * K, dtype=i32, device=dev)
    else:
        _check(row_slot, "row_slot", (T * K,), i32, dev)
    if slot_row is None:
        slot_row = torch.empty((T, K), dtype=i32, device=dev)
    else:
        _check(slot_row, "slot_row", (T, K), i32, dev)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        _check(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    _run("dispatch", dev, stream, _ptr(x), _ptr(topk_ids), _c_shape(shape), _ptr(out),
         _ptr(offsets), _ptr(row_slot), _ptr(slot_row), _ptr(workspace), workspace.numel())
    return out, offsets, row_slot, slot_row


def dispatch_backward(drows, slot_row, shape: DispatchShape, *, out=None, stream=None):
    """Gradient of dispatch with respect to x: drows [T * topk, H] -> [T, H]."""
    import torch

    T, K, H, dev = shape.T, shape.topk, shape.H, drows.device
    dt = _torch_dtype(shape.dtype)
    _check(drows, "drows", (T * K, H), dt, dev)
    _check(slot_row, "slot_row", (T, K), torch.int32, dev)
    if out is None:
        out = torch.empty((T, H), dtype=dt, device=dev)
    else:
        _check(out, "out", (T, H), dt, dev)
    _run("dispatch_backward", dev, stream, _ptr(drows), _ptr(slot_row), _c_shape(shape), _ptr(out))
    return out


def combine(rows, slot_row, topk_w, shape: DispatchShape, *, out=None, stream=None):
    """Rows back to token order: out[t] = sum_k topk_w[t, k] * rows[slot_row[t, k]].

    rows [T * topk, H]; slot_row as dispatch gives it; topk_w float32 [T, topk].
    """
    import torch

    T, K, H, dev = shape.T, shape.topk, shape.H, rows.device
    dt = _torch_dtype(shape.dtype)
    _check(rows, "rows", (T * K, H), dt, dev)
    _check(slot_row, "slot_row", (T, K), torch.int32, dev)
    _check(topk_w, "topk_w", (T, K), torch.float32, dev)
    if out is None:
        out = torch.empty((T, H), dtype=dt, device=dev)
    else:
        _check(out, "out", (T, H), dt, dev)
    _run("combine", dev, stream, _ptr(rows), _ptr(slot_row), _ptr(topk_w), _c_shape(shape),
         _ptr(out))
    return out


def combine_backward(dout, rows, slot_row, topk_w, shape: DispatchShape, *, dy=None, dw=None,
                     stream=None):
    """Gradients of combine from dout [T, H]: (drows [T * topk, H], dtopk_w
    float32 [T, topk]). Rows that no slot names stay as they were in `dy`;
    weights without a row get 0."""
    import torch

    T, K, H, dev = shape.T, shape.topk, shape.H, dout.device
    dt = _torch_dtype(shape.dtype)
    _check(dout, "dout", (T, H), dt, dev)
    _check(rows, "rows", (T * K, H), dt, dev)
    _check(slot_row, "slot_row", (T, K), torch.int32, dev)
    _check(topk_w, "topk_w", (T, K), torch.float32, dev)
    if dy is None:
        dy = torch.empty((T * K, H), dtype=dt, device=dev)
    else:
        _check(dy, "dy", (T * K, H), dt, dev)
    if dw is None:
        dw = torch.empty((T, K), dtype=torch.float32, device=dev)
    else:
        _check(dw, "dw", (T, K), torch.float32, dev)
    _run("combine_backward", dev, stream, _ptr(dout), _ptr(rows), _ptr(slot_row), _ptr(topk_w),
         _c_shape(shape), _ptr(dy), _ptr(dw))
    return dy, dw


def _w4(name, x, offsets, w, scales, shape, zeros, bias, out, stream):
    import torch

    M, N, K, E, dev = shape.M, shape.N, shape.K, shape.E, x.device
    if min(M, N - 1, K - 1, E - 1) < 0 or shape.group < 1:
        raise ValueError(f"sizes out of range: {shape}")
    dt, groups = _torch_dtype(shape.dtype), K // shape.group
    ldx = _rows_stride(x, "x", (M, K), dt, dev)

    def matrix(t, what, tail, dtype):
        bare = offsets is None and t.dim() == len(tail)  # one matrix, without its leading 1
        _check(t, what, tail if bare else (E, *tail), dtype, dev)

    matrix(w, "w", ((N + 15) // 16 * 16, K // 2), torch.uint8)
    matrix(scales, "scales", (N, groups), torch.uint8 if shape.format == "mxfp4" else dt)
    if zeros is not None:
        matrix(zeros, "zeros", (N, groups), torch.uint8)
    if bias is not None:
        matrix(bias, "bias", (N,), dt)
    odt = _torch_dtype(shape.out_dtype or shape.dtype)
    if out is None:
        out = torch.empty((M, N), dtype=odt, device=dev)
        ldo = 0
    else:
        ldo = _rows_stride(out, "out", (M, N), odt, dev)
    args = [_ptr(x)]
    if offsets is not None:
        _check(offsets, "offsets", (E + 1,), torch.int32, dev)
        args.append(_ptr(offsets))
    _run(name, dev, stream, *args, _ptr(w), _ptr(scales), _ptr(zeros), _ptr(bias),
         _c_shape(shape, ldx, ldo), _ptr(out))
    return out


def w4_linear(x, w, scales, shape: W4Shape, *, zeros=None, bias=None, out=None, stream=None):
    """out = x @ weight.T (+ bias) for a few rows of x and one 4-bit matrix.

    x [M, K] in shape.dtype (rows may be strided, multiples of 8 elements);
    w uint8 [Np, K / 2] as prepack returns it, Np = N rounded up to 16;
    scales uint8 [N, K / 32] E8M0 (mxfp4) or shape.dtype [N, K / group] (int4);
    zeros uint8 [N, K / group] (int4; None: 8); bias [N]. The matrix arrays may
    carry a leading 1. out [M, N] in shape.out_dtype (rows may be strided).
    """
    return _w4("w4_linear", x, None, w, scales, shape, zeros, bias, out, stream)


def w4_grouped_linear(x, offsets, w, scales, shape: W4Shape, *, zeros=None, bias=None, out=None,
                      stream=None):
    """Rows [offsets[e], offsets[e + 1]) of x times matrix e, as w4_linear.

    offsets int32 [E + 1] (as dispatch returns them); w [E, Np, K / 2]; scales
    and zeros [E, N, K / group]; bias [E, N]. Rows of out that no expert owns
    stay as they were.
    """
    return _w4("w4_grouped_linear", x, offsets, w, scales, shape, zeros, bias, out, stream)
