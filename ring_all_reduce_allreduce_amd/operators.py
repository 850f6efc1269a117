"""Step operators: what a rank computes next to its collectives.

Marshalling for the C ABI in ``include/ringsim_ops.h``, which defines what
every call computes:

    rms_norm(x, weight=None, *, residual=None, eps=1e-6, out_dtype=None, group=0, ...)
        -> RmsNorm(out, residual, scales)
    rms_norm_backward(grad_out, h, weight=None, *, grad_residual=None, eps=1e-6, ...)
        -> RmsNormGrads(grad_in, grad_weight)
    grad_norm(grads, *, scale=1.0, ...) -> 0-dim float32 tensor
    scale_grads(grads, norm, max_norm, *, outs=None, scale=1.0, eps=1e-6, ...)
    clip_grads(grads, max_norm, *, outs=None, scale=1.0, eps=1e-6, ...) -> 0-dim float32 tensor

Arguments are device tensors of the current device. Calls are asynchronous on
``stream`` (default: the current torch stream); results and workspaces that a
call allocates come from that stream's memory, so they are safe to use and to
drop there. A tensor the caller brings must be ready on that stream and stay
alive until the work is done, as for every call of this package. Wrong
arguments raise TypeError or ValueError before anything is enqueued; codes of
the library raise RingsimError.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Sequence

import torch

from . import _check, _current_stream, lib

FLOAT8_E4M3 = 17
OP_DTYPES = {torch.float32: 2, torch.bfloat16: 3, torch.float16: 16}
NORM_MAX_COLS = 32768
_i64x2 = ctypes.c_int64 * 2


class RmsNormArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("residual", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("residual_out", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("x_stride", _i64x2),
        ("residual_stride", _i64x2),
        ("out_stride", _i64x2),
        ("residual_out_stride", _i64x2),
        ("outer", ctypes.c_int64),
        ("inner", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("dtype", ctypes.c_int),
        ("weight_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("group", ctypes.c_int),
        ("eps", ctypes.c_float),
    ]


class RmsNormBackwardArgs(ctypes.Structure):
    _fields_ = [
        ("grad_out", ctypes.c_void_p),
        ("h", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("grad_residual", ctypes.c_void_p),
        ("grad_in", ctypes.c_void_p),
        ("grad_weight", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("grad_out_stride", _i64x2),
        ("h_stride", _i64x2),
        ("grad_residual_stride", _i64x2),
        ("grad_in_stride", _i64x2),
        ("outer", ctypes.c_int64),
        ("inner", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("dtype", ctypes.c_int),
        ("weight_dtype", ctypes.c_int),
        ("eps", ctypes.c_float),
    ]


class RmsNorm(NamedTuple):
    """``out``: the normed rows. ``residual``: x + residual, None without a
    residual. ``scales``: fp32 scales of an output in 8 bits, else None."""

    out: torch.Tensor
    residual: torch.Tensor | None
    scales: torch.Tensor | None


class RmsNormGrads(NamedTuple):
    """``grad_in``: gradient of x and of the residual alike. ``grad_weight``:
    None without a weight or where it was not wanted."""

    grad_in: torch.Tensor
    grad_weight: torch.Tensor | None


def _on(stream):
    """(context that allocates on the call's stream, its raw handle)."""
    current = _current_stream()
    if stream is None:
        return contextlib.nullcontext(), current
    raw = stream if isinstance(stream, int) else stream.cuda_stream
    if raw == current:
        return contextlib.nullcontext(), raw
    return torch.cuda.stream(torch.cuda.ExternalStream(raw) if isinstance(stream, int) else stream), raw


def _device(t, name: str) -> None:
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be a tensor on the current device")


def _rows(t, name: str, shape, dtype) -> tuple:
    """The {outer, inner} strides of a tensor whose rows are its last
    dimension: up to two leading dimensions of any strides, or more that
    follow one another in memory without gaps."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    _device(t, name)
    st = t.stride()
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    n = len(shape)
    if n == 1:
        return (0, 0)
    if n == 2:
        return (st[0], 0)
    if n > 3:
        for i in range(n - 3):
            if shape[i] != 1 and st[i] != st[i + 1] * shape[i + 1]:
                raise ValueError(f"the leading dimensions of {name} must be contiguous among themselves")
    return (st[-3], st[-2])


def _outer_inner(shape) -> tuple:
    if len(shape) <= 2:
        return (shape[0] if len(shape) == 2 else 1), 1
    outer = 1
    for s in shape[:-2]:
        outer *= s
    return outer, shape[-2]


def _norm_types(x, weight, name: str) -> tuple:
    code = OP_DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype} of {name}")
    if x.dim() == 0:
        raise ValueError(f"{name} needs at least one dimension")
    if weight is None:
        return code, code
    wcode = OP_DTYPES.get(weight.dtype)
    if wcode != code and weight.dtype != torch.float32:
        raise TypeError(f"weight must have dtype {x.dtype} or torch.float32, not {weight.dtype}")
    if weight.dim() != 1 or weight.shape[0] != x.shape[-1]:
        raise ValueError(f"weight must have shape ({x.shape[-1]},), not {tuple(weight.shape)}")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    _device(weight, "weight")
    return code, wcode


def _ptr(t):
    return None if t is None else t.data_ptr()


def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, out_dtype=None, group: int = 0, out=None,
             residual_out=None, scales=None, stream=None) -> RmsNorm:
    """Root-mean-square norm of the last dimension, with the residual added
    in front of it.

    ``out_dtype="float8_e4m3"`` (or torch.float8_e4m3fn) gives 8-bit values
    and fp32 ``scales`` of shape ``x.shape[:-1] + (groups,)``: one for every
    ``group`` columns (32, 64 or 128), or one a row (group 0).
    ``out``, ``residual_out`` and ``scales`` may be given; ``out`` and
    ``residual_out`` may be ``x`` or ``residual`` themselves."""
    code, wcode = _norm_types(x, weight, "x")
    if out_dtype is None or out_dtype is x.dtype:
        quant, out_torch, out_code = False, x.dtype, code
    elif out_dtype == "float8_e4m3" or out_dtype is torch.float8_e4m3fn:
        quant, out_torch, out_code = True, torch.float8_e4m3fn, FLOAT8_E4M3
    else:
        raise TypeError(f"unsupported out_dtype {out_dtype}")
    if group not in ((0, 32, 64, 128) if quant else (0,)):
        raise ValueError(f"unsupported group {group}")
    shape = x.shape
    xs = _rows(x, "x", shape, x.dtype)
    rs = _rows(residual, "residual", shape, x.dtype) if residual is not None else (0, 0)
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if not quant and scales is not None:
        raise ValueError("scales come with an output in 8 bits")
    ctx, raw = _on(stream)
    with ctx:
        if out is None:
            out = torch.empty(shape, dtype=out_torch, device=x.device)
        if residual is not None and residual_out is None:
            residual_out = torch.empty(shape, dtype=x.dtype, device=x.device)
        if quant:
            want = (*shape[:-1], -(-shape[-1] // group) if group else 1)
            if scales is None:
                scales = torch.empty(want, dtype=torch.float32, device=x.device)
            elif scales.dtype != torch.float32 or tuple(scales.shape) != want or not scales.is_contiguous():
                raise ValueError(f"scales must be contiguous float32 of shape {want}")
            else:
                _device(scales, "scales")
    os_ = _rows(out, "out", shape, out_torch)
    ros = _rows(residual_out, "residual_out", shape, x.dtype) if residual is not None else (0, 0)
    outer, inner = _outer_inner(shape)
    a = RmsNormArgs(x.data_ptr(), _ptr(residual), _ptr(weight), out.data_ptr(), _ptr(residual_out), _ptr(scales),
                    xs, rs, os_, ros, outer, inner, shape[-1], code, wcode, out_code, group, eps)
    _check(lib().ringsim_rms_norm(ctypes.byref(a), raw), "ringsim_rms_norm")
    return RmsNorm(out, residual_out, scales)


def rms_norm_backward(grad_out, h, weight=None, *, grad_residual=None, eps: float = 1e-6, grad_in=None,
                      grad_weight=None, need_grad_weight: bool = True, stream=None) -> RmsNormGrads:
    """Gradients of :func:`rms_norm`. ``h`` is what was normed: the forward
    call's ``residual``, or its x. ``grad_residual`` is the gradient that
    reaches h past the norm and is added to ``grad_in``. ``grad_in`` may be
    ``grad_out``, ``h`` or ``grad_residual`` itself."""
    code, wcode = _norm_types(h, weight, "h")
    shape = h.shape
    hs = _rows(h, "h", shape, h.dtype)
    gs = _rows(grad_out, "grad_out", shape, h.dtype)
    rs = _rows(grad_residual, "grad_residual", shape, h.dtype) if grad_residual is not None else (0, 0)
    if weight is None and grad_weight is not None:
        raise ValueError("grad_weight needs a weight")
    outer, inner = _outer_inner(shape)
    need = weight is not None and (need_grad_weight or grad_weight is not None)
    if grad_weight is not None:
        if grad_weight.dtype != weight.dtype or grad_weight.shape != weight.shape or not grad_weight.is_contiguous():
            raise ValueError("grad_weight must be contiguous, of the weight's shape and dtype")
        _device(grad_weight, "grad_weight")
    ctx, raw = _on(stream)
    workspace, nbytes = None, ctypes.c_size_t(0)
    with ctx:
        if grad_in is None:
            grad_in = torch.empty(shape, dtype=h.dtype, device=h.device)
        if need:
            if grad_weight is None:
                grad_weight = torch.empty_like(weight)
            _check(lib().ringsim_rms_norm_backward_workspace(outer * inner, shape[-1], nbytes),
                   "ringsim_rms_norm_backward_workspace")
            workspace = torch.empty(nbytes.value, dtype=torch.uint8, device=h.device)
    is_ = _rows(grad_in, "grad_in", shape, h.dtype)
    a = RmsNormBackwardArgs(grad_out.data_ptr(), h.data_ptr(), _ptr(weight), _ptr(grad_residual), grad_in.data_ptr(),
                            _ptr(grad_weight), _ptr(workspace), nbytes.value, gs, hs, rs, is_, outer, inner,
                            shape[-1], code, wcode, eps)
    _check(lib().ringsim_rms_norm_backward(ctypes.byref(a), raw), "ringsim_rms_norm_backward")
    return RmsNormGrads(grad_in, grad_weight)


def _list(tensors, name: str) -> list:
    tensors = list(tensors)
    device = torch.cuda.current_device()
    for t in tensors:
        if t.dtype not in OP_DTYPES:
            raise TypeError(f"unsupported dtype {t.dtype} in {name}")
        if t.get_device() != device:
            raise ValueError(f"{name} must be tensors on the current device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return tensors


def _grad_args(grads, outs) -> tuple:
    grads = _list(grads, "grads")
    n = len(grads)
    ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in grads])
    counts = (ctypes.c_int64 * n)(*[t.numel() for t in grads])
    types = (ctypes.c_int * n)(*[OP_DTYPES[t.dtype] for t in grads])
    if outs is None:
        return n, ptrs, None, counts, types
    outs = _list(outs, "outs")
    if len(outs) != n or any(o.dtype != g.dtype or o.numel() != g.numel() for o, g in zip(outs, grads)):
        raise ValueError("outs must match grads in number, sizes and dtypes")
    return n, ptrs, (ctypes.c_void_p * n)(*[t.data_ptr() for t in outs]), counts, types


def _norm_out(norm):
    if norm is None:
        return torch.empty((), dtype=torch.float32, device="cuda")
    if norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be one float32")
    _device(norm, "norm")
    return norm


def _norm_workspace(n: int):
    nbytes = ctypes.c_size_t(0)
    _check(lib().ringsim_grad_norm_workspace(n, nbytes), "ringsim_grad_norm_workspace")
    return torch.empty(nbytes.value, dtype=torch.uint8, device="cuda"), nbytes.value


def grad_norm(grads: Sequence, *, scale: float = 1.0, norm=None, stream=None):
    """|scale| times the 2-norm of all tensors of ``grads`` together, as a
    float32 tensor of one element (``norm`` if given). Contiguous tensors of
    float32, bfloat16 and float16, in any mix."""
    n, ptrs, _, counts, types = _grad_args(grads, None)
    ctx, raw = _on(stream)
    with ctx:
        norm = _norm_out(norm)
        ws, nbytes = _norm_workspace(n)
    _check(lib().ringsim_grad_norm(n, ptrs, counts, types, scale, norm.data_ptr(), ws.data_ptr(), nbytes, raw),
           "ringsim_grad_norm")
    return norm


def scale_grads(grads: Sequence, norm, max_norm: float, *, outs=None, scale: float = 1.0, eps: float = 1e-6,
                stream=None) -> None:
    """outs = grads * scale * min(1, max_norm / (norm + eps)) with ``norm``
    read from the device; in place without ``outs``."""
    n, ptrs, optrs, counts, types = _grad_args(grads, outs)
    norm = _norm_out(norm)
    _check(lib().ringsim_scale_grads(n, ptrs, optrs, counts, types, scale, norm.data_ptr(), max_norm, eps,
                                     _on(stream)[1]), "ringsim_scale_grads")


def clip_grads(grads: Sequence, max_norm: float, *, outs=None, scale: float = 1.0, eps: float = 1e-6, norm=None,
               stream=None):
    """:func:`grad_norm` of ``grads`` and :func:`scale_grads` by it in one
    call; returns the norm (before clipping)."""
    n, ptrs, optrs, counts, types = _grad_args(grads, outs)
    ctx, raw = _on(stream)
    with ctx:
        norm = _norm_out(norm)
        ws, nbytes = _norm_workspace(n)
    _check(lib().ringsim_clip_grads(n, ptrs, optrs, counts, types, scale, max_norm, eps, norm.data_ptr(),
                                    ws.data_ptr(), nbytes, raw), "ringsim_clip_grads")
    return norm
