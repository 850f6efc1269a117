"""Step operators: what a rank computes next to its collectives.

The calls of the C ABI in ``include/ringsim_ops.h``, which defines what every
one of them computes:

    rms_norm(x, weight=None, *, residual=None, eps=1e-6, out_dtype=None, group=0, ...)
        -> RmsNorm(out, residual, scales)
    rms_norm_backward(grad_out, h, weight=None, *, grad_residual=None, eps=1e-6, ...)
        -> RmsNormGrads(grad_in, grad_weight)
    grad_norm(grads, *, scale=1.0, ...) -> 0-dim float32 tensor
    scale_grads(grads, norm, max_norm, *, outs=None, scale=1.0, eps=1e-6, ...)
    clip_grads(grads, max_norm, *, outs=None, scale=1.0, eps=1e-6, ...) -> 0-dim float32 tensor

Arguments are device tensors of the current device. Calls are asynchronous on
``stream`` (a torch stream or a raw handle; default: the current torch
stream); results and workspaces that a call allocates come from that stream's
memory, so they are safe to use and to drop there. A tensor the caller brings
must be ready on that stream and stay alive until the work is done, as for
every call of this package. None of them records anything for autograd;
tensors they write advance their version, so that autograd notices a saved
tensor that was overwritten. Wrong
arguments raise TypeError or ValueError before anything is enqueued; codes of
the library raise RingsimError.

The marshalling itself is compiled (``csrc/ops_binding.cpp``); a missing
library raises.
"""
from __future__ import annotations

from typing import NamedTuple, Sequence

import torch

from . import RingsimError, lib

lib()  # libringsim first, from the package
from . import _ops_binding as _b  # noqa: E402

_b.set_errors(RingsimError, torch.OutOfMemoryError)

NORM_MAX_COLS = 32768


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
    """A context that makes ``stream`` the current one."""
    if not isinstance(stream, int):
        return torch.cuda.stream(stream)
    if stream == 0:
        return torch.cuda.stream(torch.cuda.default_stream())
    return torch.cuda.stream(torch.cuda.ExternalStream(stream))


def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, out_dtype=None, group: int = 0, out=None,
             residual_out=None, scales=None, stream=None) -> RmsNorm:
    """Root-mean-square norm of the last dimension, with the residual added
    in front of it:  h = x + residual,  out = h / sqrt(mean(h^2) + eps) * weight.

    float32, bfloat16 or float16; the weight of x's dtype or float32. Rows may
    be apart in memory: up to two leading dimensions of any strides, or more
    of which all but the last follow one another without gaps (dimensions of
    size 1 do not count).
    ``out_dtype="float8_e4m3"`` (or torch.float8_e4m3fn) gives 8-bit values
    and fp32 ``scales`` of shape ``x.shape[:-1] + (groups,)``: one for every
    ``group`` columns (32, 64 or 128), or one a row (group 0).
    ``out``, ``residual_out`` and ``scales`` may be given; ``out`` and
    ``residual_out`` may be ``x`` or ``residual`` themselves."""
    if stream is not None:
        with _on(stream):
            return rms_norm(x, weight, residual=residual, eps=eps, out_dtype=out_dtype, group=group, out=out,
                            residual_out=residual_out, scales=scales)
    quant = 0
    if out_dtype is not None:
        quant = out_dtype == "float8_e4m3" or out_dtype is torch.float8_e4m3fn
        if not quant and out_dtype is not x.dtype:
            raise TypeError(f"unsupported out_dtype {out_dtype}")
    return RmsNorm._make(_b.rms_norm(x, weight, residual, eps, quant, group, out, residual_out, scales))


def rms_norm_backward(grad_out, h, weight=None, *, grad_residual=None, eps: float = 1e-6, grad_in=None,
                      grad_weight=None, need_grad_weight: bool = True, stream=None) -> RmsNormGrads:
    """Gradients of :func:`rms_norm`. ``h`` is what was normed: the forward
    call's ``residual``, or its x. ``grad_residual`` is the gradient that
    reaches h past the norm and is added to ``grad_in``. ``grad_in`` may be
    ``grad_out``, ``h`` or ``grad_residual`` itself; ``grad_weight`` is
    overwritten."""
    if stream is not None:
        with _on(stream):
            return rms_norm_backward(grad_out, h, weight, grad_residual=grad_residual, eps=eps, grad_in=grad_in,
                                     grad_weight=grad_weight, need_grad_weight=need_grad_weight)
    return RmsNormGrads._make(_b.rms_norm_backward(grad_out, h, weight, grad_residual, eps, grad_in, grad_weight,
                                                   need_grad_weight))


def grad_norm(grads: Sequence, *, scale: float = 1.0, norm=None, stream=None):
    """|scale| times the 2-norm of all tensors of ``grads`` together, as a
    float32 tensor of one element (``norm`` if given). Contiguous tensors of
    float32, bfloat16 and float16, in any mix."""
    if stream is not None:
        with _on(stream):
            return _b.grad_norm(grads, scale, norm)
    return _b.grad_norm(grads, scale, norm)


def scale_grads(grads: Sequence, norm, max_norm: float, *, outs=None, scale: float = 1.0, eps: float = 1e-6,
                stream=None) -> None:
    """outs = grads * scale * min(1, max_norm / (norm + eps)) with ``norm``
    read from the device; in place without ``outs``."""
    if stream is not None:
        with _on(stream):
            return _b.scale_grads(grads, norm, max_norm, outs, scale, eps)
    return _b.scale_grads(grads, norm, max_norm, outs, scale, eps)


def clip_grads(grads: Sequence, max_norm: float, *, outs=None, scale: float = 1.0, eps: float = 1e-6, norm=None,
               stream=None):
    """:func:`grad_norm` of ``grads`` and :func:`scale_grads` by it in one
    call; returns the norm (before clipping)."""
    if stream is not None:
        with _on(stream):
            return _b.clip_grads(grads, max_norm, outs, scale, eps, norm)
    return _b.clip_grads(grads, max_norm, outs, scale, eps, norm)
