"""PyTorch-facing wrappers of dropout (include/dropout.h).

Argument marshalling only; the computation runs in ``liblinear_logp.so``.  The
mask is a function of (seed, offset, element index): nothing is stored, and the
backward draws it again.  Tensors are bf16, fp16 or fp32, contiguous, on a CUDA
device.
"""
from __future__ import annotations

from typing import Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .ops import _dtype_code, _need_cuda, _out, _raw_stream, on_tensor_device

_MASK64 = (1 << 64) - 1
Offset = Union[int, torch.Tensor]


def _check(x: torch.Tensor, name: str):
    _need_cuda(x, name)
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _dtype_code(x, name)


def _counter(seed: int, offset: Offset, device_offset: Optional[torch.Tensor], device):
    """(seed, host offset, device pointer or None)."""
    if device_offset is None:
        if not isinstance(offset, torch.Tensor):
            return int(seed) & _MASK64, int(offset) & _MASK64, None
        offset, device_offset = 0, offset
    if isinstance(offset, torch.Tensor):
        raise ValueError("offset must be an int beside device_offset")
    t = device_offset
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int64 or t.numel() != 1 or t.device != device:
        raise ValueError("an offset must be an int, or one int64 on the inputs' device")
    return int(seed) & _MASK64, int(offset) & _MASK64, t.data_ptr()


def _probability(p: float) -> float:
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must lie in [0, 1], got {p}")
    return p


@on_tensor_device
def dropout_fwd(x: torch.Tensor, p: float, seed: int, offset: Offset = 0, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, device_offset: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + (kept ? x / (1 - p) : 0), p rounded to a multiple of 2^-16.  ``offset`` numbers
    the mask under one seed; as an int64 tensor on the device it is read when the kernel
    runs, so that a captured graph can advance it between replays.  With ``device_offset``
    the mask's number is offset + device_offset: the layers of a captured step share one
    counter on the device (advanced by the number of layers) and each adds its own offset;
    under one number they would draw one mask.  ``out`` may be x or residual itself."""
    code = _check(x, "x")
    dev = x.device
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.shape != x.shape or residual.dtype != x.dtype:
            raise ValueError("residual must have x's shape and dtype")
        if residual.device != dev or not residual.is_contiguous():
            raise ValueError("residual must be contiguous, on x's device")
    seed, off, off_ptr = _counter(seed, offset, device_offset, dev)
    p = _probability(p)
    y = _out(out, x.shape, x.dtype, dev)
    st = _lib.load().dropout_fwd(x.data_ptr(), None if residual is None else residual.data_ptr(), code, x.numel(), p,
                                 seed, off, off_ptr, y.data_ptr(), _raw_stream(dev.index))
    _lib.check("dropout_fwd", st)
    return y


@on_tensor_device
def dropout_bwd(grad_y: torch.Tensor, p: float, seed: int, offset: Offset = 0,
                out: Optional[torch.Tensor] = None, device_offset: Optional[torch.Tensor] = None) -> torch.Tensor:
    """grad_x = kept ? grad_y / (1 - p) : 0 under the forward's p, seed and offsets."""
    code = _check(grad_y, "grad_y")
    dev = grad_y.device
    seed, off, off_ptr = _counter(seed, offset, device_offset, dev)
    p = _probability(p)
    gx = _out(out, grad_y.shape, grad_y.dtype, dev)
    st = _lib.load().dropout_bwd(grad_y.data_ptr(), code, grad_y.numel(), p, seed, off, off_ptr, gx.data_ptr(),
                                 _raw_stream(dev.index))
    _lib.check("dropout_bwd", st)
    return gx


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset, device_offset):
        ctx.p, ctx.seed, ctx.offset = p, seed, offset
        if device_offset is not None:
            ctx.save_for_backward(device_offset)
        return dropout_fwd(x, p, seed, offset, residual, device_offset=device_offset)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        device_offset = ctx.saved_tensors[0] if ctx.saved_tensors else None
        gx = None
        if ctx.needs_input_grad[0]:
            gx = dropout_bwd(grad_y.contiguous(), ctx.p, ctx.seed, ctx.offset, device_offset=device_offset)
        return gx, grad_y if ctx.needs_input_grad[1] else None, None, None, None, None


def dropout(x: torch.Tensor, p: float, seed: int, offset: Offset = 0, residual: Optional[torch.Tensor] = None,
            device_offset: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + dropout(x, p), with autograd.  x and residual may have any shape (one
    and the same); elements are numbered row-major.  The offsets are ``dropout_fwd``'s."""
    _need_cuda(x, "x")
    if residual is not None:
        _need_cuda(residual, "residual")
    r = None if residual is None else residual.contiguous()
    if isinstance(offset, torch.Tensor) and device_offset is None:
        offset, device_offset = 0, offset
    return _Dropout.apply(x.contiguous(), r, _probability(p), int(seed), offset, device_offset)
