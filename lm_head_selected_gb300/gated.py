"""PyTorch-facing wrappers of the gated linear layer (include/gated_linear.h).

Argument marshalling only; the computation runs in ``liblinear_logp.so``.  x [N, D]
and the weights [F, D] are all bf16 or all fp16, contiguous, on a CUDA device, with D
and F multiples of 8.  Every tensor starts on a 16-byte boundary; ``gated_linear`` copies an
input, or a gradient that autograd brings, which does not.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .ops import _need, _need_cuda, _out, _raw_stream, _workspace, on_tensor_device

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


def _activation(name: str) -> int:
    code = ACTIVATIONS.get(name) if isinstance(name, str) else None
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return code


def _finish(fn: str, status: int, **tensors) -> None:
    if status == _lib.LLP_ERR_MISALIGNED:
        for name, t in tensors.items():
            if t is not None and t.data_ptr() % 16:
                raise ValueError(f"{name} must start on a 16-byte boundary")
    _lib.check(fn, status)


def _movable(t: torch.Tensor) -> torch.Tensor:
    """The tensor, contiguous and on a 16-byte boundary: itself, or a copy."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _check(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor) -> int:
    _need_cuda(x, "x")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x must be bf16 or fp16, got {x.dtype}")
    dev = x.device
    _need(x, "x", x.dtype, dev, 2)
    _need(w_gate, "w_gate", x.dtype, dev, 2)
    _need(w_up, "w_up", x.dtype, dev, 2)
    D, F = x.shape[1], w_gate.shape[0]
    if w_gate.shape[1] != D or w_up.shape != w_gate.shape:
        raise ValueError(f"w_gate and w_up must both be [F, {D}], got {tuple(w_gate.shape)} and {tuple(w_up.shape)}")
    if D < 8 or F < 8 or D % 8 or F % 8:
        raise ValueError(f"D and F must be multiples of 8, got {D} and {F}")
    return 0 if x.dtype == torch.bfloat16 else 2


@on_tensor_device
def gated_linear_fwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu",
                     keep: bool = False, out: Optional[torch.Tensor] = None):
    """y [N, F] = act(x w_gate^T) * (x w_up^T); with ``keep``, (y, pre): pre [2, N, F], the two
    projections, for ``gated_linear_bwd``."""
    code = _check(x, w_gate, w_up)
    act = _activation(activation)
    dev = x.device
    N, D = x.shape
    F = w_gate.shape[0]
    y = _out(out, (N, F), x.dtype, dev)
    pre = torch.empty((2, N, F), dtype=x.dtype, device=dev) if keep else None
    st = _lib.load().gated_linear_fwd(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), code, act, N, D, F,
                                      y.data_ptr(), None if pre is None else pre.data_ptr(), _raw_stream(dev.index))
    _finish("gated_linear_fwd", st, x=x, w_gate=w_gate, w_up=w_up, out=out)
    return (y, pre) if keep else y


@on_tensor_device
def gated_linear_bwd(grad_y: torch.Tensor, pre: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor,
                     w_up: torch.Tensor, activation: str = "silu", need_x: bool = True, need_gate: bool = True,
                     need_up: bool = True, workspace: Optional[torch.Tensor] = None):
    """(grad_x, grad_w_gate, grad_w_up) in x's dtype, None for those not needed, from the
    projections that ``gated_linear_fwd(..., keep=True)`` gave."""
    code = _check(x, w_gate, w_up)
    act = _activation(activation)
    dev = x.device
    N, D = x.shape
    F = w_gate.shape[0]
    _need(grad_y, "grad_y", x.dtype, dev, 2)
    _need(pre, "pre", x.dtype, dev, 3)
    if tuple(grad_y.shape) != (N, F) or tuple(pre.shape) != (2, N, F):
        raise ValueError(f"grad_y must be [{N}, {F}] and pre [2, {N}, {F}]")
    lib = _lib.load()
    gx = torch.empty((N, D), dtype=x.dtype, device=dev) if need_x else None
    gg = torch.empty((F, D), dtype=x.dtype, device=dev) if need_gate else None
    gu = torch.empty((F, D), dtype=x.dtype, device=dev) if need_up else None
    ws = _workspace(lib.gated_linear_bwd_workspace_bytes(N, D, F), dev, workspace)
    st = lib.gated_linear_bwd(grad_y.data_ptr(), pre.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
                              code, act, N, D, F, *(None if t is None else t.data_ptr() for t in (gx, gg, gu)),
                              ws.data_ptr(), ws.numel(), _raw_stream(dev.index))
    _finish("gated_linear_bwd", st, grad_y=grad_y, pre=pre, x=x, w_gate=w_gate, w_up=w_up)
    return gx, gg, gu


class _GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation, keep):
        ctx.activation = activation
        if not keep:
            return gated_linear_fwd(x, w_gate, w_up, activation)
        y, pre = gated_linear_fwd(x, w_gate, w_up, activation, keep=True)
        ctx.save_for_backward(x, w_gate, w_up, pre)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x, w_gate, w_up, pre = ctx.saved_tensors
        return (*gated_linear_bwd(_movable(grad_y), pre, x, w_gate, w_up, ctx.activation,
                                  *ctx.needs_input_grad[:3]), None, None)


def gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu") -> torch.Tensor:
    """act(x w_gate^T) * (x w_up^T) over the last dimension, with autograd: x [..., D] -> [..., F].
    Where a gradient is wanted, both projections [2, N, F] are kept for it.  The weights must start on a
    16-byte boundary; an x that does not is copied."""
    _need_cuda(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have at least one column")
    _need_cuda(w_gate, "w_gate")
    _need_cuda(w_up, "w_up")
    keep = torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad)
    x2 = _movable(x.reshape(-1, x.shape[-1]))
    return _GatedLinear.apply(x2, w_gate, w_up, activation, keep).reshape(*x.shape[:-1], w_gate.shape[0])
