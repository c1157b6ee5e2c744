"""PyTorch-facing wrappers of layer norm (include/layer_norm.h).

Argument marshalling only; the computation runs in ``liblinear_logp.so``.
x [N, D] is bf16, fp16 or fp32 on a CUDA device, with rows of any stride;
weight and bias [D] have x's dtype or fp32, and may each be left out.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .ops import _dtype_code, _need, _need_cuda, _need_rows, _out, _raw_stream, _readable_rows, _workspace, on_tensor_device

EPS = 1e-5


def _check_x(x: torch.Tensor):
    _need_cuda(x, "x")
    code = _dtype_code(x, "x")
    stride = _need_rows(x, "x", x.device)
    if x.shape[1] < 1:
        raise ValueError("x must have at least one column")
    return code, stride


def _check_param(t: Optional[torch.Tensor], name: str, x: torch.Tensor, other: Optional[torch.Tensor]):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or (t.dtype != x.dtype and t.dtype != torch.float32):
        raise TypeError(f"{name} must be a tensor of x's dtype or fp32")
    _need(t, name, t.dtype if other is None else other.dtype, x.device, 1)
    if t.shape[0] != x.shape[1]:
        raise ValueError(f"{name} must have {x.shape[1]} entries")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


@on_tensor_device
def layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   eps: float = EPS, out: Optional[torch.Tensor] = None):
    """(y [N, D] in x's dtype, mean [N] fp32, rstd [N] fp32)."""
    code, stride = _check_x(x)
    _check_param(weight, "weight", x, None)
    _check_param(bias, "bias", x, weight)
    dev = x.device
    N, D = x.shape
    param = weight if weight is not None else bias
    y = _out(out, (N, D), x.dtype, dev)
    mean = torch.empty(N, dtype=torch.float32, device=dev)
    rstd = torch.empty(N, dtype=torch.float32, device=dev)
    st = _lib.load().layer_norm_fwd(x.data_ptr(), stride, code, N, D, _ptr(weight), _ptr(bias),
                                    code if param is None else _dtype_code(param, "weight"), eps, y.data_ptr(),
                                    mean.data_ptr(), rstd.data_ptr(), _raw_stream(dev.index))
    _lib.check("layer_norm_fwd", st)
    return y, mean, rstd


@on_tensor_device
def layer_norm_bwd(grad_y: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   weight: Optional[torch.Tensor] = None, need_x: bool = True, need_weight: bool = True,
                   need_bias: bool = True, param_dtype: Optional[torch.dtype] = None,
                   workspace: Optional[torch.Tensor] = None):
    """(grad_x [N, D] in x's dtype, grad_weight [D], grad_bias [D]), None for those not
    needed.  The parameters' gradients have weight's dtype; without a weight,
    ``param_dtype`` (default x's)."""
    code, stride = _check_x(x)
    dev = x.device
    N, D = x.shape
    if not isinstance(grad_y, torch.Tensor) or grad_y.dtype != x.dtype or grad_y.shape != x.shape:
        raise ValueError("grad_y must have x's shape and dtype")
    gy_stride = _need_rows(grad_y, "grad_y", dev)
    for name, t in (("mean", mean), ("rstd", rstd)):
        _need(t, name, torch.float32, dev, 1)
        if t.shape[0] != N:
            raise ValueError(f"{name} must have N entries")
    _check_param(weight, "weight", x, None)
    pdt = weight.dtype if weight is not None else (param_dtype or x.dtype)
    if pdt not in (x.dtype, torch.float32) or (param_dtype is not None and param_dtype != pdt):
        raise TypeError("param_dtype must be weight's dtype, or x's dtype or fp32 without a weight")
    lib = _lib.load()
    gx = torch.empty((N, D), dtype=x.dtype, device=dev) if need_x else None
    gw = torch.empty(D, dtype=pdt, device=dev) if need_weight else None
    gb = torch.empty(D, dtype=pdt, device=dev) if need_bias else None
    ws = None
    if need_weight or need_bias:
        ws = _workspace(lib.layer_norm_bwd_workspace_bytes(N, D), dev, workspace)
    st = lib.layer_norm_bwd(grad_y.data_ptr(), gy_stride, x.data_ptr(), stride, code, N, D, mean.data_ptr(),
                            rstd.data_ptr(), _ptr(weight), code if pdt == x.dtype else 1, _ptr(gx), _ptr(gw),
                            _ptr(gb), _ptr(ws), 0 if ws is None else ws.numel(), _raw_stream(dev.index))
    _lib.check("layer_norm_bwd", st)
    return gx, gw, gb


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        param = weight if weight is not None else bias
        ctx.param_dtype = None if param is None else param.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        x, weight, mean, rstd = ctx.saved_tensors
        gx, gw, gb = layer_norm_bwd(_readable_rows(grad_y), x, mean, rstd, weight, *ctx.needs_input_grad[:3], ctx.param_dtype)
        return gx, gw, gb, None


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = EPS) -> torch.Tensor:
    """(x - mean) * rstd * weight + bias over the last dimension, with autograd: x [..., D]."""
    _need_cuda(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have at least one column")
    x2 = x.reshape(-1, x.shape[-1])
    return _LayerNorm.apply(_readable_rows(x2), weight, bias, float(eps)).reshape(x.shape)
