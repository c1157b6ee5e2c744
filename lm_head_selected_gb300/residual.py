"""PyTorch-facing wrappers of the RMS norms around a block (include/residual_rms_norm.h).

Argument marshalling only; the computation runs in ``liblinear_logp.so``.  Rows [N, D] are
bf16, fp16 or fp32 on a CUDA device, with rows of any stride; weights and a gate per column
[D] have the rows' dtype or, all of them, fp32.
"""
from __future__ import annotations

import math
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .norm import EPS, _ptr
from .ops import _dtype_code, _need, _need_cuda, _need_rows, _raw_stream, _readable_rows, _workspace, on_tensor_device

_NONE, _COLUMNS, _ROWS = 0, 1, 2


def _rows(t: Optional[torch.Tensor], name: str, like: torch.Tensor) -> int:
    """Row stride of an optional tensor of like's shape and dtype."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype != like.dtype or t.shape != like.shape:
        raise ValueError(f"{name} must have x's shape and dtype")
    if t.is_contiguous() and t.get_device() == like.get_device():
        return t.stride(0)
    return _need_rows(t, name, like.device)


def _column(t: torch.Tensor, name: str, x: torch.Tensor, D: int, dtype):
    """dtype, or t's where that is None, once t is known to be a [D] parameter of it."""
    if not isinstance(t, torch.Tensor) or (t.dtype != x.dtype and t.dtype != torch.float32):
        raise TypeError(f"{name} must be a tensor of x's dtype or fp32")
    dtype = dtype or t.dtype
    if t.dtype != dtype or t.dim() != 1 or not t.is_contiguous() or t.get_device() != x.get_device():
        _need(t, name, dtype, x.device, 1)
    if t.numel() != D:
        raise ValueError(f"{name} must have {D} entries")
    return dtype


def _check(x: torch.Tensor, branch, gate, post_weight, weight, scale: float):
    """(dtype code, parameters' dtype, its code, gate kind, row strides of x, branch and gate, N, D)."""
    _need_cuda(x, "x")
    code = _dtype_code(x, "x")
    stride = _need_rows(x, "x", x.device)
    N, D = x.shape
    if D < 1:
        raise ValueError("x must have at least one column")
    if branch is None:
        if gate is not None or post_weight is not None:
            raise ValueError("gate and post_weight need a branch")
        if weight is None:
            raise ValueError("a branch, a weight or both must be given")
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    b_stride = _rows(branch, "branch", x)
    kind, g_stride, dtype = _NONE, 0, None
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a torch.Tensor")
        if gate.dim() == 1:
            kind, dtype = _COLUMNS, _column(gate, "gate", x, D, None)
        else:
            kind, g_stride = _ROWS, _rows(gate, "gate", x)
    if post_weight is not None:
        dtype = _column(post_weight, "post_weight", x, D, dtype)
    if weight is not None:
        dtype = _column(weight, "weight", x, D, dtype)
    dtype = dtype or x.dtype
    return code, dtype, code if dtype == x.dtype else 1, kind, stride, b_stride, g_stride, N, D


@on_tensor_device
def residual_rms_norm_fwd(x: torch.Tensor, branch: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                          post_weight: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                          scale: float = 1.0, eps: float = EPS):
    """(s, h, post_rstd, rstd): s = x + scale * gate * (branch, normed and times post_weight where that
    is given), h = s normed, times weight; h and rstd are None without a weight, post_rstd without a
    post_weight, and s is x itself without a branch."""
    scale = float(scale)
    code, _, pcode, kind, xs, bs, gs, N, D = _check(x, branch, gate, post_weight, weight, scale)
    dev = x.device

    def rows():
        return torch.empty_like(x) if xs == D else torch.empty((N, D), dtype=x.dtype, device=dev)

    s = None if branch is None else rows()
    h = None if weight is None else rows()
    post_rstd = None if post_weight is None else torch.empty(N, dtype=torch.float32, device=dev)
    rstd = None if weight is None else torch.empty(N, dtype=torch.float32, device=dev)
    st = _lib.load().residual_rms_norm_fwd(x.data_ptr(), xs, _ptr(branch), bs, _ptr(gate), gs, kind, _ptr(post_weight),
                                           _ptr(weight), code, pcode, N, D, scale, eps, _ptr(s), _ptr(h),
                                           _ptr(post_rstd), _ptr(rstd), _raw_stream(dev.index))
    _lib.check("residual_rms_norm_fwd", st)
    return x if s is None else s, h, post_rstd, rstd


@on_tensor_device
def residual_rms_norm_bwd(grad_s: Optional[torch.Tensor], grad_h: Optional[torch.Tensor], s: torch.Tensor,
                          branch: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                          post_weight: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                          post_rstd: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                          scale: float = 1.0, need_x: bool = True, need_branch: bool = True, need_gate: bool = True,
                          need_post_weight: bool = True, need_weight: bool = True,
                          workspace: Optional[torch.Tensor] = None):
    """(grad_x, grad_branch, grad_gate, grad_post_weight, grad_weight), None for those not needed or
    whose input is None, from the forward's s (x itself without a branch) and statistics.  grad_s may be
    None; grad_h and rstd go with weight."""
    scale = float(scale)
    code, pdt, pcode, kind, ss, bs, gts, N, D = _check(s, branch, gate, post_weight, weight, scale)
    dev = s.device
    if (grad_h is None) != (weight is None) or (rstd is None) != (weight is None):
        raise ValueError("grad_h and rstd must be given with weight, and only then")
    if (post_rstd is None) != (post_weight is None):
        raise ValueError("post_rstd must be given with post_weight, and only then")
    if grad_s is None and grad_h is None:
        raise ValueError("grad_s, grad_h or both must be given")
    gs_stride, gh_stride = _rows(grad_s, "grad_s", s), _rows(grad_h, "grad_h", s)
    for name, t in (("post_rstd", post_rstd), ("rstd", rstd)):
        if t is not None:
            _need(t, name, torch.float32, dev, 1)
            if t.numel() != N:
                raise ValueError(f"{name} must have N entries")

    def rows(wanted):
        return torch.empty((N, D), dtype=s.dtype, device=dev) if wanted else None

    def column(wanted):
        return torch.empty(D, dtype=pdt, device=dev) if wanted else None

    gx, gb = rows(need_x), rows(need_branch and branch is not None)
    gg = rows(need_gate) if kind == _ROWS else column(need_gate and kind == _COLUMNS)
    gp, gw = column(need_post_weight and post_weight is not None), column(need_weight and weight is not None)
    lib = _lib.load()
    ws = _workspace(lib.residual_rms_norm_bwd_workspace_bytes(N, D), dev, workspace)
    st = lib.residual_rms_norm_bwd(_ptr(grad_s), gs_stride, _ptr(grad_h), gh_stride, s.data_ptr(), ss, _ptr(branch), bs,
                                   _ptr(gate), gts, kind, _ptr(post_weight), _ptr(weight), _ptr(post_rstd), _ptr(rstd),
                                   code, pcode, N, D, scale, _ptr(gx), _ptr(gb), _ptr(gg), _ptr(gp), _ptr(gw),
                                   ws.data_ptr(), ws.numel(), _raw_stream(dev.index))
    _lib.check("residual_rms_norm_bwd", st)
    return gx, gb, gg, gp, gw


class _ResidualRMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, branch, gate, post_weight, weight, scale, eps):
        s, h, post_rstd, rstd = residual_rms_norm_fwd(x, branch, gate, post_weight, weight, scale, eps)
        ctx.save_for_backward(s, branch, gate, post_weight, weight, post_rstd, rstd)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return (None if branch is None else s), h

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_s, grad_h):
        s, branch, gate, post_weight, weight, post_rstd, rstd = ctx.saved_tensors
        if grad_s is None and grad_h is None:
            return (None,) * 7
        if grad_h is None:  # nothing comes through the second norm
            weight = rstd = None
        grads = residual_rms_norm_bwd(None if grad_s is None else _readable_rows(grad_s),
                                      None if grad_h is None else _readable_rows(grad_h), s, branch, gate, post_weight,
                                      weight, post_rstd, rstd, ctx.scale, *ctx.needs_input_grad[:5])
        return (*grads, None, None)


def residual_rms_norm(x: torch.Tensor, branch: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                      post_weight: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                      scale: float = 1.0, eps: float = EPS):
    """The end of a block and the start of the next, with autograd: (s, h) with s = x + scale * gate *
    norm(branch), h = norm(s) * weight, over the last dimension of x [..., D].  The branch is normed
    where post_weight is given; h is None without a weight.  gate [D] or of x's shape.  Without a
    branch s is x, and h its RMS norm."""
    _need_cuda(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have at least one column")
    for name, t in (("branch", branch), ("gate", gate)):
        if t is not None:
            _need_cuda(t, name)
            if t.shape != x.shape and not (name == "gate" and t.dim() == 1):
                raise ValueError(f"{name} must have x's shape" + (" or be [D]" if name == "gate" else ""))

    def rows(t):
        return t if t is None else _readable_rows(t.reshape(-1, t.shape[-1]))

    wide_gate = gate is not None and not (gate.dim() == 1 and gate.shape[0] == x.shape[-1])
    s, h = _ResidualRMSNorm.apply(rows(x), rows(branch), rows(gate) if wide_gate else gate, post_weight, weight,
                                  float(scale), float(eps))
    return x if s is None else s.reshape(x.shape), None if h is None else h.reshape(x.shape)
