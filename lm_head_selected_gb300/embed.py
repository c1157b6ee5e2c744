"""PyTorch-facing wrappers of the token embedding (include/embedding.h).

Argument marshalling only; the computation runs in ``liblinear_logp.so``.
tokens are int64, the table [V, D] bf16, fp16 or fp32, contiguous, on a CUDA
device.  A token that equals ``ignore_index`` or lies outside [0, V) gives a
zero row and gets no gradient.  ("Feat/nemotron h lm head logprob cuda",
summary: untied embedding lookup with a sorted-segment deterministic
grad_weight; here the sums are fp32.)
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .ops import (
    IGNORE_INDEX,
    _dtype_code,
    _need,
    _need_cuda,
    _need_rows,
    _out,
    _raw_stream,
    _readable_rows,
    _workspace,
    on_tensor_device,
)


_FP32_MAX = torch.finfo(torch.float32).max


def _check_scale(scale: float):
    if not abs(scale) <= _FP32_MAX:
        raise ValueError(f"scale must be finite in fp32, got {scale}")


@on_tensor_device
def embedding_fwd(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0, ignore_index: int = IGNORE_INDEX,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * weight[tokens], [N, D] in the table's dtype (the product in fp32, rounded once)."""
    _need_cuda(weight, "weight")
    dev = weight.device
    code = _dtype_code(weight, "weight")
    _need(weight, "weight", weight.dtype, dev, 2)
    _need(tokens, "tokens", torch.int64, dev, 1)
    V, D = weight.shape
    if V < 1 or D < 1:
        raise ValueError(f"weight must have at least one row and one column, got {(V, D)}")
    _check_scale(scale)
    N = tokens.shape[0]
    out = _out(out, (N, D), weight.dtype, dev)
    st = _lib.load().embedding_fwd(tokens.data_ptr(), weight.data_ptr(), code, N, V, D, scale, ignore_index,
                                   out.data_ptr(), _raw_stream(dev.index))
    _lib.check("embedding_fwd", st)
    return out


@on_tensor_device
def embedding_bwd(grad_out: torch.Tensor, tokens: torch.Tensor, num_rows: int, scale: float = 1.0,
                  ignore_index: int = IGNORE_INDEX, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the table, [num_rows, D] in grad_out's dtype: row v is scale times the
    sum of the rows of grad_out whose token is v, in ascending order, in fp32.

    With ``accumulate`` the sums are added to ``out`` (required then), and rows that no
    token names are neither read nor written: the form for a table tied to the LM head,
    after ``linear_logp_bwd`` has written the head's gradient.  grad_out's rows may have
    any stride."""
    _need_cuda(grad_out, "grad_out")
    dev = grad_out.device
    code = _dtype_code(grad_out, "grad_out")
    stride = _need_rows(grad_out, "grad_out", dev)
    _need(tokens, "tokens", torch.int64, dev, 1)
    N, D = grad_out.shape
    V = int(num_rows)
    if tokens.shape[0] != N:
        raise ValueError("tokens must have one entry per row of grad_out")
    if V < 1 or D < 1:
        raise ValueError("the table must have at least one row and one column")
    _check_scale(scale)
    if accumulate and out is None:
        raise ValueError("accumulate adds to out: pass it")
    out = _out(out, (V, D), grad_out.dtype, dev)
    lib = _lib.load()
    ws = _workspace(lib.embedding_bwd_workspace_bytes(N, V, D), dev, workspace)
    st = lib.embedding_bwd(tokens.data_ptr(), grad_out.data_ptr(), stride, code, N, V, D, scale, ignore_index,
                           bool(accumulate), out.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev.index))
    _lib.check("embedding_bwd", st)
    return out


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, ignore_index):
        out = embedding_fwd(tokens, weight, scale, ignore_index)
        ctx.save_for_backward(tokens)
        ctx.rows, ctx.scale, ctx.ignore_index = weight.shape[0], scale, ignore_index
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        tokens, = ctx.saved_tensors
        return None, embedding_bwd(_readable_rows(grad_out), tokens, ctx.rows, ctx.scale, ctx.ignore_index), None, None


def embedding(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
              ignore_index: int = IGNORE_INDEX) -> torch.Tensor:
    """scale * weight[tokens] with autograd: tokens [...] int64, weight [V, D] -> [..., D]."""
    _need_cuda(weight, "weight")
    if not isinstance(tokens, torch.Tensor):
        raise TypeError("tokens must be a torch.Tensor")
    out = _Embedding.apply(tokens.reshape(-1).contiguous(), weight, float(scale), int(ignore_index))
    return out.reshape(*tokens.shape, weight.shape[1])
