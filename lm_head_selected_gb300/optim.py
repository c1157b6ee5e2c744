"""PyTorch-facing wrappers of the AdamW step (include/adamw.h).

Argument marshalling only; the computation runs in ``liblinear_logp.so``: one launch for
up to 320 tensors, with nothing copied to the device.
"""
from __future__ import annotations

import array
import math
import operator
from itertools import chain, compress
from typing import List, Optional, Sequence, Tuple, Union

import torch

from . import _lib
from .ops import _DTYPE_CODES, _need_cuda, _raw_stream

BLOCK = 256  # elements of a tensor that share a scale of the 8-bit states
CODE = torch.float8_e4m3fn

Tensors = Sequence[torch.Tensor]


def adamw_state(params: Tensors, bits: int = 32, masters: bool = False) -> dict:
    """Zero states for ``adamw_step(params, grads, **state, ...)``: exp_avg and exp_avg_sq in fp32, or with
    ``bits=8`` as e4m3 codes with their scales, exp_avg_scale and exp_avg_sq_scale; with ``masters``, an fp32
    copy of every parameter that is not fp32 itself."""
    if bits not in (32, 8):
        raise ValueError(f"bits must be 32 or 8, got {bits}")
    params = list(params)
    for i, p in enumerate(params):
        _need_cuda(p, f"params[{i}]")

    def zeros(dtype, size):
        return [torch.zeros(size(p), dtype=dtype, device=p.device) for p in params]

    whole, blocks = (lambda p: p.shape), (lambda p: -(-p.numel() // BLOCK))
    state = {"exp_avg": zeros(torch.float32 if bits == 32 else CODE, whole),
             "exp_avg_sq": zeros(torch.float32 if bits == 32 else CODE, whole)}
    if bits == 8:
        state["exp_avg_scale"] = zeros(torch.float32, blocks)
        state["exp_avg_sq_scale"] = zeros(torch.float32, blocks)
    if masters:
        state["masters"] = [None if p.dtype == torch.float32 else p.detach().float().contiguous() for p in params]
    return state


def _scalar(t, name: str, dtype: torch.dtype, device: torch.device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() != 1 or t.device != device:
        raise ValueError(f"{name} must be one {dtype} value on the parameters' device")
    return t.data_ptr()


# Over a list at once, without a step of the interpreter for each tensor (41 -> 33 us of host time for a
# step over 12 tensors).
_numel, _data_ptr = torch.Tensor.numel, torch.Tensor.data_ptr
_device_of, _contiguous, _dtype = torch.Tensor.get_device, torch.Tensor.is_contiguous, operator.attrgetter("dtype")
_shape = operator.attrgetter("shape")


def _alike(tensors: list, sizes: List[int], index: int, dtype: torch.dtype) -> bool:
    """Whether all of them are contiguous tensors of dtype and of these sizes on one device."""
    try:
        return (list(map(_numel, tensors)) == sizes and list(map(_dtype, tensors)).count(dtype) == len(sizes) and
                list(map(_device_of, tensors)).count(index) == len(sizes) and all(map(_contiguous, tensors)))
    except (TypeError, AttributeError):  # no tensors
        return False


def _codes(params: list, grads: list, index: int):
    """The dtype codes of the parameters and of the gradients, and the parameters' sizes, after their checks."""
    try:
        p_code = list(map(_DTYPE_CODES.__getitem__, map(_dtype, params)))
        g_code = list(map(_DTYPE_CODES.__getitem__, map(_dtype, grads)))
        n = len(params)
        if ((p_code == g_code or g_code.count(1) == n or all(g == c or g == 1 for c, g in zip(p_code, g_code))) and
                list(map(_shape, params)) == list(map(_shape, grads)) and
                list(map(_device_of, params)).count(index) == list(map(_device_of, grads)).count(index) == n and
                all(map(_contiguous, params)) and all(map(_contiguous, grads))):
            return p_code, g_code, list(map(_numel, params))
    except (TypeError, AttributeError, KeyError):
        pass
    for i, (p, g) in enumerate(zip(params, grads)):  # one of them will not do
        if not isinstance(p, torch.Tensor) or not isinstance(g, torch.Tensor):
            raise TypeError(f"params[{i}] and grads[{i}] must be tensors")
        code, g_c = _DTYPE_CODES.get(p.dtype), _DTYPE_CODES.get(g.dtype)
        if code is None or (g_c != code and g_c != 1):
            raise TypeError(f"params[{i}] must be bf16, fp16 or fp32, grads[{i}] of the same dtype or fp32")
        if p.get_device() != index or g.get_device() != index or not p.is_contiguous() or not g.is_contiguous():
            raise ValueError(f"params[{i}] and grads[{i}] must be contiguous, on cuda:{index}")
        if g.shape != p.shape:
            raise ValueError(f"grads[{i}] must have the shape of params[{i}]")
    raise ValueError("params and grads must be tensors")


def _need_all(name: str, tensors, sizes: List[int], index: int, dtype: torch.dtype) -> List[torch.Tensor]:
    """The tensors, once they are known to be contiguous ones of dtype and of these sizes on one device."""
    tensors = list(tensors)
    if _alike(tensors, sizes, index, dtype):
        return tensors
    if len(tensors) != len(sizes):
        raise ValueError(f"{name} must have {len(sizes)} entries, got {len(tensors)}")
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype:
            raise TypeError(f"{name}[{i}] must be a tensor of {dtype}")
        if t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous, on cuda:{index}")
        if t.numel() != sizes[i]:
            raise ValueError(f"{name}[{i}] has {t.numel()} elements, which does not go with params[{i}]")
    return tensors


def adamw_step(params: Tensors, grads: Tensors, exp_avg: Tensors, exp_avg_sq: Tensors, step: int, lr: float = 1e-3,
               betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8,
               weight_decay: Union[float, Sequence[float]] = 0.01, masters: Optional[Sequence] = None,
               exp_avg_scale: Optional[Tensors] = None, exp_avg_sq_scale: Optional[Tensors] = None,
               device_step: Optional[torch.Tensor] = None, device_lr: Optional[torch.Tensor] = None,
               grad_scale: Optional[torch.Tensor] = None) -> None:
    """One AdamW step, in place, over all tensors (bf16, fp16 or fp32, each its own; gradients of the same
    dtype or fp32; contiguous, on one CUDA device).  None may be listed twice, no gradient be a parameter or a
    state too: that is refused.  Nor may what is written overlap anything else in part, which is not looked for.
    ``step`` counts from 1 (with device_step, their sum does).  States as ``adamw_state`` makes them, in 8 bits
    where the scales are given.  ``weight_decay``: one value, or one per tensor.  On the device, read when the
    kernel runs, so that a captured graph can advance them: ``device_step`` (int64, added to step), ``device_lr``
    and ``grad_scale`` (fp32, factors of lr and of the gradients)."""
    params, grads = list(params), list(grads)
    count = len(params)
    if len(grads) != count:
        raise ValueError(f"grads must have {count} entries, got {len(grads)}")
    if (exp_avg_scale is None) != (exp_avg_sq_scale is None):
        raise ValueError("exp_avg_scale and exp_avg_sq_scale must be given together")
    beta1, beta2 = float(betas[0]), float(betas[1])
    if not (0.0 <= beta1 < 1.0 and 0.0 <= beta2 < 1.0):
        raise ValueError(f"betas must lie in [0, 1), got {betas}")
    lr, eps, step = float(lr), float(eps), int(step)
    if not math.isfinite(lr) or not math.isfinite(eps) or eps < 0.0:
        raise ValueError("lr and eps must be finite, eps not negative")
    if step < (1 if device_step is None else 0):
        raise ValueError("step counts from 1")
    if count == 0:
        return
    _need_cuda(params[0], "params[0]")
    device = params[0].device
    index = device.index
    p_code, g_code, sizes = _codes(params, grads, index)
    packed = exp_avg_scale is not None
    dtype = CODE if packed else torch.float32
    # one array for all addresses and the sizes: a list after the other, `count` entries each
    lists = [params, grads, _need_all("exp_avg", exp_avg, sizes, index, dtype),
             _need_all("exp_avg_sq", exp_avg_sq, sizes, index, dtype)]
    if packed:
        blocks = [-(-n // BLOCK) for n in sizes]
        lists += [_need_all(name, t, blocks, index, torch.float32) for name, t in
                  (("exp_avg_scale", exp_avg_scale), ("exp_avg_sq_scale", exp_avg_sq_scale))]
    words = [a for t in lists for a in map(_data_ptr, t)]
    if masters is not None:
        masters = list(masters)
        if len(masters) != count:
            raise ValueError(f"masters must have {count} entries, got {len(masters)}")
        there = [t is not None for t in masters]
        _need_all("masters", compress(masters, there), list(compress(sizes, there)), index, torch.float32)
        at = map(_data_ptr, compress(masters, there))
        words += [next(at) if b else 0 for b in there]
    # what is written must be somewhere of its own
    written, read = words[:count] + words[2 * count:], words[count:2 * count]
    places, none = set(written), written.count(0)  # tensors without elements, masters that are not there
    if len(places) != len(written) - max(none - 1, 0) or not places.isdisjoint(read):
        written = [a for a, n in zip(written, sizes * (len(words) // count)) if n and a]
        places = set(written)
        if len(places) != len(written):
            raise ValueError("a parameter or a state is listed twice")
        if not places.isdisjoint(a for a, n in zip(read, sizes) if n):
            raise ValueError("a gradient is a parameter or a state too")
    words = array.array("q", words + sizes)
    codes = array.array("i", p_code + g_code)
    one = isinstance(weight_decay, (int, float))
    decay = array.array("d", [weight_decay] * count if one else weight_decay)
    if len(decay) != count or not (math.isfinite(sum(decay)) or all(map(math.isfinite, decay))):
        raise ValueError(f"weight_decay must be finite, one value or {count}")
    scalars = (None, None, None)
    if device_step is not None or device_lr is not None or grad_scale is not None:
        scalars = (_scalar(device_step, "device_step", torch.int64, device),
                   _scalar(device_lr, "device_lr", torch.float32, device),
                   _scalar(grad_scale, "grad_scale", torch.float32, device))
    at, code_at, row = words.buffer_info()[0], codes.buffer_info()[0], 8 * count
    n_lists = len(lists)
    scale_at = (at + 4 * row, at + 5 * row) if packed else (None, None)
    master_at = None if masters is None else at + n_lists * row
    size_at = at + (n_lists + (masters is not None)) * row

    def call():
        st = _lib.load().adamw_step(count, at, at + row, at + 2 * row, at + 3 * row, *scale_at, master_at, size_at,
                                    code_at, code_at + 4 * count, decay.buffer_info()[0], 8 if packed else 32, lr,
                                    beta1, beta2, eps, step, *scalars, _raw_stream(index))
        _lib.check("adamw_step", st)

    if index == torch._C._cuda_getDevice():
        call()
    else:
        with torch.cuda.device(device):
            call()
    # autograd learns that they have changed
    changed = list(chain(params, *lists[2:]))
    if masters is not None:
        changed += compress(masters, there)
    try:
        torch.autograd.graph.increment_version(changed)
    except RuntimeError:  # tensors made under inference mode have no version to count
        torch.autograd.graph.increment_version([t for t in changed if not t.is_inference()])
