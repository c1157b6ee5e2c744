"""FP64 CPU oracle for the operators around the LM head: token embedding, layer
norm, dropout.

TEST INFRASTRUCTURE ONLY (same rules as ``oracle/linear_logp.py``).  NumPy
float64 throughout, element by element from the definitions:

* embedding: out[n] = s * W[t_n], grad_W[v] = s * sum of grad_out[n] over t_n = v;
  an invalid token (the ignore index, or outside [0, V)) gives a zero row and
  no gradient;
* layer norm: h = (x - mean) / sqrt(var + eps) with the biased variance,
  y = h * w + b, and its gradients;
* dropout: element e is kept when its 16-bit lane of the Philox4x32-10 block
  e // 8 reaches T = floor(p * 65536 + 1/2); kept values are scaled by
  65536 / (65536 - T).

Pins: ``tests/test_oracle_pins_model_ops.py``.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import numpy as np


def embedding_forward(tokens: np.ndarray, weight: np.ndarray, scale: float = 1.0,
                      ignore_index: int = -100) -> np.ndarray:
    out = np.zeros((len(tokens), weight.shape[1]))
    for n, t in enumerate(tokens):
        if t != ignore_index and 0 <= t < weight.shape[0]:
            out[n] = scale * weight[t]
    return out


def embedding_backward(grad_out: np.ndarray, tokens: np.ndarray, V: int, scale: float = 1.0,
                       ignore_index: int = -100, base: Optional[np.ndarray] = None) -> np.ndarray:
    gw = np.zeros((V, grad_out.shape[1])) if base is None else base.astype(np.float64).copy()
    for n, t in enumerate(tokens):
        if t != ignore_index and 0 <= t < V:
            gw[t] += scale * grad_out[n]
    return gw


def layer_norm_forward(x: np.ndarray, weight: Optional[np.ndarray] = None, bias: Optional[np.ndarray] = None,
                       eps: float = 1e-5) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    mean = x.sum(axis=1) / x.shape[1]
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).sum(axis=1) / x.shape[1] + eps)
    h = c * rstd[:, None]
    y = h if weight is None else h * weight
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_backward(grad_y: np.ndarray, x: np.ndarray, weight: Optional[np.ndarray] = None,
                        eps: float = 1e-5) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    D = x.shape[1]
    _, mean, rstd = layer_norm_forward(x, eps=eps)
    h = (x - mean[:, None]) * rstd[:, None]
    a = grad_y if weight is None else grad_y * weight
    gx = rstd[:, None] * (a - (a.sum(axis=1) / D)[:, None] - h * ((a * h).sum(axis=1) / D)[:, None])
    return gx, (grad_y * h).sum(axis=0), grad_y.sum(axis=0)


def philox4x32_10(counter: np.ndarray, key: Tuple[int, int]) -> np.ndarray:
    """Blocks of four 32-bit words: counter [n, 4], key two words ("Parallel random numbers: as
    easy as 1, 2, 3", Salmon et al. 2011, Philox4x32 with ten rounds)."""
    lo = np.uint64(0xFFFFFFFF)
    c = [counter[:, i].astype(np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & lo, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & lo]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, axis=1).astype(np.uint32)


def dropout_keep(count: int, p: float, seed: int, offset: int = 0, first: int = 0) -> np.ndarray:
    """Whether elements first .. first + count - 1 are kept."""
    b0 = first // 8
    block = np.arange(b0, (first + count + 7) // 8, dtype=np.uint64)
    lo, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    ctr = np.stack([block & lo, block >> sh, np.full_like(block, offset & 0xFFFFFFFF),
                    np.full_like(block, (offset >> 32) & 0xFFFFFFFF)], axis=1)
    w = philox4x32_10(ctr, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    lanes = np.stack([w & np.uint32(0xFFFF), w >> np.uint32(16)], axis=2).reshape(-1)
    return lanes[first - 8 * b0: first - 8 * b0 + count].astype(np.int64) >= math.floor(p * 65536 + 0.5)


def dropout_forward(x: np.ndarray, p: float, seed: int, offset: int = 0,
                    residual: Optional[np.ndarray] = None) -> np.ndarray:
    T = math.floor(p * 65536 + 0.5)
    keep = dropout_keep(x.size, p, seed, offset).reshape(x.shape)
    y = np.zeros(x.shape)
    if T < 65536:
        y[keep] = x[keep] * (65536.0 / (65536 - T))
    return y if residual is None else y + residual
