"""FP64 definitions of the operators of a model's blocks and their optimizer (gated linear layer, RMS
norms around a block, AdamW), from the formulas alone; shares no code with the GPU path."""
import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _logistic(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def activation(name, z):
    """(act(z), act'(z))."""
    if name == "silu":
        s = _logistic(z)
        return z * s, s + z * s * (1.0 - s)
    if name == "gelu":
        phi = 0.5 * _erfc(-z / math.sqrt(2.0))
        return z * phi, phi + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    t = np.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)


def gated_forward(x, wg, wu, act):
    """(y, gate, up)."""
    gate, up = x @ wg.T, x @ wu.T
    return activation(act, gate)[0] * up, gate, up


def gated_backward(gy, gate, up, x, wg, wu, act):
    """(grad_x, grad_wg, grad_wu, dG, dU)."""
    a, slope = activation(act, gate)
    dg, du = gy * up * slope, gy * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du


def residual_forward(x, branch=None, gate=None, post_weight=None, weight=None, scale=1.0, eps=1e-5):
    """(s, h, post_rstd, rstd)."""
    s, post_rstd = x, None
    if branch is not None:
        m = branch
        if post_weight is not None:
            post_rstd = 1.0 / np.sqrt((branch ** 2).mean(1) + eps)
            m = branch * post_rstd[:, None] * post_weight
        s = x + scale * (m if gate is None else gate * m)
    if weight is None:
        return s, None, post_rstd, None
    rstd = 1.0 / np.sqrt((s ** 2).mean(1) + eps)
    return s, s * rstd[:, None] * weight, post_rstd, rstd


def residual_backward(gs, gh, s, branch=None, gate=None, post_weight=None, weight=None, post_rstd=None, rstd=None,
                      scale=1.0):
    """(grad_x, grad_branch, grad_gate, grad_post_weight, grad_weight), statistics taken as given."""
    G = np.zeros_like(s) if gs is None else gs
    g_weight = None
    if weight is not None:
        c, a = s * rstd[:, None], gh * weight
        g_weight = (gh * c).sum(0)
        G = G + rstd[:, None] * (a - c * (a * c).mean(1, keepdims=True))
    if branch is None:
        return G, None, None, None, g_weight
    k = branch if post_weight is None else branch * post_rstd[:, None]
    m = k if post_weight is None else k * post_weight
    g_gate = None
    if gate is not None:
        g_gate = scale * G * m
        g_gate = g_gate.sum(0) if gate.ndim == 1 else g_gate
    e = scale * G * (1.0 if gate is None else gate)
    if post_weight is None:
        return G, e, g_gate, None, g_weight
    g_post = (e * k).sum(0)
    e = e * post_weight
    return G, post_rstd[:, None] * (e - k * (e * k).mean(1, keepdims=True)), g_gate, g_post, g_weight


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay):
    """(parameter, first moment, second moment) after the step."""
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    with np.errstate(invalid="ignore", divide="ignore"):
        update = m / (1.0 - beta1 ** step) / (np.sqrt(v / (1.0 - beta2 ** step)) + eps)
    return p * (1.0 - lr * decay) - lr * update, m, v
