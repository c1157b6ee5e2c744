"""Pins of the FP64 oracle of the block operators: hand values, and gradients against differences."""
import math

import numpy as np
import pytest

from oracle import block_ops as bo


def test_activations_by_hand():
    z = np.array([0.0, 1.0, -2.0])
    assert np.allclose(bo.activation("silu", z)[0], [0.0, 1 / (1 + math.exp(-1)), -2 / (1 + math.exp(2))], rtol=1e-15)
    assert np.allclose(bo.activation("gelu", z)[0], [0.0, 0.8413447460685429, -2 * 0.022750131948179195], rtol=1e-12)
    assert np.allclose(bo.activation("gelu_tanh", z)[0], [0.0, 0.8411919906082768, -0.04540230591222749], rtol=1e-12)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradients_against_differences(act):
    rng = np.random.default_rng(1)
    args = [rng.normal(size=s) for s in ((3, 4), (5, 4), (5, 4))]
    gy = rng.normal(size=(3, 5))
    _, gate, up = bo.gated_forward(*args, act)
    grads = bo.gated_backward(gy, gate, up, *args, act)[:3]
    for k in range(3):
        for i in np.ndindex(args[k].shape):
            ends = []
            for h in (1e-6, -1e-6):
                moved = [a.copy() for a in args]
                moved[k][i] += h
                ends.append((bo.gated_forward(*moved, act)[0] * gy).sum())
            assert abs((ends[0] - ends[1]) / 2e-6 - grads[k][i]) < 1e-7


@pytest.mark.parametrize("gate_dim", [0, 1, 2])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_residual_gradients_against_differences(gate_dim, post, norm):
    rng = np.random.default_rng(2)
    N, D, scale = 3, 5, 0.7
    args = [rng.normal(size=(N, D)), rng.normal(size=(N, D)),
            None if gate_dim == 0 else rng.normal(size=(D,) if gate_dim == 1 else (N, D)),
            rng.normal(size=D) if post else None, rng.normal(size=D) if norm else None]
    gs, gh = rng.normal(size=(N, D)), rng.normal(size=(N, D))

    def total(a):
        s, h, _, _ = bo.residual_forward(*a, scale=scale)
        return (s * gs).sum() + (0.0 if h is None else (h * gh).sum())

    s, _, pr, r = bo.residual_forward(*args, scale=scale)
    grads = bo.residual_backward(gs, gh, s, *args[1:], pr, r, scale)
    for k in range(5):
        if args[k] is None:
            assert grads[k] is None
            continue
        for i in np.ndindex(args[k].shape):
            ends = []
            for h in (1e-6, -1e-6):
                moved = [None if a is None else a.copy() for a in args]
                moved[k][i] += h
                ends.append(total(moved))
            assert abs((ends[0] - ends[1]) / 2e-6 - grads[k][i]) < 1e-7


def test_adamw_by_hand():
    # first step from zero states: the update is the gradient's sign, up to eps
    p, m, v = bo.adamw(np.array([2.0, -1.0]), np.array([0.5, -0.25]), np.zeros(2), np.zeros(2), 1, 0.1, 0.9, 0.99, 0.0, 0.5)
    assert np.allclose(m, [0.05, -0.025]) and np.allclose(v, [0.0025, 0.000625])
    assert np.allclose(p, [2.0 * 0.95 - 0.1, -0.95 + 0.1], rtol=1e-12)
