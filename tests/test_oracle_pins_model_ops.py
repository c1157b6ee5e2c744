"""Pins of the FP64 oracle of the operators around the head (oracle/model_ops.py):
float64 torch compositions and their autograd, central differences, closed
forms, and the published known answers of Philox4x32-10."""
import math

import numpy as np
import pytest
import torch

from oracle import model_ops as mo


def test_embedding_against_torch_float64():
    rng = np.random.default_rng(1)
    V, D, N = 11, 5, 40
    w = rng.normal(size=(V, D))
    t = rng.integers(0, V, size=N)
    t[[3, 9]] = -100
    t[7], t[8] = V, -1
    g = rng.normal(size=(N, D))
    ok = torch.tensor((t >= 0) & (t < V))
    wt = torch.tensor(w, requires_grad=True)
    out = torch.where(ok[:, None], torch.nn.functional.embedding(torch.tensor(np.where(ok, t, 0)), wt) * 1.7, 0.0)
    (out * torch.tensor(g)).sum().backward()
    assert np.allclose(mo.embedding_forward(t, w, 1.7), out.detach().numpy(), atol=1e-14)
    assert np.allclose(mo.embedding_backward(g, t, V, 1.7), wt.grad.numpy(), atol=1e-13)
    base = rng.normal(size=(V, D))
    assert np.allclose(mo.embedding_backward(g, t, V, 1.7, base=base), base + wt.grad.numpy(), atol=1e-13)
    # a valid id as the ignore index
    assert np.all(mo.embedding_forward(t, w, 1.0, ignore_index=int(t[0]))[t == t[0]] == 0)


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_against_torch_float64(affine):
    rng = np.random.default_rng(2)
    N, D = 7, 13
    x, g = rng.normal(size=(N, D)) * 3 + 1, rng.normal(size=(N, D))
    w, b = (rng.normal(size=D), rng.normal(size=D)) if affine else (None, None)
    xt = torch.tensor(x, requires_grad=True)
    wt = torch.tensor(w if affine else np.ones(D), requires_grad=True)
    bt = torch.tensor(b if affine else np.zeros(D), requires_grad=True)
    y = torch.nn.functional.layer_norm(xt, (D,), wt, bt, 1e-3)
    (y * torch.tensor(g)).sum().backward()
    assert np.allclose(mo.layer_norm_forward(x, w, b, 1e-3)[0], y.detach().numpy(), atol=1e-12)
    gx, gw, gb = mo.layer_norm_backward(g, x, w, 1e-3)
    assert np.allclose(gx, xt.grad.numpy(), atol=1e-12)
    assert np.allclose(gw, wt.grad.numpy(), atol=1e-12)
    assert np.allclose(gb, bt.grad.numpy(), atol=1e-12)


def test_layer_norm_central_differences():
    rng = np.random.default_rng(3)
    x, g, w, b = (rng.normal(size=s) for s in ((3, 6), (3, 6), (6,), (6,)))
    loss = lambda x_, w_, b_: (g * mo.layer_norm_forward(x_, w_, b_)[0]).sum()  # noqa: E731
    got = mo.layer_norm_backward(g, x, w)
    for arr, grad, at in ((x, got[0], 0), (w, got[1], 1), (b, got[2], 2)):
        for i in np.ndindex(arr.shape):
            d = np.zeros_like(arr)
            d[i] = 1e-6
            args_p, args_m = [x, w, b], [x, w, b]
            args_p[at], args_m[at] = arr + d, arr - d
            assert abs((loss(*args_p) - loss(*args_m)) / 2e-6 - grad[i]) < 1e-7


def test_layer_norm_closed_forms():
    rng = np.random.default_rng(4)
    x, g = rng.normal(size=(4, 9)), rng.normal(size=(4, 9))
    y, mean, rstd = mo.layer_norm_forward(x, eps=0.0)
    assert np.allclose(y.sum(1), 0, atol=1e-12) and np.allclose((y * y).mean(1), 1, atol=1e-12)
    gx = mo.layer_norm_backward(g, x, eps=0.0)[0]
    assert np.allclose(gx.sum(1), 0, atol=1e-12) and np.allclose((gx * x).sum(1), 0, atol=1e-11)
    # a constant row: zero output, rstd = 1 / sqrt(eps)
    y, mean, rstd = mo.layer_norm_forward(np.full((1, 5), 3.0))
    assert np.all(y == 0) and mean[0] == 3.0 and math.isclose(rstd[0], 1 / math.sqrt(1e-5))


def test_philox_known_answers():
    """The published test vectors of Philox4x32-10."""
    cases = [
        ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
        ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
        ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
         (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
    ]
    for ctr, key, want in cases:
        assert tuple(int(v) for v in mo.philox4x32_10(np.array([ctr], dtype=np.uint64), key)[0]) == want


def test_dropout_mask_statistics_and_indexing():
    n = 1 << 20
    for p in (0.1, 0.5, 0.9):
        keep = mo.dropout_keep(n, p, seed=123, offset=7)
        sd = math.sqrt(p * (1 - p) / n)
        assert abs(keep.mean() - (1 - p)) < 6 * sd
    a = mo.dropout_keep(n, 0.5, 123, 7)
    for other in (mo.dropout_keep(n, 0.5, 123, 8), mo.dropout_keep(n, 0.5, 124, 7),
                  mo.dropout_keep(n, 0.5, 123 | 1 << 40, 7), mo.dropout_keep(n, 0.5, 123, 7 | 1 << 40)):
        assert abs((a == other).mean() - 0.5) < 6 * 0.5 / math.sqrt(n)
    # any window of the mask, also past 2^35 elements (block numbers past 32 bits)
    assert np.array_equal(mo.dropout_keep(1000, 0.5, 123, 7, first=13), a[13:1013])
    far = mo.dropout_keep(64, 0.5, 1, first=(1 << 35) * 8)
    assert not np.array_equal(far, mo.dropout_keep(64, 0.5, 1))


def test_dropout_values():
    x = np.arange(1.0, 33.0)
    keep = mo.dropout_keep(32, 0.25, 5, 1)
    y = mo.dropout_forward(x, 0.25, 5, 1)
    assert np.allclose(y[keep], x[keep] / 0.75) and np.all(y[~keep] == 0)
    assert np.allclose(mo.dropout_forward(x, 0.25, 5, 1, residual=-x), y - x)
    assert np.all(mo.dropout_forward(x, 0.0, 5) == x) and np.all(mo.dropout_forward(x, 1.0, 5) == 0)
