"""The gated linear layer on the GPU against its FP64 definition, at sizes no tile divides, in both types
and all activations; bounds from the arithmetic (fp32 sums on the tensor cores, one rounding)."""
import itertools

import numpy as np
import pytest
import torch

import lm_head_selected_gb300 as llp
from operator_bounds import UNIT, np64, rounded, within
from oracle import block_ops as bo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ACTS = ["silu", "gelu", "gelu_tanh"]
# fp32 sums of the tensor cores: at most one unit in the last place (2^-23) lost per addition, of at most
# as many additions as there are terms; the activation's own instructions (2^x, a quotient, erfc)
# stay below 2^-19 of its value, and below that of (1 + |z|) for the derivative
ADD, ACT = 2.0 ** -23, 2.0 ** -19


def inputs(N, D, F, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)

    return normal(N, D), normal(F, D, std=D ** -0.5), normal(F, D, std=D ** -0.5), normal(N, F)


def check_forward(y, pre, x, wg, wu, act):
    dt = y.dtype
    xn, gn, un = np64(x), np64(wg), np64(wu)
    ref, gate, up = bo.gated_forward(xn, gn, un, act)
    dg, du = (ADD * (xn.shape[1] + 4) * (np.abs(xn) @ np.abs(w).T) for w in (gn, un))
    a, _ = bo.activation(act, gate)
    # all three derivatives lie within (-0.2, 1.2)
    err = 1.2 * dg * (np.abs(up) + du) + (np.abs(a) * (1 + ACT)) * du + ACT * np.abs(ref)
    within("y", y, ref, rounded(ref, dt) + err * (1 + UNIT[dt]))
    if pre is not None:
        within("gate", pre[0], gate, rounded(gate, dt) + dg * (1 + UNIT[dt]))
        within("up", pre[1], up, rounded(up, dt) + du * (1 + UNIT[dt]))


def check_backward(grads, gy, pre, x, wg, wu, act):
    dt = x.dtype
    gyn, gate, up, xn, gn, un = (np64(t) for t in (gy, pre[0], pre[1], x, wg, wu))
    gx, gwg, gwu, dg, du = bo.gated_backward(gyn, gate, up, xn, gn, un, act)
    # dG and dU as the tensor cores take them: one rounding to the type, the activation's error
    eg = rounded(dg, dt) + ACT * (1 + np.abs(gate)) * np.abs(gyn * up)
    eu = rounded(du, dt) + ACT * np.abs(du)
    F, N = gn.shape[0], xn.shape[0]
    for name, got, ref, err, terms, depth in (
            ("grad_x", grads[0], gx, eg @ np.abs(gn) + eu @ np.abs(un), np.abs(dg) @ np.abs(gn) + np.abs(du) @ np.abs(un),
             2 * F),
            ("grad_w_gate", grads[1], gwg, eg.T @ np.abs(xn), np.abs(dg).T @ np.abs(xn), N),
            ("grad_w_up", grads[2], gwu, eu.T @ np.abs(xn), np.abs(du).T @ np.abs(xn), N)):
        if got is not None:
            within(name, got, ref, rounded(ref, dt) + (err + ADD * (depth + 4) * (terms + err)) * (1 + UNIT[dt]))


SIZES = [(1, 8, 8), (1, 64, 136), (2, 72, 64), (16, 128, 128), (31, 200, 1000), (32, 264, 520), (33, 512, 256),
         (127, 96, 264), (128, 1000, 136), (129, 64, 384), (257, 136, 72), (300, 320, 648), (1111, 72, 200)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,D,F", SIZES)
def test_forward_and_gradients(N, D, F, dtype):
    act = ACTS[(N + D + F) // 8 % 3]
    x, wg, wu, gy = inputs(N, D, F, dtype)
    y, pre = llp.gated_linear_fwd(x, wg, wu, act, keep=True)
    check_forward(y, pre, x, wg, wu, act)
    assert torch.equal(llp.gated_linear_fwd(x, wg, wu, act), y)  # kept or not
    grads = llp.gated_linear_bwd(gy, pre, x, wg, wu, act)
    check_backward(grads, gy, pre, x, wg, wu, act)
    assert llp.device_status() == 0


@pytest.mark.parametrize("act", ACTS)
def test_every_activation(act):
    x, wg, wu, gy = inputs(96, 64, 128, torch.bfloat16)
    x = x * torch.logspace(-3, 1.2, 96, device=DEV)[:, None].to(torch.bfloat16)  # projections far into both tails
    y, pre = llp.gated_linear_fwd(x, wg, wu, act, keep=True)
    check_forward(y, pre, x, wg, wu, act)
    check_backward(llp.gated_linear_bwd(gy, pre, x, wg, wu, act), gy, pre, x, wg, wu, act)


@pytest.mark.parametrize("act", ACTS)
def test_projections_far_outside(act):
    """Kept projections of up to 1e30: the derivative is 0 or 1 there, and the product finite."""
    z = torch.tensor([-1e30, -1e10, -300.0, -90.0, -20.0, 0.0, 20.0, 90.0, 300.0, 1e10, 1e30], dtype=torch.bfloat16)
    F = 16
    gate = torch.zeros(1, F, dtype=torch.bfloat16)
    gate[0, :11] = z
    pre = torch.stack([gate, torch.full_like(gate, 0.5)]).to(DEV)
    gy = torch.ones(1, F, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(1, 8, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(F, 8, dtype=torch.bfloat16, device=DEV)
    _, gg, gu = llp.gated_linear_bwd(gy, pre, x, w, w, act)
    slope = np.where(np64(gate[0]) > 10, 0.5, 0.0)  # up is 0.5
    far = np.abs(np64(gate[0])) >= 20
    assert np.allclose(np64(gg[:, 0])[far], slope[far], atol=1e-6)
    a = np.maximum(np64(gate[0]), 0.0)
    assert np.allclose(np64(gu[:, 0])[far], a[far], rtol=1e-6, atol=1e-6)


def test_subsets_of_the_gradients():
    x, wg, wu, gy = inputs(65, 72, 264, torch.bfloat16)
    _, pre = llp.gated_linear_fwd(x, wg, wu, keep=True)
    every = llp.gated_linear_bwd(gy, pre, x, wg, wu)
    for need in itertools.product([False, True], repeat=3):
        got = llp.gated_linear_bwd(gy, pre, x, wg, wu, "silu", *need)
        for n, a, b in zip(need, got, every):
            assert torch.equal(a, b) if n else a is None


def test_no_tokens():
    x, wg, wu, gy = inputs(0, 64, 128, torch.bfloat16)
    y, pre = llp.gated_linear_fwd(x, wg, wu, keep=True)
    assert y.shape == (0, 128) and pre.shape == (2, 0, 128)
    gx, gg, gu = llp.gated_linear_bwd(gy, pre, x, wg, wu)
    assert gx.shape == (0, 64) and not gg.any() and not gu.any() and gg.shape == gu.shape == (128, 64)


@pytest.mark.parametrize("N", [1, 7, 32, 64, 257])
def test_rows_do_not_depend_on_the_batch(N):
    """A row's result is the same in any batch: every sum runs over the same steps in the same order."""
    x, wg, wu, _ = inputs(400, 264, 520, torch.bfloat16)
    whole = llp.gated_linear_fwd(x, wg, wu)
    part = llp.gated_linear_fwd(x[100:100 + N], wg, wu)
    assert torch.equal(part, whole[100:100 + N])


def test_runs_are_the_same_and_the_workspace_may_hold_anything():
    from lm_head_selected_gb300 import _lib
    x, wg, wu, gy = inputs(1030, 200, 328, torch.float16)
    y, pre = llp.gated_linear_fwd(x, wg, wu, "gelu", keep=True)
    first = llp.gated_linear_bwd(gy, pre, x, wg, wu, "gelu")
    n = _lib.load().gated_linear_bwd_workspace_bytes(1030, 200, 328)
    for fill in (0xFF, 0x7F):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        again = llp.gated_linear_bwd(gy, pre, x, wg, wu, "gelu", workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert torch.equal(llp.gated_linear_fwd(x, wg, wu, "gelu"), y)


def test_nothing_is_written_past_the_outputs():
    N, D, F = 33, 72, 136
    x, wg, wu, gy = inputs(N, D, F, torch.bfloat16)
    room = torch.full((N * F + 4096,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = llp.gated_linear_fwd(x, wg, wu, out=room[:N * F].view(N, F))
    assert torch.equal(y, llp.gated_linear_fwd(x, wg, wu))
    assert (room[N * F:] == 7.0).all()


def test_weights_as_halves_of_one_tensor():
    D, F = 72, 136
    x, wg, wu, _ = inputs(40, D, F, torch.bfloat16)
    both = torch.cat([wg, wu])
    assert torch.equal(llp.gated_linear_fwd(x, both[:F], both[F:]), llp.gated_linear_fwd(x, wg, wu))


@pytest.mark.parametrize("N", [3, 40, 300])
@pytest.mark.parametrize("D,F", [(72, 136), (256, 8192), (256, 12288)])
def test_weights_anywhere(N, D, F):
    """The same weight twice, and the up projection's below the gate's in memory."""
    x, wg, wu, _ = inputs(N, D, F, torch.bfloat16)
    both = torch.cat([wu, wg])
    y, pre = llp.gated_linear_fwd(x, both[F:], both[:F], keep=True)
    want, want_pre = llp.gated_linear_fwd(x, wg, wu, keep=True)
    assert torch.equal(y, want) and torch.equal(pre, want_pre)
    y, pre = llp.gated_linear_fwd(x, wg, wg, keep=True)
    assert torch.equal(pre[0], pre[1]) and torch.equal(pre[0], want_pre[0])
    rows = slice(0, 3)
    check_forward(y[rows], pre[:, rows], x[rows], wg, wg, "silu")


@pytest.mark.parametrize("F", [64, 2048, 9728, 9736, 19464])
def test_rows_of_every_height_do_not_depend_on_the_batch(F):
    """Weights' rows spread over the SMs in boxes of 8 to 128."""
    x, wg, wu, _ = inputs(300, 192, F, torch.float16)
    whole, pre = llp.gated_linear_fwd(x, wg, wu, "gelu", keep=True)
    check_forward(whole[:4], pre[:, :4], x[:4], wg, wu, "gelu")
    for N in (1, 33, 128):
        y, p = llp.gated_linear_fwd(x[7:7 + N], wg, wu, "gelu", keep=True)
        assert torch.equal(y, whole[7:7 + N]) and torch.equal(p, pre[:, 7:7 + N])


def test_many_tokens():
    """Tickets, double K blocks and several waves of tiles; sampled rows and columns."""
    N, D, F = 9000, 512, 1160
    x, wg, wu, gy = inputs(N, D, F, torch.bfloat16, seed=5)
    y, pre = llp.gated_linear_fwd(x, wg, wu, keep=True)
    rows = torch.tensor([0, 255, 256, 4095, 8191, 8999], device=DEV)
    check_forward(y[rows], pre[:, rows], x[rows], wg, wu, "silu")
    gx, gg, gu = llp.gated_linear_bwd(gy, pre, x, wg, wu)
    check_backward((gx[rows], None, None), gy[rows], pre[:, rows], x[rows], wg, wu, "silu")
    cols = torch.tensor([0, 127, 128, 255, 256, 1024, 1151, 1159], device=DEV)
    check_backward((None, gg[cols], gu[cols]), gy[:, cols], pre[:, :, cols], x, wg[cols], wu[cols], "silu")


def test_autograd():
    x, wg, wu, gy = inputs(60, 64, 128, torch.bfloat16)
    ts = [t.clone().requires_grad_(True) for t in (x, wg, wu)]
    y = llp.gated_linear(ts[0].view(3, 20, 64), ts[1], ts[2], "gelu_tanh")
    assert y.shape == (3, 20, 128)
    y.backward(gy.view(3, 20, 128))
    _, pre = llp.gated_linear_fwd(x, wg, wu, "gelu_tanh", keep=True)
    for t, want in zip(ts, llp.gated_linear_bwd(gy, pre, x, wg, wu, "gelu_tanh")):
        assert torch.equal(t.grad, want)
    # an upstream gradient that is not contiguous, and only one tensor that asks
    w = wg.clone().requires_grad_(True)
    llp.gated_linear(x, w, wu).sum().backward()
    assert w.grad.shape == w.shape
    with torch.no_grad():
        assert torch.equal(llp.gated_linear(x, wg, wu, "gelu_tanh"), y.detach().view(60, 128))


def test_gradients_against_differences():
    """Of the function as computed, from both sides, along random directions: fp16 holds enough digits."""
    x, wg, wu, gy = inputs(24, 32, 64, torch.float16, seed=9)
    _, pre = llp.gated_linear_fwd(x, wg, wu, "silu", keep=True)
    grads = llp.gated_linear_bwd(gy, pre, x, wg, wu, "silu")
    g = torch.Generator().manual_seed(1)
    for k in range(3):
        v = torch.randn(grads[k].shape, generator=g, dtype=torch.float64).numpy()
        args = [np64(t) for t in (x, wg, wu)]
        ends = []
        for h in (1e-4, -1e-4):
            moved = list(args)
            moved[k] = args[k] + h * v
            ends.append((bo.gated_forward(*moved, "silu")[0] * np64(gy)).sum())
        want = (ends[0] - ends[1]) / 2e-4
        # each gradient is off by a few fp16 roundings of its terms, which add up like a random walk at worst linearly
        assert abs((np64(grads[k]) * v).sum() - want) <= 4 * UNIT[torch.float16] * (np.abs(np64(grads[k])) * np.abs(v)).sum() + 1e-3


def test_refusals():
    x, wg, wu, gy = inputs(8, 64, 128, torch.bfloat16)
    _, pre = llp.gated_linear_fwd(x, wg, wu, keep=True)
    for bad, error in ((lambda: llp.gated_linear_fwd(x.float(), wg.float(), wu.float()), TypeError),
                       (lambda: llp.gated_linear_fwd(x, wg.half(), wu), TypeError),
                       (lambda: llp.gated_linear_fwd(x, wg[:64], wu), ValueError),
                       (lambda: llp.gated_linear_fwd(x[:, :60].contiguous(), wg[:, :60].contiguous(), wu[:, :60].contiguous()), ValueError),
                       (lambda: llp.gated_linear_fwd(x, wg[:100].contiguous(), wu[:100].contiguous()), ValueError),
                       (lambda: llp.gated_linear_fwd(x.t(), wg, wu), ValueError),
                       (lambda: llp.gated_linear_fwd(x, wg, wu, "relu"), ValueError),
                       (lambda: llp.gated_linear_fwd(x, wg, wu, None), ValueError),
                       (lambda: llp.gated_linear_fwd(x, wg.cpu(), wu), ValueError),
                       (lambda: llp.gated_linear_bwd(gy[:4], pre, x, wg, wu), ValueError),
                       (lambda: llp.gated_linear_bwd(gy, pre[:1], x, wg, wu), ValueError),
                       (lambda: llp.gated_linear_bwd(gy, pre.float(), x, wg, wu), TypeError),
                       (lambda: llp.gated_linear_bwd(gy, pre, x, wg, wu, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)), ValueError)):
        with pytest.raises(error):
            bad()


@pytest.mark.parametrize("N", [1, 5, 300])
def test_weights_that_overlap(N):
    D, F = 64, 128
    x, flat, _, _ = inputs(N, D, 2 * F, torch.bfloat16)
    flat = flat.reshape(-1)
    for at in (8, D, 8 * D, F * D - 8, F * D):
        first, second = flat[:F * D].view(F, D), flat[at:at + F * D].view(F, D)
        for wg, wu in ((first, second), (second, first)):
            assert torch.equal(llp.gated_linear(x, wg, wu), llp.gated_linear(x, wg.clone(), wu.clone())), at


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,D,F", [(5000, 72, 200), (4999, 264, 520), (16391, 120, 360), (2049, 64, 8), (1537, 8, 64)])
def test_long_sums_of_few_tiles(N, D, F, dtype):
    """The weights' gradients in segments of the tokens: the same bits whichever is asked for, in every run and
    whatever the workspace holds."""
    from lm_head_selected_gb300 import _lib
    act = ACTS[N % 3]
    x, wg, wu, gy = inputs(N, D, F, dtype)
    _, pre = llp.gated_linear_fwd(x, wg, wu, act, keep=True)
    every = llp.gated_linear_bwd(gy, pre, x, wg, wu, act)
    check_backward(every, gy, pre, x, wg, wu, act)
    nbytes = _lib.load().gated_linear_bwd_workspace_bytes(N, D, F)
    ws = torch.full((nbytes + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    for need in itertools.product([False, True], repeat=3):
        got = llp.gated_linear_bwd(gy, pre, x, wg, wu, act, *need, workspace=ws[:nbytes])
        for n, a, b in zip(need, got, every):
            assert torch.equal(a, b) if n else a is None
    assert bool((ws[nbytes:] == 0xFF).all())
    assert llp.device_status() == 0
