"""AdamW late in a schedule: a decay of about fp32's step at 1, whose factor 1 - rate * decay has few digits."""
import numpy as np
import pytest
import torch

import lm_head_selected_gb300 as llp
from operator_bounds import U32, np64
from oracle import block_ops as bo
from test_gpu_adamw import filled, start, tensors

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("masters", [False, True])
@pytest.mark.parametrize("lr,decay", [(1e-6, 0.1), (1e-5, 0.01), (1e-6, 0.01), (2e-6, 0.3)])
@pytest.mark.parametrize("shift", [0, 1])
def test_one_step_rounds_the_parameter_once(lr, decay, masters, bits, shift):
    """The parameter's rounding is half a step of fp32 (U32 of its value); decay and update, a millionth of it, carry
    their own few."""
    sizes = [70001, 256]
    pdt = torch.bfloat16 if masters else torch.float32
    params, grads = tensors(sizes, pdt, torch.float32)
    state = filled(llp.adamw_state(params, bits, masters), grads)

    def moved(t):
        room = torch.empty(t.numel() + 64, dtype=t.dtype, device=DEV)
        return room[shift:shift + t.numel()].copy_(t)

    if shift:  # off the vectors' boundaries
        params, grads = [moved(t) for t in params], [moved(t) for t in grads]
        state = {k: [moved(t) for t in v] for k, v in state.items()}
    before = start(params, grads, state)
    betas, eps, step = (0.9, 0.95), 1e-8, 50
    llp.adamw_step(params, grads, **state, step=step, lr=lr, betas=betas, eps=eps, weight_decay=decay)
    for i, (p0, g, m0, v0) in enumerate(before):
        p, m, v = bo.adamw(p0, g, m0, v0, step, lr, *betas, eps, decay)
        root = np.sqrt(v / (1 - betas[1] ** step)) + eps
        upd = lr * np.abs(m / (1 - betas[0] ** step)) / root
        em = 8 * U32 * (np.abs(m0) + np.abs(g)) + 1e-44
        small = 2.0 ** -19 * upd + lr * em / (1 - betas[0] ** step) / root + 8 * U32 * lr * decay * np.abs(p0)
        got = np64(state["masters"][i] if masters else params[i])
        err = np.abs(got - p)
        assert (err <= U32 * np.abs(p) + 1.01 * small).all(), np.max((err - small) / (U32 * np.abs(p)))


@pytest.mark.parametrize("lr,decay", [(1e-6, 0.1), (1e-6, 0.01)])
def test_the_decay_of_many_steps(lr, decay):
    """The mean over elements whose roundings the updates keep apart: n of them over k steps of errors of up to
    half a step, 2^-24 for values in [1, 2): sqrt(k / (3 n)) 2^-24, five times that allowed."""
    n, steps = 1 << 16, 100
    g = torch.Generator().manual_seed(5)
    params = [(1 + torch.rand(n, generator=g) * 0.99).to(DEV)]
    state = llp.adamw_state(params)
    state["exp_avg"][0].copy_(torch.randn(n, generator=g) * 0.3)
    state["exp_avg_sq"][0].copy_((0.5 + torch.rand(n, generator=g)) ** 2)
    p, m, v = np64(params[0]), np64(state["exp_avg"][0]), np64(state["exp_avg_sq"][0])
    for step in range(50, 50 + steps):
        grads = [torch.randn(n, generator=g).to(DEV)]
        llp.adamw_step(params, grads, **state, step=step, lr=lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=decay)
        p, m, v = bo.adamw(p, np64(grads[0]), m, v, step, lr, 0.9, 0.95, 1e-8, decay)
    drift = (np64(params[0]) - p).mean()
    # updates are within 2^-19 of their size, at most about lr each
    assert abs(drift) <= 5 * 2.0 ** -24 * (steps / (3 * n)) ** 0.5 + steps * lr * 2.0 ** -19, drift / (steps * lr * decay)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_an_infinite_parameter_stays_infinite(bits, decay):
    """p (1 - rate decay) of an infinite p is infinite; others of its block are as without it."""
    params, grads = tensors([600], torch.float32, torch.float32)
    state = filled(llp.adamw_state(params, bits), grads)
    other = [params[0].clone()]
    others = {k: [t.clone() for t in v] for k, v in state.items()}
    params[0][5], params[0][300], params[0][599] = float("inf"), float("-inf"), float("nan")
    kw = dict(step=3, lr=0.01, betas=(0.9, 0.95), weight_decay=decay)
    llp.adamw_step(params, grads, **state, **kw)
    llp.adamw_step(other, grads, **others, **kw)
    assert params[0][5].item() == float("inf") and params[0][300].item() == float("-inf") and params[0][599].isnan()
    rest = torch.ones(600, dtype=torch.bool, device=DEV)
    rest[[5, 300, 599]] = False
    assert torch.allclose(params[0][rest], other[0][rest], rtol=1e-6, atol=1e-7)
    for k in state:
        assert torch.equal(state[k][0].view(torch.uint8), others[k][0].view(torch.uint8))
