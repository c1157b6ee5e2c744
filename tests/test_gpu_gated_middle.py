"""The gated linear layer where one kernel takes up to 224 tokens (rows of two waves), and its activations far
out in their tails."""
import math

import numpy as np
import pytest
import torch

import lm_head_selected_gb300 as llp
from operator_bounds import UNIT, np64, rounded, within
from oracle import block_ops as bo
from test_gpu_gated_linear import ACTS, check_forward, inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [72, 192])
def test_batches_of_129_to_224_tokens(D, dtype):
    F = 9736
    x, wg, wu, _ = inputs(300, D, F, dtype)
    whole, pre = llp.gated_linear_fwd(x, wg, wu, "silu", keep=True)
    for N in (97, 129, 144, 161, 200, 208, 224, 225):
        y, p = llp.gated_linear_fwd(x[11:11 + N], wg, wu, "silu", keep=True)
        assert torch.equal(y, whole[11:11 + N]) and torch.equal(p, pre[:, 11:11 + N]), N
        rows = torch.tensor([0, N // 2, N - 1], device=DEV)
        check_forward(y[rows], p[:, rows], x[11 + rows], wg, wu, "silu")
    assert llp.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [2, 300])
def test_activations_far_out(act, dtype, N):
    """Gates from -100 to 100 that are exact, and an up projection of 1.  An exponential of an argument t that is
    rounded a few times is off by that many 2^-24 |t|: silu's argument is rounded once, gelu's z^2 / 2
    twice, its tanh form's four times, and the constants; the rest stays below 2^-19.  A factor below fp32's
    least normal number counts as 0."""
    F = 64
    z = np.concatenate([np.linspace(-16, 16, N * F // 2), np.linspace(-100, 100, N * F - N * F // 2)])
    x = torch.zeros(N, F + 8)
    x[:, :F] = torch.from_numpy(z.reshape(N, F)).float()
    x[:, F] = 1.0
    wg, wu = torch.zeros(F, F + 8), torch.zeros(F, F + 8)
    wg[:, :F] = torch.eye(F)
    wu[:, F] = 1.0
    x, wg, wu = (t.to(dtype).to(DEV) for t in (x, wg, wu))
    y, pre = llp.gated_linear_fwd(x, wg, wu, act, keep=True)
    assert torch.equal(pre[0], x[:, :F]) and (pre[1] == 1).all()
    z = np64(x[:, :F])
    with np.errstate(over="ignore"):  # the tanh form without the difference of 1 + tanh
        ref = (bo.activation(act, z)[0] if act != "gelu_tanh" else
               z / (1.0 + np.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))))
    a = np.abs(z)
    units = {"silu": 2 * a, "gelu": 1.5 * z * z,
             "gelu_tanh": 5 * 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)}[act]
    # past the exponential's range the value itself is below the least normal number
    rel = np.minimum(2.0 ** -19 + 2.0 ** -24 * units, 1.0)
    within(act, y, ref, rounded(ref, dtype) + rel * np.abs(ref) * (1 + UNIT[dtype]) + a * 2.0 ** -126)
