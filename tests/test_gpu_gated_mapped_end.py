"""The gated linear layer where a tensor's last byte is the last of a mapped region of device memory: no
copy of a tile may fetch what lies behind it, nor between the two weights."""
import itertools

import pytest
import torch

import lm_head_selected_gb300 as llp
from mapped_region import DEV, Region, at_the_end
from test_gpu_gated_linear import ACTS, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def regions():
    return [torch.as_tensor(Region(), device=DEV) for _ in range(2)]


# D that fills no whole K blocks, then whole ones, F that fills no whole tiles
SHAPES = [(224, 80), (72, 136), (8, 8), (200, 1000), (1000, 264), (136, 4872), (64, 8), (192, 80), (448, 56), (256, 1992),
          (128, 4168)]


@pytest.mark.parametrize("D,F", SHAPES)
@pytest.mark.parametrize("N", [1, 5, 32, 139])
def test_tensors_at_the_end_of_mapped_memory(regions, N, D, F):
    x, wg, wu, _ = inputs(N, D, F, torch.bfloat16)
    act = ACTS[(N + D) % 3]
    want = llp.gated_linear_fwd(x, wg, wu, act)
    for first, second in itertools.permutations(("x", "w_gate", "w_up"), 2):
        args = {"x": x, "w_gate": wg, "w_up": wu}
        args[first], args[second] = at_the_end(regions[0], args[first]), at_the_end(regions[1], args[second])
        assert torch.equal(llp.gated_linear_fwd(**args, activation=act), want), (first, second)
    assert llp.device_status() == 0


@pytest.mark.parametrize("D,F", SHAPES)
@pytest.mark.parametrize("N", [1, 33, 300])
def test_gradients_of_tensors_at_the_end_of_mapped_memory(regions, N, D, F):
    x, wg, wu, gy = inputs(N, D, F, torch.float16)
    act = ACTS[(N + F) % 3]
    _, pre = llp.gated_linear_fwd(x, wg, wu, act, keep=True)
    want = llp.gated_linear_bwd(gy, pre, x, wg, wu, act)
    names = ("grad_y", "pre", "x", "w_gate", "w_up")
    for first, second in zip(names, names[1:] + names[:1]):
        args = dict(zip(names, (gy, pre, x, wg, wu)))
        for k, region in ((first, regions[0]), (second, regions[1])):
            if args[k].numel() * 2 <= region.numel():
                args[k] = at_the_end(region, args[k])
        for a, b in zip(llp.gated_linear_bwd(**args, activation=act), want):
            assert torch.equal(a, b), (first, second)
    assert llp.device_status() == 0
