"""AdamW's wrapper: parameters and gradients that come as iterators."""
import pytest
import torch

import lm_head_selected_gb300 as llp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def model():
    return torch.nn.Sequential(torch.nn.Linear(24, 40), torch.nn.Linear(40, 8)).to(DEV, torch.bfloat16)


@pytest.mark.parametrize("bits", [32, 8])
def test_parameters_from_an_iterator(bits):
    net = model()
    state = llp.adamw_state(net.parameters(), bits, masters=True)
    want = llp.adamw_state(list(net.parameters()), bits, masters=True)
    assert state.keys() == want.keys()
    for k in want:
        assert len(state[k]) == 4 and all(a.shape == b.shape and a.dtype == b.dtype for a, b in zip(state[k], want[k]))
    net(torch.randn(5, 24, device=DEV, dtype=torch.bfloat16)).float().pow(2).sum().backward()
    kept = [p.detach().clone() for p in net.parameters()]
    llp.adamw_step(net.parameters(), (p.grad for p in net.parameters()), **state, step=1, lr=0.01)
    assert not any(torch.equal(p, k) for p, k in zip(net.parameters(), kept))
