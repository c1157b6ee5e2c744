"""AdamW's wrapper: what autograd learns of a step."""
import pytest
import torch

import lm_head_selected_gb300 as llp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("masters", [False, True])
def test_every_written_tensor_counts_a_version(bits, masters):
    params = [torch.randn(300, device=DEV).to(torch.bfloat16), torch.randn(17, device=DEV)]
    grads = [torch.randn_like(p) for p in params]
    state = llp.adamw_state(params, bits, masters)
    written = params + [t for v in state.values() for t in v if t is not None]
    versions = [t._version for t in written]
    read = [t._version for t in grads]
    llp.adamw_step(params, grads, **state, step=1)
    assert all(t._version > v for t, v in zip(written, versions))
    assert [t._version for t in grads] == read


def test_a_graph_that_saved_a_master_copy_notices_the_step():
    params = [torch.randn(64, device=DEV).to(torch.bfloat16)]
    state = llp.adamw_state(params, masters=True)
    master = state["masters"][0]
    x = torch.randn(64, device=DEV, requires_grad=True)
    y = (x * master).sum()
    llp.adamw_step(params, [torch.randn_like(params[0])], **state, step=1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
