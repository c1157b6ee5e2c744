"""The tied language-model step of examples/tied_lm_step.py: its table gradient is the sum of
the head's and the embedding's, its steps repeat bit for bit, and it learns."""
import importlib.util
import os

import pytest
import torch

from operator_bounds import U32

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    from lm_head_selected_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("tied_lm_step", os.path.join(ROOT, "examples", "tied_lm_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_table_gradient_is_the_sum_of_both_uses(ex):
    """The accumulated bf16 gradient against the two gradients formed apart: one rounding of the
    head's part and one of the sum, against a rounding of each part."""
    import lm_head_selected_gb300 as llp
    V, D, N = 500, 128, 300
    model = ex.TiedLM(V, D, seed=3)
    tokens, targets = ex.batch(N, V, seed=4)
    _, got, inner = model.gradients(tokens, targets, 0)
    x = llp.embedding_fwd(tokens, model.table, model.scale).requires_grad_(True)
    y = model.body(x, 0)
    logp, lse = llp.linear_logp_fwd(y.detach(), model.table, targets)
    valid = torch.isfinite(lse)
    g = torch.where(valid, -1.0 / valid.sum(), 0.0).float()
    gy, head, _ = llp.linear_logp_bwd(g, lse, y.detach(), model.table, targets)
    gx, = torch.autograd.grad(y, [x], gy)
    count = torch.bincount(tokens, minlength=V)[:, None].double()
    emb = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, tokens, gx.double()) * model.scale
    size = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, tokens, gx.double().abs()) * model.scale
    want = head.double() + emb
    bound = 2.0 ** -8 * want.abs() * (1 + 1e-3) + (count + 4) * U32 * (size + head.double().abs()) + 2.0 ** -130
    assert bool(((got.double() - want).abs() <= bound).all())
    assert all(bool(torch.isfinite(gr).all()) for _, gr in inner)


def test_steps_repeat_and_learn(ex):
    losses = []
    tables = []
    for _ in range(2):
        model = ex.TiedLM(512, 128, seed=5)
        tokens, targets = ex.batch(1024, 512, seed=6)
        losses.append([float(model.step(tokens, targets, i, 2.0)) for i in range(25)])
        tables.append(model.table.clone())
    assert losses[0] == losses[1] and torch.equal(tables[0], tables[1])
    assert losses[0][-1] < 0.7 * losses[0][0]
