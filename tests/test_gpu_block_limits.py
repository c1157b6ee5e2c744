"""Tensors of more than 2^31 elements: what lies past 32 bits comes out as it does alone."""
import pytest
import torch

import lm_head_selected_gb300 as llp
from test_gpu_gated_linear import check_backward

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_gated_linear():
    N, D, F = 132000, 64, 16384
    assert N * F > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(N, D, generator=g, device=DEV).to(BF16)
    wg, wu = (torch.randn(F, D, generator=g, device=DEV).mul_(D ** -0.5).to(BF16) for _ in range(2))
    y, pre = llp.gated_linear_fwd(x, wg, wu, keep=True)
    for rows in (slice(0, 300), slice(N - 300, N)):
        part, part_pre = llp.gated_linear_fwd(x[rows].contiguous(), wg, wu, keep=True)
        assert torch.equal(y[rows], part) and torch.equal(pre[:, rows], part_pre)
    # an upstream gradient in the last rows alone: theirs are the weights' gradients of those rows
    gy = torch.zeros_like(y)
    gy[N - 300:] = torch.randn(300, F, generator=g, device=DEV).to(BF16)
    gx, gwg, gwu = llp.gated_linear_bwd(gy, pre, x, wg, wu)
    last = slice(N - 300, N)
    assert not gx[:N - 300].any()
    # the sums' order depends on N: held against the definition with the bounds of the layer's own tests,
    # whose terms are additions on the tensor cores of up to one unit in the last place each
    check_backward((gx[last], gwg, gwu), gy[last], pre[:, last], x[last], wg, wu, "silu")


@pytest.mark.parametrize("gate", ["columns", "rows"])
def test_residual_rms_norm(gate):
    N, D = 525000, 4096
    assert N * D > 2 ** 31
    x = torch.empty(N, D, dtype=BF16, device=DEV).normal_()
    b = torch.empty(N, D, dtype=BF16, device=DEV).normal_()
    w, pw = (torch.rand(D, device=DEV) + 0.5 for _ in range(2))
    gt = torch.rand(D, device=DEV) if gate == "columns" else x
    last = slice(N - 5, N)
    s, h, pr, r = llp.residual_rms_norm_fwd(x, b, gt, pw, w, scale=0.5)
    cut = [t[last] if t.dim() == 2 else t for t in (x, b, gt)]
    part = llp.residual_rms_norm_fwd(*cut, pw, w, scale=0.5)
    for a, c in zip((s, h, pr, r), part):
        assert torch.equal(a[last], c)
    del x
    grads = llp.residual_rms_norm_bwd(h, b, s, b, gt, pw, w, pr, r, 0.5)
    want = llp.residual_rms_norm_bwd(h[last], b[last], s[last], b[last], cut[2], pw, w, pr[last], r[last], 0.5)
    for a, c in zip(grads[:2], want[:2]):
        assert torch.equal(a[last], c)
    if gate == "rows":
        assert torch.equal(grads[2][last], want[2])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(bits):
    n = 2 ** 31 + 256 * 20 + 77
    p = torch.zeros(n, dtype=BF16, device=DEV)
    g = torch.empty(n, dtype=BF16, device=DEV).normal_()
    state = llp.adamw_state([p], bits)
    at = 2 ** 31 - 256 * 4
    end_p, end_g = p[at:].clone(), g[at:].clone()
    end = llp.adamw_state([end_p], bits)
    for step in (1, 2):
        llp.adamw_step([p], [g], **state, step=step, lr=0.01)
        llp.adamw_step([end_p], [end_g], **end, step=step, lr=0.01)
    assert torch.equal(p[at:], end_p)
    for k, t in end.items():
        have = state[k][0][at // 256:] if k.endswith("scale") else state[k][0][at:]
        assert torch.equal(have.view(torch.uint8), t[0].view(torch.uint8)), k
    assert p[:1024].ne(0).all() and p[2 ** 30:2 ** 30 + 1024].ne(0).all()
