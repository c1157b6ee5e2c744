"""The gated linear layer on tensors that start off a 16-byte boundary: autograd hands over gradients at any
place, and an input may be a view into a flat buffer."""
import pytest
import torch

import lm_head_selected_gb300 as llp

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def inputs(N, D, F, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(N + D + F)
    return [(torch.randn(*s, generator=g) * k).to(dtype).to(DEV)
            for s, k in (((N, D), 1.0), ((F, D), D ** -0.5), ((F, D), D ** -0.5), ((N, F), 1.0))]


def shifted(t, by):
    """A copy that starts `by` elements into a buffer of its own."""
    room = torch.empty(t.numel() + 64, dtype=t.dtype, device=t.device)
    v = room[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16 == 2 * by % 16
    return v


def gradients(x, wg, wu, gy, loss):
    ts = [t.detach().requires_grad_(True) for t in (x, wg, wu)]
    loss(llp.gated_linear(*ts), gy).backward()
    return [t.grad for t in ts]


@pytest.mark.parametrize("N", [1, 40, 300])
@pytest.mark.parametrize("ahead", [1, 3, 7, 8])
def test_an_upstream_gradient_anywhere(N, ahead):
    """y flattened behind a few other values: the gradient that comes back is a contiguous view at an odd place."""
    x, wg, wu, gy = inputs(N, 64, 136)
    other = torch.ones(ahead, dtype=x.dtype, device=DEV)

    def joined(y, gy):
        return (torch.cat([other, y.flatten()]) * torch.cat([other, gy.flatten()])).sum()

    want = gradients(x, wg, wu, gy, lambda y, gy: (y * gy).sum())
    for a, b in zip(gradients(x, wg, wu, gy, joined), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("by", [1, 4, 5])
def test_an_input_anywhere(by, dtype):
    x, wg, wu, gy = inputs(33, 72, 64, dtype)
    moved = shifted(x, by)
    with torch.no_grad():
        assert torch.equal(llp.gated_linear(moved, wg, wu), llp.gated_linear(x, wg, wu))
    loss = lambda y, gy: (y * gy).sum()  # noqa: E731
    for a, b in zip(gradients(moved, wg, wu, gy, loss), gradients(x, wg, wu, gy, loss)):
        assert torch.equal(a, b)


def test_a_captured_step_with_an_input_anywhere():
    x, wg, wu, _ = inputs(40, 64, 128)
    moved = shifted(x, 3)
    want = llp.gated_linear_fwd(x, wg, wu)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.no_grad(), torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        y = llp.gated_linear(moved, wg, wu)
    torch.cuda.current_stream().wait_stream(side)
    moved.zero_()
    moved.copy_(x)
    graph.replay()
    assert torch.equal(y, want)


def test_other_tensors_off_the_boundary_are_refused_by_name():
    x, wg, wu, gy = inputs(8, 64, 128)
    _, pre = llp.gated_linear_fwd(x, wg, wu, keep=True)
    for name, call in (("w_gate", lambda: llp.gated_linear(x, shifted(wg, 1), wu)),
                       ("w_up", lambda: llp.gated_linear(x, wg, shifted(wu, 4))),
                       ("x", lambda: llp.gated_linear_fwd(shifted(x, 1), wg, wu)),
                       ("out", lambda: llp.gated_linear_fwd(x, wg, wu, out=shifted(gy, 1))),
                       ("grad_y", lambda: llp.gated_linear_bwd(shifted(gy, 3), pre, x, wg, wu)),
                       ("pre", lambda: llp.gated_linear_bwd(gy, shifted(pre, 1), x, wg, wu))):
        with pytest.raises(ValueError, match=f"^{name} must start on a 16-byte boundary"):
            call()
