"""Dropout layers that share one counter on the device: each adds its own offset on the host."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from lm_head_selected_gb300 import build
    build.build()


@pytest.mark.parametrize("base", [0, 5, (1 << 63) - 2, -3])
def test_the_mask_number_is_the_sum_of_both(base):
    import lm_head_selected_gb300 as llp
    x = torch.randn(3000, generator=torch.Generator().manual_seed(1)).cuda()
    counter = torch.tensor([base], device="cuda")
    masks = []
    for layer in (0, 1, 2, -1):
        y = llp.dropout_fwd(x, 0.5, 7, layer, device_offset=counter)
        assert torch.equal(y, llp.dropout_fwd(x, 0.5, 7, base + layer))  # modulo 2^64
        assert torch.equal(llp.dropout_bwd(x, 0.5, 7, layer, device_offset=counter), y)
        masks.append(y != 0)
    for i in range(len(masks)):
        for j in range(i):  # 3000 coins: 1500 agree, with a deviation of 27
            assert abs(int((masks[i] == masks[j]).sum()) - 1500) < 8 * 27


def test_layers_of_a_captured_step_draw_their_own_masks_and_the_backward_draws_them_again():
    import lm_head_selected_gb300 as llp
    layers = 3
    x = torch.randn(40, 100, generator=torch.Generator().manual_seed(2)).cuda()
    counter = torch.zeros((), dtype=torch.int64, device="cuda")

    def step():
        leaf = x.detach().requires_grad_(True)
        h, outs = leaf, []
        for layer in range(layers):
            h = llp.dropout(torch.ones_like(x) * leaf, 0.3, 9, layer, residual=h.detach(), device_offset=counter)
            outs.append(h)
        return outs, torch.autograd.grad(sum(o.sum() for o in outs), leaf)[0]

    def expected(number):
        leaf = x.detach().requires_grad_(True)
        h, outs = leaf, []
        for layer in range(layers):
            h = llp.dropout(leaf * 1.0, 0.3, 9, number + layer, residual=h.detach())
            outs.append(h)
        return outs, torch.autograd.grad(sum(o.sum() for o in outs), leaf)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, grad = step()
        counter.add_(layers)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want, want_grad = expected(k * layers)
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and torch.equal(grad, want_grad)
    assert int(counter) == 3 * layers


def test_a_counter_that_moves_before_the_backward_is_noticed():
    import lm_head_selected_gb300 as llp
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    x = torch.ones(64, device="cuda", requires_grad=True)
    y = llp.dropout(x, 0.5, 1, 2, device_offset=counter)
    counter.add_(1)
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_refusals():
    import lm_head_selected_gb300 as llp
    x, one = torch.zeros(4, 8, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    for call in (llp.dropout_fwd, llp.dropout_bwd, llp.dropout):
        for offset, device_offset in ((one, one), (0, 3), (0, one.cpu()), (0, one.int()), (0, one.expand(2)), (0, one[:0])):
            with pytest.raises(ValueError):
                call(x, 0.1, 1, offset, device_offset=device_offset)
        call(x, 0.1, 1, one)
