"""The autograd entry points of the operators around the head: inputs and upstream gradients
in layouts that the kernels do not read in place."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from lm_head_selected_gb300 import build
    build.build()


def _windows(N, D, hop, dtype, seed):
    """N windows of D elements, `hop` apart, in one buffer."""
    flat = torch.randn(N * hop + D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    return flat.as_strided((N, D), (hop, 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hop", [1, 4, 63])
def test_layer_norm_of_overlapping_windows(dtype, hop):
    import lm_head_selected_gb300 as llp
    N, D = 30, 64
    signal = torch.randn((N - 1) * hop + D, generator=torch.Generator().manual_seed(hop)).to(dtype).cuda()
    w = torch.randn(D, generator=torch.Generator().manual_seed(2)).cuda()
    results = []
    for copy in (False, True):
        s, p = signal.clone().requires_grad_(True), w.clone().requires_grad_(True)
        x = s.unfold(0, D, hop)
        y = llp.layer_norm(x.contiguous() if copy else x, p)
        y.float().square().sum().backward()
        results.append((y, p.grad, s.grad))
    for got, want in zip(*results):
        assert torch.equal(got, want)


@pytest.mark.parametrize("hop", [1, 4, 63])
def test_upstream_gradients_of_overlapping_rows(hop):
    import lm_head_selected_gb300 as llp
    N, D, V = 30, 64, 9
    g = torch.Generator().manual_seed(hop)
    grad = _windows(N, D, hop, torch.float32, hop)
    table = torch.randn(V, D, generator=g).cuda()
    t = torch.randint(0, V, (N,), generator=g).cuda()
    x, w = torch.randn(N, D, generator=g).cuda(), torch.randn(D, generator=g).cuda()
    calls = {"embedding": (lambda w_: llp.embedding(t, w_), table), "norm": (lambda x_: llp.layer_norm(x_, w), x),
             "dropout": (lambda x_: llp.dropout(x_, 0.3, 5), x)}
    for name, (call, value) in calls.items():
        grads = []
        for up in (grad, grad.contiguous()):
            leaf = value.clone().requires_grad_(True)
            call(leaf).backward(up)
            grads.append(leaf.grad)
        assert torch.equal(*grads), name


def test_rows_that_can_be_read_in_place_are_not_copied():
    from lm_head_selected_gb300.ops import _readable_rows
    buf = torch.randn(20, 100, device="cuda")
    for t in (buf, buf[:, 3:40], buf[::2], buf[:1].expand(7, 100), buf[:, :1], buf[:1], buf[:0], buf[:1].t()[:, :1]):
        assert _readable_rows(t) is t
    for t in (buf.t(), buf[:, ::2], buf.as_strided((5, 10), (4, 1)), buf.expand(2, 20, 100)[:, :, 0]):
        assert _readable_rows(t) is not t and torch.equal(_readable_rows(t), t)


def test_refusals():
    import lm_head_selected_gb300 as llp
    x, t = torch.zeros(4, 8, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: llp.layer_norm(x[0, 0]), lambda: llp.layer_norm(x[:, :0]), lambda: llp.layer_norm(x[:0, :0]),
                lambda: llp.dropout(x, 0.1, 1, residual=3.0), lambda: llp.dropout(x, 0.1, 1, residual=x.cpu()),
                lambda: llp.embedding(t, x[0, 0]), lambda: llp.embedding(t, x[0]), lambda: llp.embedding(t.cpu(), x)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: llp.embedding(None, x), lambda: llp.embedding([1, 2], x), lambda: llp.embedding(t.int(), x),
                lambda: llp.layer_norm(x.double()), lambda: llp.dropout(x.double(), 0.1, 1)):
        with pytest.raises(TypeError):
            bad()


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf"), 1e39])
def test_scales_that_are_not_finite(scale):
    import lm_head_selected_gb300 as llp
    w, t = torch.zeros(4, 8, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: llp.embedding(t, w, scale), lambda: llp.embedding_fwd(t, w, scale),
                lambda: llp.embedding_bwd(w[:3], t, 4, scale),
                lambda: llp.embedding_bwd(w[:3], t, 4, scale, out=w, accumulate=True)):
        with pytest.raises(ValueError, match="scale"):
            bad()
    assert not w.any()
