"""Dropout against the FP64 oracle: the mask element by element, values, types,
sizes, alignment, counters past 32 bits, graphs."""
import numpy as np
import pytest
import torch

from operator_bounds import DTYPES, U32, np64, rounded, within
from oracle import model_ops as mo

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from lm_head_selected_gb300 import build
    build.build()


def _check(x, p, seed, offset, residual=None):
    import lm_head_selected_gb300 as llp
    y = llp.dropout_fwd(x.cuda(), p, seed, offset, None if residual is None else residual.cuda())
    rn = None if residual is None else np64(residual)
    ref = mo.dropout_forward(np64(x), p, seed, offset, rn)
    part = mo.dropout_forward(np.abs(np64(x)), p, seed, offset, None if rn is None else np.abs(rn))
    assert y.dtype == x.dtype
    within("y", y, ref, rounded(ref, x.dtype) * (1 + 1e-3) + 3 * U32 * part)
    if residual is None:
        assert torch.equal(llp.dropout_bwd(x.cuda(), p, seed, offset), y)
        keep = mo.dropout_keep(x.numel(), p, seed, offset).reshape(x.shape)
        assert np.all(np64(y)[~keep] == 0)
    return y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 5), (64, 256), (33, 1001), (5, 3, 2688), (1111, 77)])
@pytest.mark.parametrize("residual", [False, True])
def test_parity(dtype, shape, residual):
    g = torch.Generator().manual_seed(len(shape) + shape[0])
    x = torch.randn(*shape, generator=g).to(dtype)
    r = torch.randn(*shape, generator=g).to(dtype) if residual else None
    _check(x, 0.1, 1234567, 0, r)
    _check(x, 0.5, -5 % (1 << 64), (1 << 63) - 3, r)


@pytest.mark.parametrize("p", [0.0, 1.0, 1.0 / 65536, 65535.0 / 65536, 2.0 ** -18, 0.3, 0.999999])
def test_probabilities(p):
    x = torch.randn(4096, generator=torch.Generator().manual_seed(1))
    y = _check(x, p, 99, 3)
    if p in (0.0, 2.0 ** -18):
        assert torch.equal(y.cpu(), x)
    if p in (1.0, 0.999999):
        assert torch.all(y == 0)


def test_dropped_elements_are_zero_whatever_they_hold():
    import lm_head_selected_gb300 as llp
    keep = torch.from_numpy(mo.dropout_keep(1000, 0.5, 7, 1))
    for bad in (NAN, float("inf"), -float("inf")):
        x = torch.where(keep, torch.ones(1000), torch.full((1000,), bad)).cuda()
        assert torch.equal(llp.dropout_fwd(x, 0.5, 7, 1).cpu(), keep.float() * 2)
        assert torch.equal(llp.dropout_bwd(x, 0.5, 7, 1).cpu(), keep.float() * 2)
        assert torch.equal(llp.dropout_fwd(x, 0.5, 7, 1, residual=torch.ones(1000, device="cuda")).cpu(),
                           keep.float() * 2 + 1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_alignment_and_in_place(dtype):
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(2)
    buf = torch.randn(3000, generator=g).to(dtype).cuda()
    res = torch.randn(3000, generator=g).to(dtype).cuda()
    for a, b, c in ((0, 0, 0), (1, 0, 0), (0, 3, 0), (0, 0, 1), (5, 2, 7)):
        x, r = buf[a:a + 2001], res[b:b + 2001]
        want = llp.dropout_fwd(x.clone(), 0.2, 3, 4, residual=r.clone())
        out = torch.zeros(2010, dtype=dtype, device="cuda")
        llp.dropout_fwd(x, 0.2, 3, 4, residual=r, out=out[c:c + 2001])
        assert torch.equal(out[c:c + 2001], want)
        assert torch.all(out[:c] == 0) and torch.all(out[c + 2001:] == 0)
        for target in (x.clone(), r.clone()):
            xi, ri = (target, r) if torch.equal(target, x) else (x, target)
            assert torch.equal(llp.dropout_fwd(xi, 0.2, 3, 4, residual=ri, out=target), want)


def test_elements_past_32_bits():
    """Windows of a tensor of more than 2^31 elements, far apart."""
    import lm_head_selected_gb300 as llp
    n = (1 << 31) + 12345
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = llp.dropout_fwd(x, 0.5, 11, 2)
    for first in (0, 1 << 20, (1 << 31) - 40, n - 77):
        count = min(5000, n - first)
        keep = mo.dropout_keep(count, 0.5, 11, 2, first=first)
        assert np.array_equal(np64(y[first:first + count]), keep * 2.0)


def test_device_offset_and_graph():
    """An offset on the device is read when the kernel runs: replays of one graph draw new masks."""
    import lm_head_selected_gb300 as llp
    x = torch.randn(5000, generator=torch.Generator().manual_seed(3)).cuda()
    off = torch.tensor([5], device="cuda")
    assert torch.equal(llp.dropout_fwd(x, 0.3, 1, off), llp.dropout_fwd(x, 0.3, 1, 5))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = llp.dropout_fwd(x, 0.3, 1, off)
        g = llp.dropout_bwd(x, 0.3, 1, off)
        off.add_(1)
    for k in range(5, 8):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, llp.dropout_fwd(x, 0.3, 1, k)) and torch.equal(g, y)


def test_autograd_and_differences():
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(4)
    x = torch.randn(6, 50, generator=g).cuda().requires_grad_(True)
    r = torch.randn(6, 50, generator=g).cuda().requires_grad_(True)
    c = torch.randn(6, 50, generator=g).cuda()
    (llp.dropout(x, 0.4, 21, 6, residual=r) * c).sum().backward()
    keep = torch.from_numpy(mo.dropout_keep(300, 0.4, 21, 6)).view(6, 50).cuda()
    s = 65536.0 / (65536 - 26214)
    assert torch.allclose(x.grad, torch.where(keep, c * s, 0.0), rtol=4 * U32, atol=0)
    assert torch.equal(r.grad, c)
    # linear in x: a step of 2^-4 gives the same slope as the gradient up to fp32 rounding
    for i, j in ((0, 0), (2, 17), (5, 49)):
        d = torch.zeros_like(x)
        d[i, j] = 2.0 ** -4
        up, down = (llp.dropout(x.detach() + e, 0.4, 21, 6)[i, j].double() for e in (d, -d))
        slope = float((up - down) * 8) * float(c[i, j])
        assert abs(slope - float(x.grad[i, j])) <= 8 * 16 * 8 * U32
    # a broadcast upstream gradient, a strided input, an offset on the device
    llp.dropout(x, 0.4, 21).sum().backward()
    xt = torch.randn(50, 6, generator=g).cuda()
    assert torch.equal(llp.dropout(xt.t(), 0.4, 21), llp.dropout(xt.t().contiguous(), 0.4, 21))
    off = torch.tensor(9, device="cuda")
    xg = x.detach().clone().requires_grad_(True)
    llp.dropout(xg, 0.4, 21, off).sum().backward()
    assert torch.equal(xg.grad, llp.dropout_bwd(torch.ones_like(xg), 0.4, 21, 9))
    assert llp.dropout_fwd(torch.zeros(0, 4, device="cuda"), 0.5, 1).shape == (0, 4)


def test_on_another_stream():
    import lm_head_selected_gb300 as llp
    x = torch.randn(10000, generator=torch.Generator().manual_seed(5)).cuda()
    want = llp.dropout_fwd(x, 0.5, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = llp.dropout_fwd(x, 0.5, 2)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    import lm_head_selected_gb300 as llp
    x = torch.zeros(4, 8, device="cuda")
    for bad in (lambda: llp.dropout_fwd(x.cpu(), 0.1, 1), lambda: llp.dropout_fwd(x.t(), 0.1, 1),
                lambda: llp.dropout_fwd(x, -0.1, 1), lambda: llp.dropout_fwd(x, 1.1, 1),
                lambda: llp.dropout_fwd(x, NAN, 1), lambda: llp.dropout_fwd(x, 0.1, 1, residual=x[:2]),
                lambda: llp.dropout_fwd(x, 0.1, 1, residual=x.half()),
                lambda: llp.dropout_fwd(x, 0.1, 1, residual=torch.zeros(8, 4, device="cuda").t()),
                lambda: llp.dropout_fwd(x, 0.1, 1, residual=x.cpu()), lambda: llp.dropout_fwd(x, 0.1, 1, out=x[:2]),
                lambda: llp.dropout_fwd(x, 0.1, 1, torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: llp.dropout_fwd(x, 0.1, 1, torch.zeros(1, device="cuda")),
                lambda: llp.dropout_fwd(x, 0.1, 1, torch.zeros(1, dtype=torch.int64)),
                lambda: llp.dropout_bwd(x.t(), 0.1, 1), lambda: llp.dropout_bwd(x, 2.0, 1)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        llp.dropout_fwd(x.double(), 0.1, 1)
