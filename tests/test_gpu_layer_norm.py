"""Layer norm and its gradients against the FP64 oracle: types, sizes,
parameters, strides, alignment, degenerate rows, invariance."""
import numpy as np
import pytest
import torch

from operator_bounds import DTYPES, U32, np64, rounded, sum_depth, within
from oracle import model_ops as mo

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from lm_head_selected_gb300 import build
    build.build()


def _problem(N, D, dtype, pdtype, seed, weight=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, D, generator=g) * (1 + 5 * torch.rand(N, 1, generator=g))
         + torch.randn(N, 1, generator=g)).to(dtype)
    gy = torch.randn(N, D, generator=g).to(dtype)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(pdtype) if weight else None
    b = torch.randn(D, generator=g).to(pdtype) if bias else None
    return x, gy, w, b


def _none(t, f):
    return None if t is None else f(t)


def _stat_errors(x, eps):
    """Oracle statistics with the bounds of their fp32 forms: mean (absolute) and rstd (relative)."""
    D = x.shape[1]
    _, mean, rstd = mo.layer_norm_forward(x, eps=eps)
    k = sum_depth(D) * U32
    dm = k * np.abs(x).mean(1) + 2 * U32 * np.abs(mean)
    # the variance: its sum, the rounding of each centred value (relative 3 roundings after
    # squaring), and the square of the mean's own error
    rel_var = k + 6 * U32 + dm * dm * rstd * rstd
    dr = 0.5 * rel_var * (1 + rel_var) + 4 * U32
    return mean, rstd, dm, dr


def _check(x, gy, w, b, eps=1e-5, xd=None, gyd=None):
    """xd, gyd: device tensors with the values of x, gy in another layout."""
    import lm_head_selected_gb300 as llp
    dt = x.dtype
    xd = x.cuda() if xd is None else xd
    gyd = gy.cuda() if gyd is None else gyd
    wd, bd = _none(w, torch.Tensor.cuda), _none(b, torch.Tensor.cuda)
    y, mean, rstd = llp.layer_norm_fwd(xd, wd, bd, eps)
    pdt = w.dtype if w is not None else b.dtype if b is not None else dt
    gx, gw, gb = llp.layer_norm_bwd(gyd, xd, mean, rstd, wd, param_dtype=pdt)
    assert y.dtype == gx.dtype == dt and gw.dtype == gb.dtype == pdt
    xn, gn, wn, bn = np64(x), np64(gy), _none(w, np64), _none(b, np64)
    eps = float(np.float32(eps))
    m_ref, r_ref, dm, dr = _stat_errors(xn, eps)
    y_ref = mo.layer_norm_forward(xn, wn, bn, eps)[0]
    within("mean", mean, m_ref, dm + U32 * np.abs(m_ref))
    within("rstd", rstd, r_ref, (dr + U32) * r_ref)
    h = np.abs((xn - m_ref[:, None]) * r_ref[:, None])
    dh = r_ref[:, None] * dm[:, None] + h * (dr[:, None] + 3 * U32)
    wa = np.ones(x.shape[1]) if wn is None else np.abs(wn)
    ba = np.zeros(x.shape[1]) if bn is None else np.abs(bn)
    slack = 1 + 1e-2  # second-order terms
    within("y", y, y_ref, slack * (rounded(y_ref, dt) + wa * dh + 2 * U32 * (h * wa + ba)))
    gx_ref, gw_ref, gb_ref = mo.layer_norm_backward(gn, xn, wn, eps)
    a = np.abs(gn) * wa
    k = sum_depth(x.shape[1]) * U32
    s1, s2 = a.mean(1)[:, None], (a * h).mean(1)[:, None]
    ds1 = (k + 3 * U32) * s1
    ds2 = (k + 4 * U32) * s2 + (a * dh).mean(1)[:, None]
    egx = r_ref[:, None] * (ds1 + h * ds2 + dh * s2 + 6 * U32 * (a + s1 + h * s2)) + np.abs(gx_ref) * dr[:, None]
    within("grad_x", gx, gx_ref, slack * (rounded(gx_ref, dt) + egx))
    kn = (x.shape[0] + 8) * U32
    within("grad_weight", gw, gw_ref,
           slack * (rounded(gw_ref, pdt) + kn * (np.abs(gn) * h).sum(0) + (np.abs(gn) * dh).sum(0)))
    within("grad_bias", gb, gb_ref, slack * (rounded(gb_ref, pdt) + kn * np.abs(gn).sum(0)))
    return y, mean, rstd, gx, gw, gb


SHAPES = [(1, 1), (3, 2), (5, 7), (1, 64), (33, 31), (64, 256), (257, 1000), (9, 1001), (40, 2688), (17, 4096),
          (130, 264), (2, 8200), (3, 20000), (2, 70001), (1000, 40), (700, 8)]


TYPES = [(dt, dt) for dt in DTYPES] + [(torch.bfloat16, torch.float32), (torch.float16, torch.float32)]


@pytest.mark.parametrize("dtype,pdt", TYPES)
@pytest.mark.parametrize("N,D", SHAPES)
def test_parity(dtype, pdt, N, D):
    _check(*_problem(N, D, dtype, pdt, seed=N + D))


@pytest.mark.parametrize("N", [2047, 4865, 16385])
def test_many_rows(N):
    _check(*_problem(N, 72, torch.bfloat16, torch.float32, seed=N))


@pytest.mark.parametrize("dtype,pdt", TYPES)
@pytest.mark.parametrize("N,D", [(5, 8200), (155, 9001), (309, 12288), (3, 16376), (160, 16384), (2, 16392), (7, 4100),
                                 (200, 8191)])
def test_wide_rows(dtype, pdt, N, D):
    """Rows of more vectors than up to three per thread take, of twice as many, and of more."""
    _check(*_problem(N, D, dtype, pdt, seed=N + D))


@pytest.mark.parametrize("weight,bias", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("D", [24, 513])
def test_optional_parameters(weight, bias, D):
    _check(*_problem(50, D, torch.float16, torch.float32, seed=D, weight=weight, bias=bias))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 96, 33])
def test_strides_and_alignment(dtype, D):
    """Column windows of a wider buffer, every n-th row, one repeated row; outputs are bitwise
    those of contiguous copies."""
    import lm_head_selected_gb300 as llp
    N = 45
    x, gy, w, b = _problem(N, 200, dtype, dtype, seed=D)
    w, b = w[:D].contiguous(), b[:D].contiguous()
    bx, bg = x.cuda(), gy.cuda()
    want = None
    for c0 in (0, 1, 8, 101):
        xv, gv = bx[:, c0:c0 + D], bg[:, c0:c0 + D]
        got = _check(x[:, c0:c0 + D], gy[:, c0:c0 + D], w, b, xd=xv, gyd=gv)
        want = _check(x[:, c0:c0 + D], gy[:, c0:c0 + D], w, b, xd=xv.contiguous(), gyd=gv.contiguous())
        for p, q in zip(got, want):
            assert torch.equal(p, q)
    _check(x[::3, :D], gy[::3, :D], w, b, xd=bx[::3, :D], gyd=bg[::3, :D])
    _check(x[:1, :D].expand(N, D), gy[:1, :D].expand(N, D), w, b, xd=bx[:1, :D].expand(N, D),
           gyd=bg[:1, :D].expand(N, D))
    # parameters and outputs that start at an odd element
    odd = lambda t: torch.cat([t[:1], t]).cuda()[1:]  # noqa: E731
    y0 = llp.layer_norm_fwd(bx[:, :D], w.cuda(), b.cuda())[0]
    flat = torch.zeros(N * D + 1, dtype=dtype, device="cuda")
    y1 = llp.layer_norm_fwd(bx[:, :D], odd(w), odd(b), out=flat[1:].view(N, D))[0]
    assert torch.equal(y0, y1) and flat[0] == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [4104, 8200, 9001, 16384, 16392])
def test_layouts_of_wide_rows(dtype, D):
    """Odd strides and starts give the bits of contiguous rows, whichever kernel takes them."""
    import lm_head_selected_gb300 as llp
    x, gy, w, b = (t.cuda() for t in _problem(160, D, dtype, dtype, seed=D))
    y, m, r = llp.layer_norm_fwd(x, w, b)
    grads = llp.layer_norm_bwd(gy, x, m, r, w)

    def odd(t, pad):
        wide = torch.full((t.shape[0], D + pad), float("nan"), dtype=dtype, device="cuda")
        wide[:, 1:1 + D] = t
        return wide[:, 1:1 + D]

    for pad in (3, 8):
        xo, go = odd(x, pad), odd(gy, pad + 2)
        for got, want in zip(llp.layer_norm_fwd(xo, w, b), (y, m, r)):
            assert torch.equal(got, want)
        for got, want in zip(llp.layer_norm_bwd(go, xo, m, r, w), grads):
            assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_degenerate_rows(dtype):
    """Constant rows, huge and tiny values, zeros; eps decides where the variance vanishes."""
    x = torch.randn(6, 128, generator=torch.Generator().manual_seed(1))
    x[1] = 3.0
    x[2] = 0.0
    x[3] *= 1e4 if dtype != torch.float16 else 1e3
    x[4] *= 1e-4
    x[5] += 100.0
    _, gy, w, b = _problem(6, 128, dtype, dtype, seed=2)
    _check(x.to(dtype), gy, w, b)
    _check(x.to(dtype), gy, w, b, eps=0.1)


@pytest.mark.parametrize("D", [40, 1001, 2688])
def test_non_finite_rows_stay_apart(D):
    import lm_head_selected_gb300 as llp
    x, gy, w, b = (t.cuda() for t in _problem(40, D, torch.bfloat16, torch.bfloat16, seed=3))
    y0, m0, r0 = llp.layer_norm_fwd(x, w, b)
    gx0 = llp.layer_norm_bwd(gy, x, m0, r0, w)[0]
    bad = x.clone()
    bad[7, 3], bad[20, 0] = NAN, float("inf")
    y, m, r = llp.layer_norm_fwd(bad, w, b)
    gx = llp.layer_norm_bwd(gy, bad, m, r, w)[0]
    keep = [i for i in range(40) if i not in (7, 20)]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(gx[keep], gx0[keep])
    assert torch.isnan(y[7]).all() and torch.isnan(y[20]).any()
    with pytest.raises(ValueError):
        llp.layer_norm_bwd(gy[:39], bad, m, r, w)


@pytest.mark.parametrize("D", [40, 1001, 2688, 4096])
def test_rows_do_not_depend_on_the_batch_and_runs_repeat(D):
    import lm_head_selected_gb300 as llp
    x, gy, w, b = (t.cuda() for t in _problem(3000, D, torch.bfloat16, torch.float32, seed=4))
    y, m, r = llp.layer_norm_fwd(x, w, b)
    gx, gw, gb = llp.layer_norm_bwd(gy, x, m, r, w)
    for size in (1, 7, 64, 257):
        i = torch.randperm(3000, generator=torch.Generator().manual_seed(size))[:size].cuda()
        ys, ms, rs = llp.layer_norm_fwd(x[i], w, b)
        assert torch.equal(ys, y[i]) and torch.equal(ms, m[i]) and torch.equal(rs, r[i])
        assert torch.equal(llp.layer_norm_bwd(gy[i], x[i], ms, rs, w)[0], gx[i])
        # without the parameters' gradients
        assert torch.equal(llp.layer_norm_bwd(gy[i], x[i], ms, rs, w, need_weight=False, need_bias=False)[0], gx[i])
    for _ in range(3):
        again = llp.layer_norm_bwd(gy, x, m, r, w)
        assert torch.equal(again[0], gx) and torch.equal(again[1], gw) and torch.equal(again[2], gb)


@pytest.mark.parametrize("need", [(True, False, False), (False, True, True), (False, True, False),
                                  (False, False, True), (True, False, True), (False, False, False)])
def test_partial_gradients(need):
    import lm_head_selected_gb300 as llp
    x, gy, w, b = (t.cuda() for t in _problem(300, 136, torch.bfloat16, torch.bfloat16, seed=5))
    _, m, r = llp.layer_norm_fwd(x, w, b)
    full = llp.layer_norm_bwd(gy, x, m, r, w)
    for got, want, needed in zip(llp.layer_norm_bwd(gy, x, m, r, w, *need), full, need):
        assert (got is None) if not needed else torch.equal(got, want)


def test_workspace_is_not_read_before_it_is_written():
    import lm_head_selected_gb300 as llp
    from lm_head_selected_gb300 import _lib
    x, gy, w, b = (t.cuda() for t in _problem(900, 264, torch.bfloat16, torch.bfloat16, seed=6))
    _, m, r = llp.layer_norm_fwd(x, w, b)
    want = llp.layer_norm_bwd(gy, x, m, r, w)
    nbytes = _lib.load().layer_norm_bwd_workspace_bytes(900, 264)
    for fill in (0, 255, 127):
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            for p, q in zip(llp.layer_norm_bwd(gy, x, m, r, w, workspace=ws), want):
                assert torch.equal(p, q)


def test_no_rows():
    import lm_head_selected_gb300 as llp
    x = torch.zeros(0, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    y, m, r = llp.layer_norm_fwd(x, w, w)
    assert y.shape == (0, 16) and m.shape == (0,)
    gx, gw, gb = llp.layer_norm_bwd(x, x, m, r, w)
    assert gx.shape == (0, 16) and torch.all(gw == 0) and torch.all(gb == 0)


def test_offsets_past_32_bits():
    import lm_head_selected_gb300 as llp
    N, D = 600001, 4096
    x = torch.empty(N, D, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(7))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    y, m, r = llp.layer_norm_fwd(x, w)
    rows = torch.tensor([0, 1, 524287, 524288, 600000], device="cuda")
    ys, ms, rs = llp.layer_norm_fwd(x[rows], w)
    assert torch.equal(y[rows], ys) and torch.equal(m[rows], ms) and torch.equal(r[rows], rs)
    gx = llp.layer_norm_bwd(y, x, m, r, w)[0]
    assert torch.equal(gx[rows], llp.layer_norm_bwd(ys, x[rows], ms, rs, w)[0])


def test_autograd_and_finite_differences():
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(8)
    x = torch.randn(2, 3, 12, generator=g).cuda().requires_grad_(True)
    w = torch.randn(12, generator=g).cuda().requires_grad_(True)
    b = torch.randn(12, generator=g).cuda().requires_grad_(True)
    c = torch.randn(2, 3, 12, generator=g).cuda()
    loss = lambda x_, w_, b_: (llp.layer_norm(x_, w_, b_).double() * c.double()).sum()  # noqa: E731
    loss(x, w, b).backward()
    # step h: the truncation is h^2 times a third derivative of order 10, the rounding of
    # 36 outputs of order 1 to fp32 divided by h
    h = 2.0 ** -8
    tol = 10 * h * h + 72 * 8 * U32 / h
    for k, t in enumerate((x, w, b)):
        flat = t.detach().reshape(-1)
        for i in (0, 5, flat.numel() - 1):
            d = torch.zeros_like(flat)
            d[i] = h
            d = d.view_as(t)
            p, q = [x.detach(), w.detach(), b.detach()], [x.detach(), w.detach(), b.detach()]
            p[k], q[k] = t.detach() + d, t.detach() - d
            diff = float((loss(*p) - loss(*q)) / (2 * h))
            assert abs(diff - float(t.grad.reshape(-1)[i])) <= tol
    # an expanded upstream gradient, a transposed input, no parameters
    llp.layer_norm(x, w, b).sum().backward()
    xt = torch.randn(12, 5, generator=g).cuda()
    assert torch.equal(llp.layer_norm(xt.t()), llp.layer_norm(xt.t().contiguous()))
    xb = x.detach().clone().requires_grad_(True)
    llp.layer_norm(xb, None, b).square().sum().backward()


def test_on_another_stream_and_in_a_graph():
    import lm_head_selected_gb300 as llp
    x, gy, w, b = (t.cuda() for t in _problem(500, 264, torch.bfloat16, torch.bfloat16, seed=9))
    y, m, r = llp.layer_norm_fwd(x, w, b)
    want = llp.layer_norm_bwd(gy, x, m, r, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ys, ms, rs = llp.layer_norm_fwd(x, w, b)
        got = llp.layer_norm_bwd(gy, x, ms, rs, w)
    s.synchronize()
    assert torch.equal(ys, y) and all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    sx = x.clone()
    with torch.cuda.graph(graph):
        yo, mo_, ro = llp.layer_norm_fwd(sx, w, b)
        out = llp.layer_norm_bwd(gy, sx, mo_, ro, w)
    for k in (1, 2):
        sx.copy_(x * k)
        graph.replay()
        torch.cuda.synchronize()
        yk, mk, rk = llp.layer_norm_fwd(x * k, w, b)
        assert torch.equal(yo, yk)
        assert all(torch.equal(p, q) for p, q in zip(out, llp.layer_norm_bwd(gy, x * k, mk, rk, w)))


def test_refusals():
    import lm_head_selected_gb300 as llp
    x = torch.zeros(3, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    m = torch.zeros(3, device="cuda")
    for bad in (lambda: llp.layer_norm_fwd(x.cpu(), w), lambda: llp.layer_norm_fwd(x, w.cpu()),
                lambda: llp.layer_norm_fwd(x, w[:7]), lambda: llp.layer_norm_fwd(x.t(), None),
                lambda: llp.layer_norm_fwd(x[0], w), lambda: llp.layer_norm_fwd(x[:, :0], None),
                lambda: llp.layer_norm_fwd(x, w, out=x.double()), lambda: llp.layer_norm_bwd(x[:2], x, m, m, w),
                lambda: llp.layer_norm_bwd(x.half(), x, m, m, w), lambda: llp.layer_norm_bwd(x, x, m[:2], m, w),
                lambda: llp.layer_norm_bwd(x, x, m, m, w, workspace=torch.zeros(1, dtype=torch.uint8, device="cuda")),
                lambda: llp.layer_norm_fwd(torch.zeros(30, device="cuda").as_strided((3, 8), (4, 1)), w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: llp.layer_norm_fwd(x.double(), w), lambda: llp.layer_norm_fwd(x, w.half()),
                lambda: llp.layer_norm_fwd(x.half(), w.half(), w), lambda: llp.layer_norm_bwd(x, x, m.half(), m, w),
                lambda: llp.layer_norm_bwd(x, x, m, m, w, param_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    for eps in (-1e-5, float("nan"), float("inf")):
        with pytest.raises(RuntimeError):
            llp.layer_norm_fwd(x, w, None, eps)
