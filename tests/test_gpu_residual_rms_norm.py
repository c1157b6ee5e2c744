"""The RMS norms around a block on the GPU against their FP64 definition: every combination of the optional
inputs, all types, ragged and strided rows; bounds from the arithmetic (fp32 sums, one rounding)."""
import itertools

import numpy as np
import pytest
import torch

import lm_head_selected_gb300 as llp
from operator_bounds import DTYPES, U32, np64, rounded, sum_depth
from operator_bounds import within as within_range
from oracle import block_ops as bo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-5


def inputs(N, D, dtype, pdt, gate, post, norm, branch=True, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dt=dtype):
        return (torch.randn(*shape, generator=g) * std + mean).to(dt).to(DEV)

    x = normal(N, D, mean=0.5)
    return [x, normal(N, D, std=3.0) if branch else None,
            {"none": None, "columns": normal(D, dt=pdt), "rows": normal(N, D)}[gate],
            normal(D, std=0.3, mean=1.0, dt=pdt) if post else None, normal(D, std=0.3, mean=1.0, dt=pdt) if norm else None]


def within(name, got, ref, bound):
    """within(), for outputs that may pass the type's range: half a step past its largest value and
    further out, rounding to nearest gives infinity (65520 in fp16, whose largest is 65504).  bound is the
    one rounding's error and that of the value v in fp32 before it, |v - ref| <= err.  The output is infinite
    where |v| >= edge: surely where |ref| - err >= edge, never where |ref| + err < edge, and between the two
    either that or, as everywhere else, a value within the bound."""
    top = torch.finfo(got.dtype).max
    edge = top + 2.0 ** np.floor(np.log2(top)) * torch.finfo(got.dtype).eps / 2
    err = bound - rounded(ref, got.dtype)
    value, infinite = np64(got), np.copysign(np.inf, ref)
    surely = np.abs(ref) - err >= edge
    assert (value[surely] == infinite[surely]).all(), name
    over = surely | ((np.abs(ref) + err >= edge) & (value == infinite))
    within_range(name, torch.from_numpy(np.where(over, ref, value)), ref, bound)


def test_what_counts_as_infinite():
    half, inf = torch.float16, float("inf")

    def passes(got, ref, err):
        ref = np.array([ref])
        try:
            within("", torch.tensor([got], dtype=half), ref, rounded(ref, half) + err)
        except AssertionError:
            return False
        return True

    assert passes(inf, 65524.3, 0.1) and not passes(65504.0, 65524.3, 0.1)   # past the edge
    assert passes(65504.0, 65516.0, 0.1) and not passes(inf, 65516.0, 0.1)   # before it
    assert passes(inf, 65518.0, 4.0) and passes(65504.0, 65518.0, 4.0)       # either side of it within err
    assert passes(-inf, -65524.3, 0.1) and not passes(inf, -65524.3, 0.1) and not passes(inf, 100.0, 0.1)


def n64(t):
    return None if t is None else np64(t)


def check_forward(got, args, scale):
    """Each row sum loses at most depth additions' roundings of its (all positive) terms; rstd half of
    that and the few of its own; s and h the products' and sums' on top."""
    x, b, gate, pw, w = (n64(t) for t in args)
    dt, D = args[0].dtype, x.shape[1]
    ref = bo.residual_forward(x, b, gate, pw, w, scale, EPS)
    stat = (sum_depth(D) + 8) * U32  # of a row's statistic, relative
    s, h, post_rstd, rstd = got
    t = np.abs(ref[0] - x)
    if b is None:
        assert s is args[0]
        err = np.zeros_like(x)
    else:
        err = (stat + 8 * U32) * t + 2 * U32 * (np.abs(x) + t)
        within("s", s, ref[0], rounded(ref[0], dt) + err * 1.01)
    if pw is not None:
        within("post_rstd", post_rstd, ref[2], stat * ref[2])
    if w is not None:
        # the sum of s^2 moves with s's own error
        moved = 2 * (err * np.abs(ref[0])).sum(1) / np.maximum((ref[0] ** 2).sum(1), 1e-300) + stat
        within("rstd", rstd, ref[3], moved * ref[3])
        within("h", h, ref[1], rounded(ref[1], dt) + 1.01 * ((moved[:, None] + 6 * U32) * np.abs(ref[1]) +
                                                           err * np.abs(ref[3][:, None] * w)))


def check_backward(got, gs, gh, s, args, post_rstd, rstd, scale):
    _, b, gate, pw, w = (n64(t) for t in args)
    gs, gh, sn, pr, r = (n64(t) for t in (gs, gh, s, post_rstd, rstd))
    dt, (N, D) = s.dtype, sn.shape
    pdt = next((t.dtype for t in (args[4], args[3], args[2]) if t is not None), dt)
    ref = bo.residual_backward(gs, gh, sn, b, gate, pw, w, pr, r, scale)
    K, few = (sum_depth(D) + 8) * U32, 8 * U32
    eG = 2 * U32 * np.abs(ref[0]) + (0 if gs is None else few * np.abs(gs))
    if w is not None:
        c, a = sn * r[:, None], gh * w
        eG = eG + r[:, None] * (few * (np.abs(a) + np.abs(c) * np.abs((a * c).mean(1, keepdims=True))) +
                                np.abs(c) * K * np.abs(a * c).mean(1, keepdims=True))
        # rows in any order: at most N additions
        e = (N + 8) * U32 * np.abs(gh * c).sum(0)
        if got[4] is not None:
            within("grad_weight", got[4], ref[4], rounded(ref[4], pdt) + e * 1.01)
    if got[0] is not None:
        within("grad_x", got[0], ref[0], rounded(ref[0], dt) + eG * 1.01)
    if b is None:
        return
    k = b if pw is None else b * pr[:, None]
    m = k if pw is None else k * pw
    gate_ = np.ones_like(sn) if gate is None else np.broadcast_to(gate, sn.shape)
    G = np.abs(ref[0])
    if got[2] is not None:
        terms, e = np.abs(scale) * G * np.abs(m), np.abs(scale) * (eG + few * G) * np.abs(m)
        if gate.ndim == 1:
            within("grad_gate", got[2], ref[2], rounded(ref[2], pdt) + 1.01 * (e.sum(0) + (N + 8) * U32 * terms.sum(0)))
        else:
            within("grad_gate", got[2], ref[2], rounded(ref[2], dt) + 1.01 * e)
    e1, err = np.abs(scale * gate_) * G, np.abs(scale * gate_) * (eG + few * G)
    if got[3] is not None:
        within("grad_post_weight", got[3], ref[3], rounded(ref[3], pdt) +
               1.01 * ((err * np.abs(k)).sum(0) + (N + 8) * U32 * (e1 * np.abs(k)).sum(0)))
    if got[1] is None:
        return
    if pw is not None:
        e1, err = e1 * np.abs(pw), err * np.abs(pw)
        err = np.abs(pr[:, None]) * (err + few * (e1 + np.abs(k) * (e1 * np.abs(k)).mean(1, keepdims=True)) +
                                     np.abs(k) * ((err * np.abs(k)).mean(1, keepdims=True) +
                                                  K * (e1 * np.abs(k)).mean(1, keepdims=True)))
    within("grad_branch", got[1], ref[1], rounded(ref[1], dt) + err * 1.01)


def both(N, D, dtype, pdt, gate, post, norm, branch=True, stream=True, scale=0.75, seed=0):
    args = inputs(N, D, dtype, pdt, gate, post, norm, branch, seed)
    got = llp.residual_rms_norm_fwd(*args, scale=scale, eps=EPS)
    check_forward(got, args, scale)
    s, h, pr, r = got
    g = torch.Generator().manual_seed(seed + 1)
    gs, gh = (torch.randn(N, D, generator=g).to(dtype).to(DEV) for _ in range(2))
    gs, gh = gs if stream or not norm else None, gh if norm else None
    grads = llp.residual_rms_norm_bwd(gs, gh, s, *args[1:], pr, r, scale=scale)
    check_backward(grads, gs, gh, s, args, pr, r, scale)
    return args, got, (gs, gh), grads


COMBOS = [c for c in itertools.product(["none", "columns", "rows"], [False, True], [False, True], [False, True])
          if c[3] or (c[0] == "none" and not c[1] and c[2])]


@pytest.mark.parametrize("stream", [True, False])
@pytest.mark.parametrize("gate,post,norm,branch", COMBOS)
def test_every_combination(gate, post, norm, branch, stream):
    both(37, 264, torch.bfloat16, torch.bfloat16, gate, post, norm, branch, stream)
    both(21, 100, torch.float32, torch.float32, gate, post, norm, branch, stream)


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32), (torch.float32, torch.float32)]


@pytest.mark.parametrize("dtype,pdt", TYPES)
@pytest.mark.parametrize("N,D", [(1, 1), (3, 2), (1, 7), (5, 31), (257, 33), (700, 64), (130, 255), (64, 512), (50, 768),
                                 (33, 1001), (65, 1024), (9, 2049), (17, 2688), (20, 4096), (6, 4100), (5, 6001),
                                 (4, 8192), (4, 8200), (3, 16384), (2, 17001)])
def test_sizes_and_types(N, D, dtype, pdt):
    for i, (gate, post) in enumerate((("columns", True), ("rows", True), ("rows", False))):
        both(N, D, dtype, pdt, gate, post, True, seed=i)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [96, 101, 2688])
def test_strided_and_offset_rows(dtype, D):
    N, P = 40, D + 24
    wide = [t for t in inputs(N, P + 3, dtype, dtype, "rows", False, False)[:3]]
    pw, w = inputs(N, D, dtype, dtype, "none", True, True)[3:]
    for first in (0, 1, 3):
        views = [t[:, first:first + D] for t in wide]
        plain = [t.contiguous() for t in views]
        got, want = (llp.residual_rms_norm_fwd(*v, pw, w, scale=0.5) for v in (views, plain))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        s, _, pr, r = want
        room = torch.zeros(N, P + 3, dtype=dtype, device=DEV)
        sv = room[:, first:first + D].copy_(s)
        g = [llp.residual_rms_norm_bwd(a[0], a[1], t, a[1], a[2], pw, w, pr, r, scale=0.5)
             for a, t in ((views, sv), (plain, s))]
        assert all(torch.equal(a, b) for a, b in zip(*g))


def test_a_repeated_row():
    """Stride 0: one gradient row for all (the gradient of a sum)."""
    N, D = 30, 264
    args = inputs(N, D, torch.bfloat16, torch.bfloat16, "columns", True, True)
    s, h, pr, r = llp.residual_rms_norm_fwd(*args)
    one = torch.randn(1, D, device=DEV).to(torch.bfloat16)
    rep = one.expand(N, D)
    got, want = (llp.residual_rms_norm_bwd(g, g, s, *args[1:], pr, r) for g in (rep, rep.contiguous()))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("D", [264, 77])
def test_one_row_for_all_in_the_forward(D):
    """Stride 0 of the stream, the branch or the gate."""
    N = 30
    args = inputs(N, D, torch.bfloat16, torch.bfloat16, "rows", True, True)
    for k in range(3):
        rep = list(args)
        rep[k] = args[k][:1].expand(N, D)
        plain = [t.contiguous() for t in rep]
        for a, b in zip(llp.residual_rms_norm_fwd(*rep), llp.residual_rms_norm_fwd(*plain)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_zeros_and_of_large_values(dtype):
    args = inputs(6, 264, dtype, dtype, "columns", True, True)
    args[0][1] = 0
    args[1][1] = 0          # s is 0: rstd is 1 / sqrt(eps), h is 0
    args[1][2] = 0
    big = 3e4 if dtype == torch.float16 else 1e15
    args[1][3] *= big / 20  # its norm is as any other's
    args[0][4] *= big / 20 if dtype != torch.float16 else 100
    got = llp.residual_rms_norm_fwd(*args, scale=0.5)
    check_forward(got, args, 0.5)
    assert not got[1][1].any() and got[3][1].item() == pytest.approx(EPS ** -0.5, rel=1e-6)
    g = torch.randn(6, 264, device=DEV).to(dtype)
    grads = llp.residual_rms_norm_bwd(g, g, got[0], *args[1:], got[2], got[3], scale=0.5)
    check_backward(grads, g, g, got[0], args, got[2], got[3], 0.5)


def test_a_row_with_nan_or_infinity_spoils_itself_alone():
    args = inputs(8, 520, torch.bfloat16, torch.bfloat16, "columns", True, True)
    clean = llp.residual_rms_norm_fwd(*args)
    args[0][2, 5] = float("nan")
    args[1][5, 7] = float("inf")
    got = llp.residual_rms_norm_fwd(*args)
    keep = [0, 1, 3, 4, 6, 7]
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])
    assert got[1][2].isnan().all() and got[1][5].isnan().any()


def test_subsets_of_the_gradients():
    for gate in ("columns", "rows"):
        args, (s, h, pr, r), (gs, gh), every = both(41, 200, torch.bfloat16, torch.float32, gate, True, True)
        for need in itertools.product([False, True], repeat=5):
            got = llp.residual_rms_norm_bwd(gs, gh, s, *args[1:], pr, r, 0.75, *need)
            for n, a, b in zip(need, got, every):
                assert torch.equal(a, b) if n else a is None


def test_no_rows():
    args = inputs(0, 64, torch.bfloat16, torch.float32, "columns", True, True)
    s, h, pr, r = llp.residual_rms_norm_fwd(*args)
    assert s.shape == h.shape == (0, 64)
    gx, gb, gg, gp, gw = llp.residual_rms_norm_bwd(s, h, s, *args[1:], pr, r)
    assert gx.shape == gb.shape == (0, 64) and not (gg.any() or gp.any() or gw.any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [77, 2688])
def test_rows_do_not_depend_on_the_batch_and_runs_are_the_same(dtype, D):
    args, got, (gs, gh), grads = both(411, D, dtype, dtype, "rows", True, True)
    again = llp.residual_rms_norm_fwd(*args, scale=0.75)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    s, h, pr, r = got
    assert all(torch.equal(a, b) for a, b in zip(grads, llp.residual_rms_norm_bwd(gs, gh, s, *args[1:], pr, r, 0.75)))
    for lo, n in ((0, 1), (5, 64), (200, 211)):
        cut = [t[lo:lo + n] for t in args[:3]] + args[3:]
        part = llp.residual_rms_norm_fwd(*cut, scale=0.75)
        assert all(torch.equal(a, b[lo:lo + n]) for a, b in zip(part, got))
        pg = llp.residual_rms_norm_bwd(gs[lo:lo + n], gh[lo:lo + n], part[0], *cut[1:], part[2], part[3], 0.75)
        assert all(torch.equal(a, b[lo:lo + n]) for a, b in zip(pg[:3], grads[:3]))


def test_many_rows():
    both(16500, 136, torch.bfloat16, torch.bfloat16, "columns", True, True)
    both(5000, 101, torch.float32, torch.float32, "rows", True, True)


def test_autograd():
    N, D = 24, 136
    args = inputs(N, D, torch.float32, torch.float32, "columns", True, True)
    leaves = [t.clone().requires_grad_(True) for t in args]
    s, h = llp.residual_rms_norm(leaves[0].view(4, 6, D), leaves[1].view(4, 6, D), *leaves[2:], scale=0.5)
    assert s.shape == h.shape == (4, 6, D)
    g = torch.randn(4, 6, D, device=DEV)
    (h * g).sum().backward(retain_graph=True)
    s2, _, pr, r = llp.residual_rms_norm_fwd(*args, scale=0.5)
    zero = torch.zeros_like(s2)
    for t, want in zip(leaves, llp.residual_rms_norm_bwd(zero, g.view(N, D), s2, *args[1:], pr, r, 0.5)):
        assert torch.equal(t.grad, want)
        t.grad = None
    s.backward(g)  # nothing comes through the second norm
    for t, want in zip(leaves[:4], llp.residual_rms_norm_bwd(g.view(N, D), None, s2, *args[1:4], None, pr, None, 0.5)):
        assert torch.equal(t.grad, want)
    assert leaves[4].grad is None or not leaves[4].grad.any()


def test_autograd_with_a_gate_for_each_token_and_plain_norm():
    N, D = 12, 72
    args = inputs(N, D, torch.bfloat16, torch.float32, "rows", False, True)
    leaves = [None if t is None else t.clone().requires_grad_(True) for t in args]
    s, h = llp.residual_rms_norm(*[None if t is None else t.view(3, 4, D) if t.dim() == 2 else t for t in leaves])
    h.sum().backward()  # an upstream gradient that repeats one value
    assert leaves[2].grad.shape == (N, D) and leaves[1].grad.shape == (N, D) and leaves[4].grad.dtype == torch.float32
    x = args[0].clone().requires_grad_(True)
    s, h = llp.residual_rms_norm(x, weight=args[4])
    assert s is x
    h.float().square().sum().backward()
    assert x.grad.shape == x.shape
    # a branch without any norm or gate: a plain sum
    s, h = llp.residual_rms_norm(x, args[1])
    assert h is None and torch.equal(s, x + args[1])


def test_refusals():
    x, b, gate, pw, w = inputs(8, 64, torch.bfloat16, torch.bfloat16, "columns", True, True)
    s, h, pr, r = llp.residual_rms_norm_fwd(x, b, gate, pw, w)
    f, bw = llp.residual_rms_norm_fwd, llp.residual_rms_norm_bwd
    for bad, error in ((lambda: f(x), ValueError), (lambda: f(x, None, gate, None, w), ValueError),
                       (lambda: f(x, None, None, pw, w), ValueError), (lambda: f(x, b[:4], weight=w), ValueError),
                       (lambda: f(x, b.float(), weight=w), ValueError), (lambda: f(x, b, gate[:32], weight=w), ValueError),
                       (lambda: f(x, b, gate.float(), pw, w), TypeError), (lambda: f(x, b, gate.half()), TypeError),
                       (lambda: f(x, b, x[:4]), ValueError), (lambda: f(x, b.t(), weight=w), ValueError),
                       (lambda: f(x, b, weight=w, scale=float("nan")), ValueError),
                       (lambda: f(x, b, weight=w.cpu()), ValueError), (lambda: f(x.double(), weight=w), TypeError),
                       (lambda: f(x.as_strided((8, 64), (1, 1)), weight=w), ValueError),
                       (lambda: bw(s, h, s, b, gate, pw, w, pr), ValueError),
                       (lambda: bw(s, None, s, b, gate, pw, w, pr, r), ValueError),
                       (lambda: bw(s, h, s, b, gate, pw, w, None, r), ValueError),
                       (lambda: bw(None, None, s, b), ValueError), (lambda: bw(s, h, s, b, gate, pw, w, pr, r[:4]), ValueError),
                       (lambda: bw(s[:4], h, s, b, gate, pw, w, pr, r), ValueError),
                       (lambda: f(x, weight=w, eps=-1.0), Exception),
                       (lambda: llp.residual_rms_norm(x, b[:, :32], weight=w), ValueError)):
        with pytest.raises(error):
            bad()


def same_places(name, got, ref):
    """NaN and both infinities where the reference has them."""
    got = np64(got)
    assert (np.isnan(got) == np.isnan(ref)).all(), name
    assert (np.where(np.isinf(got), got, 0) == np.where(np.isinf(ref), ref, 0)).all(), name


@pytest.mark.parametrize("N,D,dtype", [(5, 200, torch.bfloat16), (3, 1001, torch.float32), (4, 640, torch.float16),
                                       (3, 5000, torch.float32), (3, 5001, torch.bfloat16), (3, 8200, torch.float32)])
def test_an_infinite_weight_of_the_first_column_stays_there(N, D, dtype):
    args = inputs(N, D, dtype, torch.float32, "columns", True, True)
    g = torch.Generator().manual_seed(5)
    gs, gh = (torch.randn(N, D, generator=g).to(dtype).to(DEV) for _ in range(2))
    clean = llp.residual_rms_norm_fwd(*args)
    grads = llp.residual_rms_norm_bwd(gs, gh, clean[0], *args[1:], clean[2], clean[3])
    for which in (3, 4):
        bad = list(args)
        bad[which] = args[which].clone()
        bad[which][0] = float("inf")
        with np.errstate(invalid="ignore", over="ignore"):
            ref = bo.residual_forward(*(n64(t) for t in bad), 1.0, EPS)
            back = bo.residual_backward(*(n64(t) for t in (gs, gh, clean[0], *bad[1:], clean[2], clean[3])), 1.0)
        got = llp.residual_rms_norm_fwd(*bad)
        for name, a, b in zip(("s", "h", "post_rstd", "rstd"), got, ref):
            same_places(name, a, b)
        assert torch.equal(got[0][:, 1:], clean[0][:, 1:]) and torch.equal(got[2], clean[2])
        got = llp.residual_rms_norm_bwd(gs, gh, clean[0], *bad[1:], clean[2], clean[3])
        same_places("grad_x", got[0], back[0])
        same_places("grad_branch", got[1], back[1])
        same_places("grad_post_weight", got[3], back[3])
        assert torch.equal(got[4], grads[4])
        if which == 3:
            assert torch.equal(got[0], grads[0]) and torch.equal(got[3], grads[3])
