"""Layer norm on rows far from zero: the gradients with exact statistics, constant rows,
rows of two neighbouring values."""
import numpy as np
import pytest
import torch

from operator_bounds import DTYPES, U32, np64, rounded, sum_depth, within

pytestmark = pytest.mark.gpu

# in the pipelined kernel with one to four vectors per thread, and in the one for wider rows
WIDTHS = [24, 40, 1000, 1001, 2688, 4104, 8200, 9001, 16392]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from lm_head_selected_gb300 import build
    build.build()


def _offset_rows(D, g):
    """Rows with an offset, in values that all types hold where they are not random."""
    pair = 300.0 + 2.0 * torch.randint(0, 2, (D,), generator=g)
    return torch.stack([torch.full((D,), 1000.0), pair, 1000 + torch.randn(D, generator=g),
                        30 + torch.randn(D, generator=g), torch.full((D,), -0.375), torch.randn(D, generator=g)])


def _check_gradients(x, gy, w, eps=1e-5):
    """The gradients against the formula in 64 bits, with the fp32 statistics that they are given.
    The bound leaves no room for an error of the mean: h = (x - mean) * rstd has two roundings."""
    import lm_head_selected_gb300 as llp
    dt, (N, D) = x.dtype, x.shape
    xn, gn = np64(x), np64(gy)
    wn = np.ones(D) if w is None else np64(w)
    mean = torch.from_numpy(xn.mean(1)).float()
    rstd = torch.from_numpy(1.0 / np.sqrt(((xn - np64(mean)[:, None]) ** 2).mean(1) + eps)).float()
    gx, gw, gb = llp.layer_norm_bwd(gy.cuda(), x.cuda(), mean.cuda(), rstd.cuda(), None if w is None else w.cuda(),
                                    param_dtype=torch.float32)
    m, r = np64(mean)[:, None], np64(rstd)[:, None]
    h = (xn - m) * r
    a = gn * wn
    gx_ref = r * (a - a.mean(1, keepdims=True) - h * (a * h).mean(1, keepdims=True))
    h, a = np.abs(h), np.abs(a)
    dh = 2 * U32 * h
    k = sum_depth(D) * U32
    s1, s2 = a.mean(1, keepdims=True), (a * h).mean(1, keepdims=True)
    ds1 = (k + 3 * U32) * s1
    ds2 = (k + 4 * U32) * s2 + (a * dh).mean(1, keepdims=True)
    slack = 1 + 1e-2  # second-order terms
    egx = r * (ds1 + h * ds2 + dh * s2 + 6 * U32 * (a + s1 + h * s2))
    kn = (N + 8) * U32
    within("grad_weight", gw, (gn * (xn - m) * r).sum(0),
           slack * (rounded((gn * (xn - m) * r).sum(0), torch.float32) + kn * (np.abs(gn) * h).sum(0)
                    + (np.abs(gn) * dh).sum(0)))
    within("grad_x", gx, gx_ref, slack * (rounded(gx_ref, dt) + egx))
    within("grad_bias", gb, gn.sum(0), slack * (rounded(gn.sum(0), torch.float32) + kn * np.abs(gn).sum(0)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_gradients_with_exact_statistics(dtype, D):
    g = torch.Generator().manual_seed(D)
    x = _offset_rows(D, g).to(dtype)
    gy = torch.randn(x.shape, generator=g).to(dtype)
    _check_gradients(x, gy, 1 + 0.3 * torch.randn(D, generator=g))
    for row in (0, 1):  # by themselves: no other row's h to hide behind
        _check_gradients(x[row:row + 1], gy[row:row + 1], None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", WIDTHS)
def test_gradients_of_a_constant_row_whose_mean_times_rstd_is_past_the_largest_float(dtype, D):
    g = torch.Generator().manual_seed(D)
    x = torch.full((2, D), 2.0 ** 123)
    x[1] = torch.randn(D, generator=g)
    _check_gradients(x.to(dtype), torch.randn(2, D, generator=g).to(dtype), 1 + 0.3 * torch.randn(D, generator=g))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", WIDTHS + [7, 49, 383, 769])
def test_forward_of_constant_rows(dtype, D):
    """Values of at most nine bits: sums of up to 2^15 of them are exact in fp32, so the mean, a
    quotient that fits, has to be exact too, and y is the bias."""
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(D)
    values = torch.tensor([3000.0, 1000.0, -0.375, 7.0, 0.0, -491.0]).to(dtype)
    x = values[:, None].expand(-1, D).contiguous().cuda()
    w, b = (1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda(), torch.randn(D, generator=g).to(dtype).cuda()
    y, mean, rstd = llp.layer_norm_fwd(x, w, b)
    assert torch.equal(mean.cpu(), values.float())
    assert torch.equal(y, b.expand_as(y)) and not llp.layer_norm_fwd(x)[0].any()
    r = 1 / np.sqrt(float(np.float32(1e-5)))
    within("rstd", rstd, np.full(len(values), r), 4 * U32 * r)  # two units in the last place


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", WIDTHS + [7, 49, 383, 769])
def test_gradients_of_one_upstream_value_per_row(dtype, D):
    """grad_x without a weight: a - mean(a) is 0, and so is all of grad_x for a constant row of x;
    for another one -h * mean(a h) * rstd is left, of the size of the rounding of a sum of h."""
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(D)
    a = torch.tensor([1.0, 491.0, -0.375, 3.0, 7.0]).to(dtype)
    x = torch.full((5, D), 5.0)
    x[3:] = torch.randn(2, D, generator=g)
    x = x.to(dtype)
    xn, an = np64(x), np64(a)[:, None]
    mean = torch.from_numpy(xn.mean(1)).float()
    rstd = torch.from_numpy(1.0 / np.sqrt(((xn - np64(mean)[:, None]) ** 2).mean(1) + 1e-5)).float()
    gx = llp.layer_norm_bwd(a[:, None].expand(-1, D).contiguous().cuda(), x.cuda(), mean.cuda(), rstd.cuda(),
                            need_weight=False, need_bias=False)[0]
    assert not gx[:3].any()
    m, r = np64(mean)[:, None], np64(rstd)[:, None]
    h = (xn - m) * r
    ref = -h * (an * h).mean(1, keepdims=True) * r
    # the sum of a h, the roundings of h and of the terms, one of the result
    s2 = np.abs(an * h).mean(1, keepdims=True)
    err = r * np.abs(h) * (sum_depth(D) + 8) * U32 * s2
    within("grad_x", gx, ref, (1 + 1e-2) * (rounded(ref, dtype) + err))
