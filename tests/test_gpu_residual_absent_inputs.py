"""The RMS norms around a block on odd 16-bit rows where an input is not there, or not needed: its place in the
kernels' shared memory reads as 0 whatever earlier launches left in it."""
import numpy as np
import pytest
import torch

import lm_head_selected_gb300 as llp
from lm_head_selected_gb300 import _lib
from test_gpu_residual_rms_norm import both, check_backward, inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALVES = [torch.bfloat16, torch.float16]
SHAPES = [(1, 1), (3, 7), (37, 101), (700, 733), (300, 1951), (40, 8232), (9, 12155)]


def shifted(t, by=1):
    """A copy whose rows, of an odd stride, start anywhere."""
    N, D = t.shape
    P = D + 1 - D % 2
    v = torch.zeros(N * P + 64, dtype=t.dtype, device=DEV)[by:by + N * P].view(N, P)[:, :D]
    return v.copy_(t)


def leave_nan_behind(N, D, dtype):
    """Every input there and NaN, in rows laid out as the test's: what the kernels' slots hold afterwards."""
    N = max(N, 3000)
    nan = shifted(torch.full((N, D), float("nan"), dtype=dtype, device=DEV))
    one = torch.ones(D, dtype=dtype, device=DEV)
    st = torch.ones(N, device=DEV)
    for gate in (None, nan):
        llp.residual_rms_norm_fwd(nan, nan, gate, one, one)
        llp.residual_rms_norm_bwd(nan, nan, nan, nan, gate, one, one, st, st)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("N,D", SHAPES)
def test_a_branch_without_gate_and_norm(N, D, norm, dtype):
    args = inputs(N, D, dtype, dtype, "none", False, norm)
    args[:2] = [shifted(t) for t in args[:2]]
    g = torch.Generator().manual_seed(N + D)
    gs, gh = (torch.randn(N, D, generator=g).to(dtype).to(DEV) for _ in range(2))
    gh = gh if norm else None
    s, _, pr, r = llp.residual_rms_norm_fwd(*args, scale=0.75)
    leave_nan_behind(N, D, dtype)
    got = llp.residual_rms_norm_bwd(gs, gh, s, *args[1:], pr, r, scale=0.75)
    check_backward(got, gs, gh, s, args, pr, r, 0.75)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("N,D", SHAPES)
def test_rows_without_a_branch_or_an_upstream_gradient(N, D, dtype):
    leave_nan_behind(N, D, dtype)
    both(N, D, dtype, dtype, "none", False, True, branch=False)
    leave_nan_behind(N, D, dtype)
    both(N, D, dtype, dtype, "none", False, True, branch=False, stream=False)
    leave_nan_behind(N, D, dtype)
    both(N, D, dtype, dtype, "rows", True, True, stream=False)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("N,D", SHAPES)
def test_strides_of_tensors_that_are_not_there_are_not_looked_at(N, D, dtype):
    """Through the C entries, which take a stride beside a NULL."""
    lib, code = _lib.load(), 0 if dtype == torch.bfloat16 else 2
    x, _, _, _, w = inputs(N, D, dtype, dtype, "none", False, True, branch=False)
    _, h, _, r = llp.residual_rms_norm_fwd(x, weight=w)
    gh = torch.randn(N, D, device=DEV).to(dtype)
    want = llp.residual_rms_norm_bwd(None, gh, x, weight=w, rstd=r)
    h2, r2, gx, gw = torch.empty_like(h), torch.empty_like(r), torch.empty_like(x), torch.empty_like(w)
    nbytes = lib.residual_rms_norm_bwd_workspace_bytes(N, D)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    p = [t.data_ptr() for t in (x, w, h2, r2, gh, gx, gw, ws)]
    for odd in (1, 2 * D + 1):
        leave_nan_behind(N, D, dtype)
        _lib.check("fwd", lib.residual_rms_norm_fwd(p[0], D, None, odd, None, odd, 0, None, p[1], code, code, N, D, 1.0, 1e-5,
                                                    None, p[2], None, p[3], stream))
        leave_nan_behind(N, D, dtype)
        _lib.check("bwd", lib.residual_rms_norm_bwd(None, odd, p[4], D, p[0], D, None, odd, None, odd, 0, None, p[1], None, p[3],
                                                    code, code, N, D, 1.0, p[5], None, None, None, p[6], p[7], nbytes,
                                                    stream))
        assert torch.equal(h2, h) and torch.equal(r2, r)
        assert torch.equal(gx, want[0]) and torch.equal(gw, want[4])
    assert np.isfinite(float(gx.float().sum()))
