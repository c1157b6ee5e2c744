"""CPU-only checks of the C ABI of the block operators and the optimizer: exports, workspace sizes, the
status codes of bad arguments before any device call, and what the wrappers refuse."""
import ctypes
import os
import re

import pytest
import torch

import lm_head_selected_gb300 as llp
from lm_head_selected_gb300 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, MISALIGNED, SMALL = 0, -1, -2, -3, -5


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_headers_declare_what_the_library_exports(lib):
    names = set()
    for header in ("gated_linear", "residual_rms_norm", "adamw"):
        with open(os.path.join(ROOT, "include", header + ".h")) as f:
            names |= set(re.findall(rf"^(?:int|size_t) ({header}_[a-z_0-9]+)\s*\(", f.read(), re.M))
    assert names == set(_lib.EXPORTED_BLOCKS)
    for n in names:
        assert hasattr(lib, n)


def test_gated_linear_rejects_bad_arguments_on_host(lib):
    def fwd(x=0x1000, g=0x2000, u=0x3000, dt=0, act=0, N=4, D=8, F=16, y=0x4000, pre=None):
        return lib.gated_linear_fwd(x, g, u, dt, act, N, D, F, y, pre, None)

    def bwd(gy=0x1000, pre=0x2000, x=0x3000, g=0x4000, u=0x5000, dt=0, act=0, N=4, D=8, F=16, gx=0x6000, gg=0x7000,
            gu=0x8000, ws=0x9000, wsb=1 << 40):
        return lib.gated_linear_bwd(gy, pre, x, g, u, dt, act, N, D, F, gx, gg, gu, ws, wsb, None)

    for call in (fwd, bwd):
        assert call(dt=1) == call(dt=3) == call(act=3) == call(act=-1) == call(N=-1) == call(N=1 << 31) == SHAPE
        assert call(D=0) == call(D=4) == call(D=12) == call(F=0) == call(F=20) == call(D=1 << 30) == call(F=1 << 30) == SHAPE
    assert fwd(x=None) == fwd(g=None) == fwd(u=None) == fwd(y=None) == NULL
    assert fwd(x=0x1002) == fwd(g=0x2008) == fwd(u=0x3008) == fwd(y=0x4008) == fwd(pre=0x5002) == MISALIGNED
    assert fwd(N=0, x=None, g=None, u=None, y=None) == OK
    assert bwd(gy=None) == bwd(pre=None) == bwd(x=None) == bwd(g=None) == bwd(u=None) == bwd(ws=None) == NULL
    assert bwd(gy=0x1008) == bwd(pre=0x2008) == bwd(gx=0x6008) == bwd(gu=0x8008) == bwd(ws=0x9008) == MISALIGNED
    need = lib.gated_linear_bwd_workspace_bytes(4, 8, 16)
    assert need >= 4 * 2 * 16 * 2 and bwd(wsb=need - 1) == SMALL
    assert bwd(gx=None, gg=None, gu=None) == OK
    assert bwd(N=0, gg=None, gu=None) == OK
    ask = lib.gated_linear_bwd_workspace_bytes
    assert ask(0, 8, 16) == ask(4, 7, 16) == ask(4, 8, 17) == ask(1 << 31, 8, 16) == 0


def test_residual_rms_norm_rejects_bad_arguments_on_host(lib):
    def fwd(x=0x1000, xs=8, b=0x2000, bs=8, g=0x3000, gs=8, kind=1, pw=0x4000, w=0x5000, dt=0, pdt=0, N=4, D=8,
            scale=1.0, eps=1e-5, s=0x6000, h=0x7000, pr=0x8000, r=0x9000):
        return lib.residual_rms_norm_fwd(x, xs, b, bs, g, gs, kind, pw, w, dt, pdt, N, D, scale, eps, s, h, pr, r, None)

    def bwd(gs=0x1000, gss=8, gh=0x2000, ghs=8, s=0x3000, ss=8, b=0x4000, bs=8, g=0x5000, gts=8, kind=1, pw=0x6000,
            w=0x7000, pr=0x8000, r=0x9000, dt=0, pdt=0, N=4, D=8, scale=1.0, gx=0xA000, gb=0xB000, gg=0xC000,
            gp=0xD000, gw=0xE000, ws=0xF000, wsb=1 << 40):
        return lib.residual_rms_norm_bwd(gs, gss, gh, ghs, s, ss, b, bs, g, gts, kind, pw, w, pr, r, dt, pdt, N, D,
                                         scale, gx, gb, gg, gp, gw, ws, wsb, None)

    nan, inf = float("nan"), float("inf")
    for call in (fwd, bwd):
        assert call(dt=3) == call(pdt=2) == call(dt=1, pdt=0) == call(N=-1) == call(D=0) == call(D=1 << 24) == SHAPE
        assert call(kind=3) == call(kind=0) == call(scale=nan) == call(scale=inf) == call(bs=7) == SHAPE
        assert call(kind=2, g=0x3000, **({"gs": 7} if call is fwd else {"gts": 7})) == SHAPE
        assert call(g=None) == call(b=None) == NULL
    assert fwd(xs=7) == fwd(eps=-1.0) == fwd(eps=nan) == SHAPE
    assert fwd(x=None) == fwd(s=None) == fwd(h=None) == fwd(pr=None) == fwd(r=None) == NULL
    assert fwd(b=None, g=None, kind=0, pw=None, w=None, s=None, h=None, pr=None, r=None) == NULL
    assert fwd(b=None, g=None, kind=0, pw=None, pr=None) == NULL  # s without a branch
    assert fwd(x=0x1001) == fwd(b=0x2001) == fwd(g=0x3001) == fwd(pdt=1, g=0x3002) == fwd(h=0x7001) == MISALIGNED
    assert fwd(pr=0x8002) == fwd(s=0x6001) == fwd(w=0x5001) == MISALIGNED
    assert fwd(N=0, x=None, b=None, g=None, s=None, h=None, pr=None, r=None) == OK
    assert bwd(gss=7) == bwd(ghs=7) == bwd(ss=7) == SHAPE
    assert bwd(gh=None) == bwd(s=None) == bwd(pr=None) == bwd(r=None) == bwd(ws=None) == NULL
    assert bwd(gs=None, w=None, gw=None) == NULL  # no gradient comes in
    assert bwd(w=None) == bwd(pw=None) == bwd(g=None, kind=0) == NULL  # gradients of what is not there
    assert bwd(gs=0x1001) == bwd(gb=0xB001) == bwd(gw=0xE001) == bwd(ws=0xF008) == bwd(r=0x9002) == MISALIGNED
    need = lib.residual_rms_norm_bwd_workspace_bytes(4, 8)
    assert need > 0 and bwd(wsb=need - 1) == SMALL
    assert bwd(gx=None, gb=None, gg=None, gp=None, gw=None) == OK
    ask = lib.residual_rms_norm_bwd_workspace_bytes
    assert ask(0, 8) == ask(4, 0) == ask(1 << 31, 8) == ask(4, 1 << 24) == 0


def _adamw(lib, bits=32, n=8, **over):
    a = dict(count=1, p=0x1000, g=0x2000, m=0x3000, v=0x4000, ms=0x5000 if bits == 8 else None,
             vs=0x6000 if bits == 8 else None, master=None, n=n, pd=0, gd=0, decay=0.0, bits=bits, lr=1e-3, b1=0.9,
             b2=0.99, eps=1e-8, step=1, dstep=None, dlr=None, gscale=None)
    a.update(over)

    def one(v):
        return (ctypes.c_void_p * 1)(v)

    scales = [one(a[k]) if a["bits"] == 8 else None for k in ("ms", "vs")]
    return lib.adamw_step(a["count"], one(a["p"]), one(a["g"]), one(a["m"]), one(a["v"]), *scales,
                          one(a["master"]) if a["master"] else None, (ctypes.c_int64 * 1)(a["n"]),
                          (ctypes.c_int32 * 1)(a["pd"]), (ctypes.c_int32 * 1)(a["gd"]),
                          (ctypes.c_double * 1)(a["decay"]), a["bits"], a["lr"], a["b1"], a["b2"], a["eps"], a["step"],
                          a["dstep"], a["dlr"], a["gscale"], None)


def test_adamw_rejects_bad_arguments_on_host(lib):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(count=-1), dict(bits=16), dict(pd=3), dict(pd=0, gd=2), dict(pd=1, gd=0), dict(n=-1),
                dict(n=1 << 50), dict(decay=nan), dict(lr=inf), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0),
                dict(b2=nan), dict(eps=-1.0), dict(eps=inf), dict(step=0), dict(step=-1, dstep=0x9000)):
        assert _adamw(lib, **bad) == SHAPE, bad
    for bad in (dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(bits=8, ms=None, vs=0x10),
                dict(bits=8, ms=0x10, vs=None)):
        assert _adamw(lib, **bad) == NULL, bad
    for bad in (dict(p=0x1001), dict(g=0x2001), dict(m=0x3002), dict(v=0x4001), dict(master=0x7002),
                dict(pd=1, gd=1, p=0x1002), dict(gd=1, g=0x2002), dict(bits=8, ms=0x12, vs=0x10),
                dict(dstep=0x9004), dict(dlr=0x9002), dict(gscale=0x9001)):
        assert _adamw(lib, **bad) == MISALIGNED, bad
    assert _adamw(lib, count=0) == _adamw(lib, n=0, p=None, g=None, m=None, v=None) == OK


def test_python_wrappers_fail_closed_without_gpu():
    x, w = torch.zeros(4, 8), torch.zeros(16, 8)
    v = torch.zeros(8)
    for call in (lambda: llp.gated_linear_fwd(x, w, w), lambda: llp.gated_linear_bwd(x, x, x, w, w),
                 lambda: llp.gated_linear(x, w, w), lambda: llp.gated_linear(None, w, w),
                 lambda: llp.residual_rms_norm_fwd(x, weight=v), lambda: llp.residual_rms_norm(x, weight=v),
                 lambda: llp.residual_rms_norm_bwd(None, x, x, weight=v, rstd=v), lambda: llp.residual_rms_norm(None),
                 lambda: llp.adamw_state([x]), lambda: llp.adamw_step([x], [x], [x], [x], 1),
                 lambda: llp.adamw_state([None])):
        with pytest.raises(ValueError):
            call()


def test_adamw_wrapper_refuses_before_it_looks_at_tensors():
    for bad in (dict(step=0), dict(step=1, betas=(1.0, 0.9)), dict(step=1, lr=float("nan")), dict(step=1, eps=-1.0),
                dict(step=1, exp_avg_scale=[])):
        with pytest.raises(ValueError):
            llp.adamw_step([None], [None], [None], [None], **bad)
    with pytest.raises(ValueError):
        llp.adamw_step([None], [], [], [], 1)
    llp.adamw_step([], [], [], [], 1)  # nothing to do
