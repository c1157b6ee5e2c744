"""CPU-only checks of the C ABI of the operators around the head: exports,
workspace sizes, and the status codes of bad arguments, all before any device
call."""
import ctypes
import os
import re

import pytest

from lm_head_selected_gb300 import _lib, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, MISALIGNED, SMALL = 0, -1, -2, -3, -5


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_headers_declare_what_the_library_exports(lib):
    names = set()
    for header in ("embedding", "layer_norm", "dropout"):
        with open(os.path.join(ROOT, "include", header + ".h")) as f:
            names |= set(re.findall(rf"^(?:int|size_t) ({header}_[a-z_0-9]+)\s*\(", f.read(), re.M))
    assert names == set(_lib.EXPORTED_OPERATORS)
    for n in names:
        assert hasattr(lib, n)


def test_embedding_rejects_bad_arguments_on_host(lib):
    def fwd(t=0x1000, w=0x2000, dt=0, N=4, V=10, D=8, out=0x3000):
        return lib.embedding_fwd(t, w, dt, N, V, D, 1.0, -100, out, None)

    def bwd(t=0x1000, g=0x2000, stride=8, dt=0, N=4, V=10, D=8, acc=0, gw=0x3000, ws=0x4000, wsb=1 << 40):
        return lib.embedding_bwd(t, g, stride, dt, N, V, D, 1.0, -100, acc, gw, ws, wsb, None)

    assert fwd(dt=3) == fwd(N=-1) == fwd(V=0) == fwd(D=0) == fwd(N=1 << 31) == fwd(V=1 << 31) == SHAPE
    assert fwd(D=1 << 24) == SHAPE
    assert fwd(t=None) == fwd(w=None) == fwd(out=None) == NULL
    assert fwd(t=0x1004) == fwd(w=0x2001) == fwd(out=0x3001) == fwd(dt=1, w=0x2002) == MISALIGNED
    assert fwd(N=0, t=None, out=None) == OK
    assert bwd(dt=-1) == bwd(N=-1) == bwd(V=0) == bwd(D=0) == bwd(stride=7) == bwd(stride=-8) == SHAPE
    assert bwd(t=None) == bwd(g=None) == bwd(gw=None) == bwd(ws=None) == NULL
    assert bwd(t=0x1004) == bwd(g=0x2001) == bwd(gw=0x3001) == bwd(ws=0x4008) == MISALIGNED
    need = lib.embedding_bwd_workspace_bytes(4, 10, 8)
    assert need > 0 and bwd(wsb=need - 1) == SMALL
    assert bwd(N=0, acc=1, t=None, g=None, gw=None, ws=None) == OK
    assert bwd(N=0, gw=None) == NULL
    ask = lib.embedding_bwd_workspace_bytes
    assert ask(0, 10, 8) == ask(4, 0, 8) == ask(4, 10, 0) == ask(1 << 31, 10, 8) == 0


def test_layer_norm_rejects_bad_arguments_on_host(lib):
    def fwd(x=0x1000, stride=8, dt=0, N=4, D=8, w=0x2000, b=0x3000, pdt=0, eps=1e-5, y=0x4000, m=0x5000, r=0x6000):
        return lib.layer_norm_fwd(x, stride, dt, N, D, w, b, pdt, eps, y, m, r, None)

    def bwd(gy=0x1000, gs=8, x=0x2000, xs=8, dt=0, N=4, D=8, m=0x3000, r=0x4000, w=0x5000, pdt=0, gx=0x6000,
            gw=0x7000, gb=0x8000, ws=0x9000, wsb=1 << 40):
        return lib.layer_norm_bwd(gy, gs, x, xs, dt, N, D, m, r, w, pdt, gx, gw, gb, ws, wsb, None)

    assert fwd(dt=3) == fwd(dt=0, pdt=2) == fwd(dt=1, pdt=0) == fwd(N=-1) == fwd(D=0) == fwd(stride=7) == SHAPE
    assert fwd(eps=-1.0) == fwd(eps=float("nan")) == fwd(eps=float("inf")) == fwd(D=1 << 24) == SHAPE
    assert fwd(x=None) == fwd(y=None) == fwd(m=None) == fwd(r=None) == NULL
    assert fwd(x=0x1001) == fwd(w=0x2001) == fwd(b=0x3001) == fwd(pdt=1, w=0x2002) == fwd(m=0x5002) == MISALIGNED
    assert fwd(N=0, x=None, y=None, m=None, r=None) == OK
    assert bwd(dt=3) == bwd(pdt=2) == bwd(gs=7) == bwd(xs=1) == bwd(N=1 << 31) == SHAPE
    assert bwd(gy=None) == bwd(x=None) == bwd(m=None) == bwd(r=None) == bwd(ws=None) == NULL
    assert bwd(gy=0x1001) == bwd(gx=0x6001) == bwd(gw=0x7001) == bwd(r=0x4002) == bwd(ws=0x9008) == MISALIGNED
    need = lib.layer_norm_bwd_workspace_bytes(4, 8)
    assert need > 0 and bwd(wsb=need - 1) == SMALL
    assert bwd(gx=None, gw=None, gb=None) == OK
    assert bwd(N=0, gw=None, gb=None) == OK
    ask = lib.layer_norm_bwd_workspace_bytes
    assert ask(0, 8) == ask(4, 0) == ask(1 << 31, 8) == ask(4, 1 << 24) == 0


def test_dropout_rejects_bad_arguments_on_host(lib):
    def fwd(x=0x1000, r=0x2000, dt=0, n=100, p=0.1, off=None, y=0x3000):
        return lib.dropout_fwd(x, r, dt, n, p, 1, 2, off, y, None)

    assert fwd(dt=3) == fwd(n=-1) == fwd(n=1 << 62) == fwd(p=-0.1) == fwd(p=1.5) == fwd(p=float("nan")) == SHAPE
    assert fwd(x=None) == fwd(y=None) == NULL
    assert fwd(x=0x1001) == fwd(r=0x2001) == fwd(y=0x3001) == fwd(dt=1, y=0x3002) == fwd(off=0x4004) == MISALIGNED
    assert fwd(n=0, x=None, r=None, y=None) == OK
    assert lib.dropout_bwd(None, 0, 8, 0.1, 1, 2, None, 0x3000, None) == NULL
    assert lib.dropout_bwd(0x1000, 0, 0, 0.1, 1, 2, None, None, None) == OK


def test_workspace_sizes(lib):
    # the sort's arrays are linear in the tokens and the table's rows; the partial sums stay
    # below one fp32 row per 16 tokens
    n, v, d = 65600, 131072, 2688
    assert lib.embedding_bwd_workspace_bytes(n, v, d) <= 64 * n + 16 * v + (n // 16 + 64) * d * 4 + (1 << 20)
    assert lib.layer_norm_bwd_workspace_bytes(n, d) <= 4096 * d * 8 + (1 << 20)


def test_python_wrappers_fail_closed_without_gpu():
    import torch
    import lm_head_selected_gb300 as llp
    x, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: llp.embedding_fwd(t, x), lambda: llp.embedding_bwd(x, t, 4), lambda: llp.layer_norm_fwd(x),
                 lambda: llp.layer_norm_bwd(x, x, x[:, 0], x[:, 0]), lambda: llp.dropout_fwd(x, 0.1, 1),
                 lambda: llp.dropout_bwd(x, 0.1, 1), lambda: llp.embedding(t, x), lambda: llp.layer_norm(x),
                 lambda: llp.dropout(x, 0.1, 1)):
        with pytest.raises(ValueError):
            call()
    assert ctypes.sizeof(ctypes.c_void_p) == 8
