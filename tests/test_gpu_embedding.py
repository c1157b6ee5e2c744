"""The token embedding and its gradient against the FP64 oracle: types, sizes,
repeated and invalid tokens, strides, alignment, accumulation, invariance."""
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


def _tokens(kind, N, V, g):
    if kind == "uniform":
        t = torch.randint(0, V, (N,), generator=g)
    elif kind == "zipf":
        t = (torch.exp(torch.rand(N, generator=g, dtype=torch.float64) * np.log(V + 1.0)).long() - 1).clamp(0, V - 1)
    elif kind == "one":
        t = torch.full((N,), V - 1)
    elif kind == "last_rows":
        t = V - 1 - torch.randint(0, min(V, 3), (N,), generator=g)
    elif kind == "descending":
        t = (V - 1 - torch.arange(N)) % V
    else:
        assert kind == "invalid"
        return torch.tensor([-100, V, -1, V + 5, 1 << 40, -(1 << 40)])[torch.arange(N) % 6]
    if N >= 8 and kind in ("uniform", "zipf"):
        t[1], t[4], t[6] = -100, V, -7
    return t


def _bwd_ref(g, t, V, scale, ignore, base):
    """Oracle gradient and its bound (in place of the output type's rounding)."""
    ref = mo.embedding_backward(g, t, V, scale, ignore, base)
    size = mo.embedding_backward(np.abs(g), t, V, abs(scale), ignore, None if base is None else np.abs(base))
    count = mo.embedding_backward(np.ones((len(t), 1)), t, V, 1.0, ignore)
    return ref, (count + 4) * U32 * size


def _check_bwd(g, t, V, dtype, scale=1.0, ignore=-100, base=None):
    import lm_head_selected_gb300 as llp
    out = None if base is None else base.cuda()
    gw = llp.embedding_bwd(g.cuda() if not g.is_cuda else g, t.cuda(), V, scale, ignore, out=out,
                           accumulate=base is not None)
    ref, err = _bwd_ref(np64(g), t.numpy(), V, float(np.float32(scale)), ignore, None if base is None else np64(base))
    assert gw.dtype == dtype and gw.shape == (V, g.shape[1])
    within("grad_weight", gw, ref, rounded(ref, dtype) * (1 + 1e-3) + err)
    named = np.zeros(V, dtype=bool)
    tn = t.numpy()
    named[tn[(tn >= 0) & (tn < V) & (tn != ignore)]] = True
    rest = np64(gw)[~named]
    assert np.array_equal(rest, np.zeros_like(rest) if base is None else np64(base)[~named])
    return gw


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,D,V", [(1, 1, 1), (7, 64, 30), (33, 1001, 100), (300, 264, 5000), (5, 2688, 131),
                                   (1000, 24, 17), (64, 4100, 64)])
def test_forward(dtype, N, D, V):
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(N + D)
    w = torch.randn(V, D, generator=g).to(dtype)
    t = _tokens("uniform", N, V, g)
    for scale in (1.0, 51.846):
        out = llp.embedding_fwd(t.cuda(), w.cuda(), scale)
        ref = mo.embedding_forward(t.numpy(), np64(w), float(np.float32(scale)))
        assert out.dtype == dtype
        within("out", out, ref, rounded(ref, dtype) * (1 + 1e-3) + U32 * np.abs(ref))
        if scale == 1.0:
            assert np.array_equal(np64(out), ref)


def test_forward_does_not_read_for_invalid_tokens_and_keeps_nan_rows_apart():
    import lm_head_selected_gb300 as llp
    w = torch.full((10, 128), NAN, dtype=torch.bfloat16)
    w[3] = 2.0
    t = torch.tensor([3, -100, 10, -1, 1 << 40, -(1 << 40), 3, 4])
    out = llp.embedding_fwd(t.cuda(), w.cuda(), 0.5, ignore_index=4).float().cpu()
    assert torch.all(out[[0, 6]] == 1.0) and torch.all(out[[1, 2, 3, 4, 5, 7]] == 0.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["uniform", "zipf", "one", "last_rows", "descending", "invalid"])
@pytest.mark.parametrize("N,D,V", [(1, 1, 1), (6, 8, 3), (65, 40, 9), (257, 264, 1000), (1000, 129, 50),
                                   (2049, 72, 300)])
def test_backward(dtype, kind, N, D, V):
    g = torch.Generator().manual_seed(3 * N + D)
    t = _tokens(kind, N, V, g)
    go = torch.randn(N, D, generator=g).to(dtype)
    _check_bwd(go, t, V, dtype)
    _check_bwd(go, t, V, dtype, scale=3.5, base=torch.randn(V, D, generator=g).to(dtype))


@pytest.mark.parametrize("N", [0, 1, 2, 31, 63, 64, 65, 127, 128, 129, 4095, 4096, 4097, 8193, 20000])
def test_backward_counts_around_the_piece_lengths(N):
    """One row named N times, next to rows named once: segments of every number of pieces."""
    g = torch.Generator().manual_seed(N)
    V, D = 40, 16
    t = torch.cat([torch.full((N,), 7), torch.arange(V), torch.full((3,), -100)])
    t = t[torch.randperm(len(t), generator=g)]
    _check_bwd(torch.randn(len(t), D, generator=g), t, V, torch.float32)


@pytest.mark.parametrize("N", [511, 512, 513, 544, 545, 16383, 16384, 16385, 131073])
def test_backward_counts_around_the_group_lengths(N):
    """Rows whose pieces are joined at once, in groups, and with the next length of a piece;
    a second long row begins where the first one ends."""
    g = torch.Generator().manual_seed(N)
    V, D = 3, 24
    t = torch.cat([torch.full((N,), 1), torch.full((33,), 2), torch.tensor([0, -100])])
    t = t[torch.randperm(len(t), generator=g)]
    base = torch.randn(V, D, generator=g)
    go = torch.randn(len(t), D, generator=g)
    _check_bwd(go, t, V, torch.float32)
    _check_bwd(go, t, V, torch.float32, scale=0.5, base=base)


@pytest.mark.parametrize("V", [1, 2, 255, 256, 257, 1023, 4097, 131072])
@pytest.mark.parametrize("N", [3, 700, 5000])
def test_backward_table_sizes(N, V):
    g = torch.Generator().manual_seed(N + V)
    for kind in ("uniform", "zipf"):
        _check_bwd(torch.randn(N, 8, generator=g).to(torch.bfloat16), _tokens(kind, N, V, g), V, torch.bfloat16)


def test_backward_ignores_a_valid_id_and_never_reads_ignored_rows():
    g = torch.Generator().manual_seed(5)
    N, D, V = 200, 48, 12
    t = _tokens("uniform", N, V, g)
    go = torch.randn(N, D, generator=g)
    ok = (t >= 0) & (t < V) & (t != 5)
    clean = go.clone()
    go[~ok] = NAN
    clean[~ok] = 0.0
    import lm_head_selected_gb300 as llp
    a = llp.embedding_bwd(go.cuda(), t.cuda(), V, 1.0, ignore_index=5)
    b = llp.embedding_bwd(clean.cuda(), t.cuda(), V, 1.0, ignore_index=5)
    assert torch.equal(a, b) and torch.all(a[5] == 0) and torch.all(torch.isfinite(a))


@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_strides_and_alignment(dtype):
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(6)
    N, V, D = 150, 40, 64
    t = _tokens("uniform", N, V, g)
    buf = torch.randn(N, 200, generator=g).to(dtype).cuda()
    for c0 in (0, 1, 8, 129):
        view = buf[:, c0:c0 + D]
        want = llp.embedding_bwd(view.contiguous(), t.cuda(), V)
        assert torch.equal(llp.embedding_bwd(view, t.cuda(), V), want)
        _check_bwd(view, t, V, dtype)
    row = buf[:1, :D].expand(N, D)  # one row for every token
    assert torch.equal(llp.embedding_bwd(row, t.cuda(), V), llp.embedding_bwd(row.contiguous(), t.cuda(), V))
    # tables and outputs that start at an odd element
    flat = torch.zeros(V * D + 1, dtype=dtype, device="cuda")
    out = flat[1:].view(V, D)
    llp.embedding_bwd(view, t.cuda(), V, out=out)
    assert torch.equal(out, want) and flat[0] == 0
    w = torch.randn(V * D + 1, generator=g).to(dtype).cuda()
    table = w[1:].view(V, D)
    assert torch.equal(llp.embedding_fwd(t.cuda(), table, 2.0), llp.embedding_fwd(t.cuda(), table.clone(), 2.0))


def test_backward_row_depends_on_its_own_tokens_alone_and_repeats():
    """A row's bits are the same whatever the other tokens are, in every run."""
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(7)
    N, D, V = 9000, 136, 700
    t = _tokens("zipf", N, V, g)
    go = torch.randn(N, D, generator=g).cuda()
    full = llp.embedding_bwd(go, t.cuda(), V)
    for _ in range(3):
        assert torch.equal(full, llp.embedding_bwd(go, t.cuda(), V))
    for v in (0, 1, 2, 50, 699):
        only = torch.where(t == v, t, torch.full_like(t, -100))
        assert torch.equal(full[v], llp.embedding_bwd(go, only.cuda(), V)[v])
        sel = torch.nonzero(t == v).flatten()
        if len(sel):
            assert torch.equal(full[v], llp.embedding_bwd(go[sel.cuda()], t[sel].cuda(), V)[v])


def test_backward_workspace_is_not_read_before_it_is_written():
    import lm_head_selected_gb300 as llp
    from lm_head_selected_gb300 import _lib
    g = torch.Generator().manual_seed(8)
    N, D, V = 3000, 40, 90
    t, go = _tokens("zipf", N, V, g).cuda(), torch.randn(N, D, generator=g).cuda()
    nbytes = _lib.load().embedding_bwd_workspace_bytes(N, V, D)
    want = llp.embedding_bwd(go, t, V)
    for fill in (0, 255, 127):
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(want, llp.embedding_bwd(go, t, V, workspace=ws))
        assert torch.equal(want, llp.embedding_bwd(go, t, V, workspace=ws))  # on its own leftovers


def test_no_tokens():
    import lm_head_selected_gb300 as llp
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    w = torch.ones(5, 8, device="cuda")
    assert llp.embedding_fwd(t, w).shape == (0, 8)
    assert torch.all(llp.embedding_bwd(torch.zeros(0, 8, device="cuda"), t, 5) == 0)
    assert torch.all(llp.embedding_bwd(torch.zeros(0, 8, device="cuda"), t, 5, out=w, accumulate=True) == 1)


def test_offsets_past_32_bits():
    """A table of more than 2^31 elements, named at both of its ends."""
    import lm_head_selected_gb300 as llp
    V, D = 70001, 32768
    t = torch.tensor([V - 1, 0, 65536, V - 1, 123], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    go = torch.randn(5, D, device="cuda", generator=g).to(torch.bfloat16)
    gw = llp.embedding_bwd(go, t, V)
    assert torch.equal(gw[65536], go[2]) and torch.equal(gw[0], go[1]) and torch.equal(gw[123], go[4])
    assert torch.equal(gw[V - 1], (go[0].float() + go[3].float()).to(torch.bfloat16))
    assert int((gw != 0).any(1).sum()) == 4
    assert torch.equal(llp.embedding_fwd(t, gw)[[0, 2]], gw[t[[0, 2]]])


def test_autograd_and_finite_differences():
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(10)
    w = torch.randn(9, 6, generator=g).cuda().requires_grad_(True)
    t = torch.randint(0, 9, (2, 5), generator=g).cuda()
    c = torch.randn(2, 5, 6, generator=g).cuda()
    loss = lambda w_: (llp.embedding(t, w_, 0.25).double() * c.double()).sum()  # noqa: E731
    loss(w).backward()
    assert llp.embedding(t, w, 0.25).shape == (2, 5, 6)
    for i, j in ((0, 0), (3, 5), (8, 2)):
        d = torch.zeros_like(w)
        d[i, j] = 0.5
        # linear in w: the central difference is exact up to fp32 rounding of ten products near 1
        diff = float((loss(w.detach() + d) - loss(w.detach() - d)) / 1.0)
        assert abs(diff - float(w.grad[i, j])) <= 20 * 4 * U32
    llp.embedding(t, w).sum().backward()  # an expanded upstream gradient


def test_on_another_stream_and_in_a_graph():
    import lm_head_selected_gb300 as llp
    g = torch.Generator().manual_seed(11)
    N, D, V = 500, 64, 77
    t = _tokens("zipf", N, V, g).cuda()
    go = torch.randn(N, D, generator=g).cuda()
    want = llp.embedding_bwd(go, t, V)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = llp.embedding_bwd(go, t, V)
        fwd = llp.embedding_fwd(t, got)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    st, sg = t.clone(), go.clone()
    with torch.cuda.graph(graph):
        out = llp.embedding_bwd(sg, st, V)
        fw = llp.embedding_fwd(st, out)
    for k in range(2):
        st.copy_(t.roll(k))
        sg.copy_(go * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, llp.embedding_bwd(go * (k + 1), t.roll(k), V))
        assert torch.equal(fw, llp.embedding_fwd(t.roll(k), out))
    assert torch.equal(fwd, llp.embedding_fwd(t, want))


def test_refusals():
    import lm_head_selected_gb300 as llp
    w = torch.zeros(4, 8, device="cuda")
    t = torch.zeros(3, dtype=torch.int64, device="cuda")
    g = torch.zeros(3, 8, device="cuda")
    for bad in (lambda: llp.embedding_fwd(t.cpu(), w), lambda: llp.embedding_fwd(t, w.cpu()),
                lambda: llp.embedding_fwd(t.view(3, 1), w), lambda: llp.embedding_fwd(t, w.t()),
                lambda: llp.embedding_fwd(t, w[0]), lambda: llp.embedding_fwd(t, w[:0]),
                lambda: llp.embedding_fwd(t, w, out=torch.zeros(3, 9, device="cuda")),
                lambda: llp.embedding_bwd(g, t[:2], 4), lambda: llp.embedding_bwd(g, t, 0),
                lambda: llp.embedding_bwd(g, t, 4, accumulate=True),
                lambda: llp.embedding_bwd(g, t, 4, out=torch.zeros(5, 8, device="cuda")),
                lambda: llp.embedding_bwd(g.t(), t, 4), lambda: llp.embedding_bwd(g[0], t, 4),
                lambda: llp.embedding_bwd(g, t, 4, workspace=torch.zeros(1, dtype=torch.uint8, device="cuda")),
                lambda: llp.embedding_bwd(torch.zeros(30, device="cuda").as_strided((3, 8), (4, 1)), t, 4)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: llp.embedding_fwd(t.int(), w), lambda: llp.embedding_fwd(t, w.double()),
                lambda: llp.embedding_bwd(g.long(), t, 4)):
        with pytest.raises(TypeError):
            bad()
