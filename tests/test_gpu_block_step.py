"""Gated linear layer, RMS norms around a block and AdamW together, as a training step uses them: the example's
model, the calls without autograd, and captured graphs."""
import importlib.util
import os

import pytest
import torch

import lm_head_selected_gb300 as llp

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("tied_lm_step", os.path.join(ROOT, "examples", "tied_lm_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_of_the_gated_model(ex):
    """The example's gradients through autograd are those of the calls chained by hand, bit for bit (each call
    is held against its definition in 64 bits by its own tests)."""
    V, D, N = 500, 128, 300
    model = ex.TiedLM(V, D, seed=3, gated=True)
    tokens, targets = ex.batch(N, V, seed=4)
    loss, g_table, inner = model.gradients(tokens, targets, 0)
    got = {id(t): g for t, g in inner}
    with torch.no_grad():
        x = llp.embedding_fwd(tokens, model.table, model.scale)
        h = llp.dropout_fwd(x, model.p, model.seed, 0)
        norms = [b["w"] for b in model.blocks] + [model.norm["w"]]
        s, y, _, r = llp.residual_rms_norm_fwd(h, weight=norms[0])
        first, kept = (s, r), []
        for i, b in enumerate(model.blocks):
            a, pre = llp.gated_linear_fwd(y, b["gate"], b["up"], "silu", keep=True)
            d = llp.dropout_fwd(a @ b["down"], model.p, model.seed, 1 + i)
            s, y2, pr, r = llp.residual_rms_norm_fwd(s, d, b["layer_scale"], b["post"], norms[i + 1])
            kept.append((y, a, pre, d, s, pr, r))
            y = y2
        logp, lse = llp.linear_logp_fwd(y, model.table, targets)
        valid = torch.isfinite(lse)
        n = valid.sum().clamp(min=1)
        gl = torch.where(valid, -1.0 / n, 0.0).float()
        gy, g_tab, _ = llp.linear_logp_bwd(gl, lse, y, model.table, targets)
        gs = None
        for i in reversed(range(len(model.blocks))):
            b = model.blocks[i]
            yi, a, pre, d, s, pr, r = kept[i]
            gs, gd, g_scale, g_post, g_w = llp.residual_rms_norm_bwd(gs, gy, s, d, b["layer_scale"], b["post"],
                                                                     norms[i + 1], pr, r)
            for t, g in ((b["layer_scale"], g_scale), (b["post"], g_post), (norms[i + 1], g_w)):
                assert torch.equal(got[id(t)], g)
            gd = llp.dropout_bwd(gd, model.p, model.seed, 1 + i)
            assert torch.equal(got[id(b["down"])], a.t() @ gd)
            gy, gg, gu = llp.gated_linear_bwd(gd @ b["down"].t(), pre, yi, b["gate"], b["up"])
            assert torch.equal(got[id(b["gate"])], gg) and torch.equal(got[id(b["up"])], gu)
        # the first norm's output alone goes on; its stream is the embedding itself, whose gradients autograd adds
        gx, _, _, _, g_w = llp.residual_rms_norm_bwd(None, gy, first[0], weight=norms[0], rstd=first[1])
        assert torch.equal(got[id(norms[0])], g_w)
        gx = llp.dropout_bwd(gx + gs, model.p, model.seed, 0)
        llp.embedding_bwd(gx, tokens, V, model.scale, out=g_tab, accumulate=True)
        assert torch.equal(g_table, g_tab)
    assert torch.isfinite(loss)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_steps_repeat(ex, gated, bits):
    ends = []
    for _ in range(2):
        model = ex.TiedLM(512, 128, seed=5, gated=gated)
        adamw = model.optimizer(bits)
        tokens, targets = ex.batch(700, 512, seed=6)
        losses = [float(model.step(tokens, targets, i, 0.003, adamw)) for i in range(5)]
        assert all(l == l for l in losses)
        ends.append((losses, [p.clone() for p in model.parameters()]))
    assert ends[0][0] == ends[1][0]
    assert all(torch.equal(a, b) for a, b in zip(ends[0][1], ends[1][1]))
    assert llp.device_status() == 0


class Block:
    """A block's forward and backward through the calls without autograd, on given buffers."""

    def __init__(self, N, D, F, seed=0):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std=1.0, dt=torch.bfloat16):
            return (torch.randn(*shape, generator=g) * std).to(dt).to(DEV)

        self.x, self.gs, self.gh = normal(N, D), normal(N, D), normal(N, D)
        self.wg, self.wu, self.down = normal(F, D, std=D ** -0.5), normal(F, D, std=D ** -0.5), normal(F, D, std=F ** -0.5)
        self.w0, self.w1, self.post, self.gate = (1 + normal(D, std=0.1, dt=torch.float32) for _ in range(4))
        self.params = [self.wg, self.wu, self.down, self.w0, self.w1, self.post, self.gate]
        self.state = llp.adamw_state(self.params, 8, masters=True)
        self.count = torch.zeros(1, dtype=torch.int64, device=DEV)

    def step(self, ws_gated=None, ws_norm=None):
        _, y, _, r0 = llp.residual_rms_norm_fwd(self.x, weight=self.w0)
        a, pre = llp.gated_linear_fwd(y, self.wg, self.wu, keep=True)
        b = a @ self.down
        s, h, pr, r = llp.residual_rms_norm_fwd(self.x, b, self.gate, self.post, self.w1, scale=0.5)
        gx, gb, gg, gp, gw1 = llp.residual_rms_norm_bwd(self.gs, self.gh, s, b, self.gate, self.post, self.w1, pr, r, 0.5,
                                                        workspace=ws_norm)
        gd = a.t() @ gb
        gy, gwg, gwu = llp.gated_linear_bwd(gb @ self.down.t(), pre, y, self.wg, self.wu, workspace=ws_gated)
        gx0, _, _, _, gw0 = llp.residual_rms_norm_bwd(gx, gy, self.x, weight=self.w0, rstd=r0, workspace=ws_norm)
        self.count += 1
        llp.adamw_step(self.params, [gwg, gwu, gd, gw0, gw1, gp, gg], **self.state, step=0, lr=0.01, device_step=self.count)
        return s, h, gx0


@pytest.mark.parametrize("N", [1, 40, 700])
def test_captured_steps(N):
    """Two blocks' steps in a graph each, sharing workspaces, replayed in turn: what they give eagerly."""
    from lm_head_selected_gb300 import _lib
    lib = _lib.load()
    D, F = 136, 264
    ws = [torch.empty(lib.gated_linear_bwd_workspace_bytes(N, D, F), dtype=torch.uint8, device=DEV),
          torch.empty(lib.residual_rms_norm_bwd_workspace_bytes(N, D), dtype=torch.uint8, device=DEV)]
    eager = [Block(N, D, F, seed=k) for k in range(2)]
    blocks = [Block(N, D, F, seed=k) for k in range(2)]
    Block(N, D, F, seed=9).step()  # libraries warm up outside the capture
    graphs, outs = [], []
    for b in blocks:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(b.step(*ws))
        graphs.append(graph)
    for _ in range(3):
        for k in range(2):
            want = eager[k].step()
            graphs[k].replay()
            for a, c in zip(outs[k], want):
                assert torch.equal(a, c)
    for b, e in zip(blocks, eager):
        assert int(b.count) == 3
        for p, q in zip(b.params, e.params):
            assert torch.equal(p, q)
    assert llp.device_status() == 0


def test_two_streams_at_once():
    """Calls on two streams with buffers of their own do not disturb one another."""
    blocks, alone = [Block(300, 136, 264, seed=k) for k in range(2)], [Block(300, 136, 264, seed=k) for k in range(2)]
    want = [[b.step() for _ in range(4)][-1] for b in alone]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(4):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k] = blocks[k].step()
    torch.cuda.synchronize()
    for k in range(2):
        for a, c in zip(got[k], want[k]):
            assert torch.equal(a, c)
        for p, q in zip(blocks[k].params, alone[k].params):
            assert torch.equal(p, q)


def test_autograd_captured():
    """Forward and backward through autograd in a graph."""
    N, D, F = 50, 64, 128
    b = Block(N, D, F)
    leaves = [t.clone().requires_grad_(True) for t in (b.x, b.wg, b.wu, b.w0, b.w1, b.post, b.gate)]

    def run():
        x, wg, wu, w0, w1, post, gate = leaves
        _, y = llp.residual_rms_norm(x, weight=w0)
        z = llp.gated_linear(y, wg, wu, "gelu")
        s, h = llp.residual_rms_norm(x, z[:, :D].contiguous(), gate, post, w1)
        return torch.autograd.grad([s, h], leaves, [b.gs, b.gh])

    want = run()
    del_side = torch.cuda.Stream()
    del_side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(del_side):
        run()
    torch.cuda.current_stream().wait_stream(del_side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(got, want):
        assert torch.equal(a, c)
