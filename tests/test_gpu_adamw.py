"""The AdamW step on the GPU against its FP64 definition: types, odd sizes and places, many tensors, states
in 32 and 8 bits, values that come from the device, and captured steps."""
import numpy as np
import pytest
import torch

import lm_head_selected_gb300 as llp
from operator_bounds import U32, np64, rounded, within
from oracle import block_ops as bo

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HYPER = dict(lr=0.01, betas=(0.9, 0.95), eps=1e-8)
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32), (torch.float32, torch.float32)]
BLOCK, TOP, LEAST = 256, 448.0, 2.0 ** -9


def tensors(sizes, pdt, gdt, seed=0):
    g = torch.Generator().manual_seed(seed)
    params = [(torch.randn(n, generator=g)).to(pdt).to(DEV) for n in sizes]
    grads = [(torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g)) * 0.01).to(gdt).to(DEV) for n in sizes]
    return params, grads


def filled(state, grads, seed=1):
    """A state some steps into training."""
    g = torch.Generator().manual_seed(seed)
    packed = "exp_avg_scale" in state
    for i, gr in enumerate(grads):
        n = gr.numel()
        m = torch.randn(n, generator=g).to(DEV) * 0.005
        u = torch.rand(n, generator=g).to(DEV) * 0.02
        if not packed:
            state["exp_avg"][i].copy_(m)
            state["exp_avg_sq"][i].copy_(u * u)
            continue
        for key, t in (("exp_avg", m), ("exp_avg_sq", u)):
            b = torch.nn.functional.pad(t, (0, -n % BLOCK)).view(-1, BLOCK)
            sc = b.abs().amax(1) / TOP
            state[key + "_scale"][i].copy_(sc)
            state[key][i].copy_((b / sc.clamp(min=1e-30)[:, None]).view(-1)[:n].to(torch.float8_e4m3fn).view_as(gr))
    return state


def value(code, scale):
    """What codes and scales stand for."""
    c = np64(code.float()).reshape(-1)
    return c * np.repeat(np64(scale), BLOCK)[:c.size]


def start(params, grads, state):
    out = []
    for i, p in enumerate(params):
        top = state["masters"][i] if "masters" in state and state["masters"][i] is not None else p
        if "exp_avg_scale" in state:
            m = value(state["exp_avg"][i], state["exp_avg_scale"][i])
            v = value(state["exp_avg_sq"][i], state["exp_avg_sq_scale"][i]) ** 2
        else:
            m, v = np64(state["exp_avg"][i]).reshape(-1), np64(state["exp_avg_sq"][i]).reshape(-1)
        out.append((np64(top).reshape(-1), np64(grads[i]).reshape(-1), m, v))
    return out


def check(params, state, before, step, decay, lr=HYPER["lr"], scale=1.0, betas=HYPER["betas"], eps=HYPER["eps"]):
    """fp32 steps: a handful of roundings each, of the terms' sizes; the update's quotient within 2^-20."""
    for i, (p0, g, m0, v0) in enumerate(before):
        g = g * scale
        p, m, v = bo.adamw(p0, g, m0, v0, step, lr, *betas, eps, decay[i])
        em = 8 * U32 * (np.abs(m0) + np.abs(g)) + 1e-44
        ev = 8 * U32 * (v0 + g * g) + 1e-44
        root = np.sqrt(v / (1 - betas[1] ** step))
        upd = lr * np.abs(m / (1 - betas[0] ** step)) / (root + eps)
        # m may be a difference of larger terms: its error divided as m is
        ep = 4 * U32 * np.abs(p0) + 2.0 ** -19 * upd + lr * em / (1 - betas[0] ** step) / (root + eps)
        got = params[i].reshape(-1)
        if "masters" in state and state["masters"][i] is not None:
            top = state["masters"][i].reshape(-1)
            within("master", top, p, ep)
            assert torch.equal(got, top.to(got.dtype))
        else:
            within("param", got, p, rounded(p, got.dtype) + 1.01 * ep)
        if "exp_avg_scale" not in state:
            within("m", state["exp_avg"][i].reshape(-1), m, em)
            within("v", state["exp_avg_sq"][i].reshape(-1), v, ev)
            continue
        for key, t, e in (("exp_avg", m, em), ("exp_avg_sq", np.sqrt(v), 8 * U32 * np.sqrt(v + v0 + g * g))):
            sc = np64(state[key + "_scale"][i])
            b = np.pad(np.abs(t), (0, -t.size % BLOCK)).reshape(-1, BLOCK)
            eb = np.pad(e, (0, -e.size % BLOCK)).reshape(-1, BLOCK)
            within(key + "_scale", state[key + "_scale"][i], b.max(1) / TOP, eb.max(1) / TOP + 4 * U32 * b.max(1) / TOP)
            each = np.repeat(sc, BLOCK)[:t.size]
            want = t if key == "exp_avg" else np.where(t > 0, np.maximum(t, LEAST * each), 0.0)
            # half a step of three fraction bits, or of the smallest exponent's; the quotient's roundings
            half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * each) * (1 + 2.0 ** -10) + 2 * e
            got = value(state[key][i], state[key + "_scale"][i])
            assert (np.abs(got - want) <= half).all(), (key, i, np.max(np.abs(got - want) - half))
            if key == "exp_avg_sq":
                assert (got[t > 1e-30] > 0).all()


SIZES = [1, 2, 7, 8, 9, 255, 256, 257, 1000, 4095, 4096, 4097, 12345, 70001]


@pytest.mark.parametrize("masters", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", TYPES)
def test_sizes_and_types(pdt, gdt, bits, masters):
    params, grads = tensors(SIZES, pdt, gdt)
    state = filled(llp.adamw_state(params, bits, masters), grads)
    decay = [0.1 * (i % 3) for i in range(len(params))]
    for step in (3, 4):
        before = start(params, grads, state)
        llp.adamw_step(params, grads, **state, step=step, weight_decay=decay, **HYPER)
        check(params, state, before, step, decay)


@pytest.mark.parametrize("bits", [32, 8])
def test_from_zero_states(bits):
    params, grads = tensors([300, 5000], torch.float32, torch.float32)
    grads[0][:] = 0
    grads[1][::3] = 0
    state = llp.adamw_state(params, bits)
    for step in range(1, 6):
        before = start(params, grads, state)
        llp.adamw_step(params, grads, **state, step=step, weight_decay=0.0, **HYPER)
        check(params, state, before, step, [0.0, 0.0])
    assert torch.equal(params[0], tensors([300, 5000], torch.float32, torch.float32)[0][0])  # no gradient ever


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_places_inside_flat_buffers(bits, shift):
    """Views that start anywhere, all at one element or each at its own."""
    n = 9001
    for own in (False, True):
        ref_p, ref_g = tensors([n], torch.bfloat16, torch.bfloat16)
        ref = filled(llp.adamw_state(ref_p, bits, True), ref_g)

        def moved(t, by):
            room = torch.empty(t.numel() + 64, dtype=t.dtype, device=DEV)
            return room[by:by + t.numel()].copy_(t.reshape(-1))

        params, grads = [moved(ref_p[0], shift)], [moved(ref_g[0], shift + 2 * own)]
        state = {k: [moved(v[0], shift + own * j)] for j, (k, v) in enumerate(ref.items())}
        llp.adamw_step(params, grads, **state, step=2, **HYPER)
        llp.adamw_step(ref_p, ref_g, **ref, step=2, **HYPER)
        assert torch.equal(params[0], ref_p[0])
        for k in ref:
            assert torch.equal(state[k][0].view(torch.uint8), ref[k][0].view(torch.uint8)), k


def test_nothing_else_is_written():
    n = 1003
    for bits in (32, 8):
        params, grads = tensors([n], torch.bfloat16, torch.float32)
        state = llp.adamw_state(params, bits, True)
        rooms, views = [], {}
        for k, v in [("p", params), *state.items()]:
            raw = v[0].view(torch.uint8).reshape(-1)
            room = torch.full((raw.numel() + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
            room[2048:2048 + raw.numel()] = raw
            rooms.append((room, raw.numel()))
            views[k] = [room[2048:2048 + raw.numel()].view(v[0].dtype)]
        p = views.pop("p")
        llp.adamw_step(p, grads, **views, step=1, **HYPER)
        assert not torch.equal(p[0], params[0])
        for room, size in rooms:
            assert (room[:2048] == 0x5A).all() and (room[2048 + size:] == 0x5A).all()


@pytest.mark.parametrize("count", [41, 320, 321, 700])
def test_many_tensors(count):
    """More than one launch's parameters hold; each result as if it were alone."""
    sizes = [(i * 37) % 600 + (0 if i % 50 == 3 else 1) for i in range(count)]
    sizes[5] = 0
    for bits in (32, 8):
        params, grads = tensors(sizes, torch.bfloat16, torch.bfloat16)
        state = filled(llp.adamw_state(params, bits), grads)
        alone_p = [p.clone() for p in params]
        alone_s = {k: [t.clone() for t in v] for k, v in state.items()}
        llp.adamw_step(params, grads, **state, step=7, **HYPER)
        for i in range(0, count, 23):
            llp.adamw_step(alone_p[i:i + 1], grads[i:i + 1], **{k: v[i:i + 1] for k, v in alone_s.items()}, step=7, **HYPER)
            assert torch.equal(params[i], alone_p[i])
            for k in state:
                assert torch.equal(state[k][i].view(torch.uint8), alone_s[k][i].view(torch.uint8))


def test_mixed_types_shapes_and_decays():
    params = [torch.randn(33, 65, device=DEV).to(torch.bfloat16), torch.randn(129, device=DEV),
              torch.randn(4, 5, 6, device=DEV).half()]
    grads = [torch.randn_like(params[0]), torch.randn_like(params[1]), torch.randn(4, 5, 6, device=DEV)]
    state = llp.adamw_state(params, 32, masters=True)
    assert state["masters"][1] is None
    before = start(params, grads, state)
    versions = [p._version for p in params]
    llp.adamw_step(params, grads, **state, step=1, weight_decay=[0.1, 0.0, 0.2], **HYPER)
    check(params, state, before, 1, [0.1, 0.0, 0.2])
    assert all(p._version > v for p, v in zip(params, versions))


@pytest.mark.parametrize("bits", [32, 8])
def test_values_on_the_device(bits):
    params, grads = tensors([5000, 31], torch.float32, torch.float32)
    state = filled(llp.adamw_state(params, bits), grads)
    before = start(params, grads, state)
    llp.adamw_step(params, grads, **state, step=2, weight_decay=0.1, lr=0.5, betas=(0.9, 0.95), eps=1e-8,
                   device_step=torch.tensor(3, device=DEV), device_lr=torch.tensor(0.02, device=DEV),
                   grad_scale=torch.tensor([0.25], device=DEV))
    check(params, state, before, 5, [0.1, 0.1], lr=0.5 * np.float64(np.float32(0.02)), scale=0.25)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_advance(bits):
    params, grads = tensors([3000, 256], torch.bfloat16, torch.bfloat16)
    state = llp.adamw_state(params, bits, True)
    other_p = [p.clone() for p in params]
    other = {k: [t.clone() for t in v] for k, v in state.items()}
    counter = torch.zeros(1, dtype=torch.int64, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            counter += 1
            llp.adamw_step(params, grads, **state, step=0, device_step=counter, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(1, 5):
        graph.replay()
        llp.adamw_step(other_p, grads, **other, step=step, **HYPER)
    # the corrections come from 64-bit powers on either side, rounded once to fp32: at most one unit apart
    for a, b in zip(state["masters"], other["masters"]):
        within("master", a, np64(b), 16 * U32 * (np.abs(np64(b)) + HYPER["lr"] * 4 * 4))


@pytest.mark.parametrize("bits", [32, 8])
def test_values_next_to_a_block_s_largest(bits):
    """One gradient a million times the others: in 8 bits the others' roots are stored as the least
    code, not as 0, so that no later step divides by eps alone."""
    params, grads = tensors([512], torch.float32, torch.float32)
    params[0][:] = 0
    grads[0][:] = 1e-6
    grads[0][100] = 1.0
    state = llp.adamw_state(params, bits)
    for step in range(1, 30):
        before = start(params, grads, state)
        llp.adamw_step(params, grads, **state, step=step, weight_decay=0.0, lr=1e-3, betas=(0.9, 0.999), eps=1e-15)
        check(params, state, before, step, [0.0], lr=1e-3, betas=(0.9, 0.999), eps=1e-15)
    assert params[0].abs().max().item() <= 30 * 1e-3 * 1.01


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-18, 1e15])
def test_gradients_of_extreme_sizes(size):
    for bits in (32, 8):
        params, grads = tensors([700], torch.float32, torch.float32)
        grads[0].mul_(size * 100)
        state = llp.adamw_state(params, bits)
        for step in (1, 2):
            before = start(params, grads, state)
            llp.adamw_step(params, grads, **state, step=step, weight_decay=0.0, **HYPER)
        assert params[0].isfinite().all()
        for k in state:
            assert state[k][0].float().isfinite().all()
        m = value(state["exp_avg"][0], state["exp_avg_scale"][0]) if bits == 8 else np64(state["exp_avg"][0])
        want = 0.19 * np64(grads[0]) if bits == 32 else 0.9 * before[0][2] + 0.1 * np64(grads[0])
        assert np.abs(m - want).max() <= (2.0 ** -4 if bits == 8 else 1e-5) * np.abs(want).max() + 1e-44


def test_what_is_not_finite_stays_where_it_is():
    params, grads = tensors([1024], torch.float32, torch.float32)
    grads[0][300] = float("nan")
    state = llp.adamw_state(params, 32)
    llp.adamw_step(params, grads, **state, step=1, **HYPER)
    assert params[0].isnan().sum().item() == 1
    params, _ = tensors([1024], torch.float32, torch.float32)
    state = llp.adamw_state(params, 8)
    llp.adamw_step(params, grads, **state, step=1, **HYPER)
    assert params[0].isnan().sum().item() == 1  # the codes of its block are spoilt, no others
    scales = state["exp_avg_scale"][0]
    assert scales[1].isnan() and scales[[0, 2, 3]].isfinite().all()


def test_another_stream_and_other_order():
    sizes = [100, 5000, 77]
    params, grads = tensors(sizes, torch.bfloat16, torch.bfloat16)
    state = filled(llp.adamw_state(params, 8), grads)
    other_p = [p.clone() for p in params][::-1]
    other = {k: [t.clone() for t in v][::-1] for k, v in state.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        llp.adamw_step(params, grads, **state, step=2, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    llp.adamw_step(other_p, grads[::-1], **other, step=2, **HYPER)
    for a, b in zip(params, other_p[::-1]):
        assert torch.equal(a, b)


def codes_in_fp32(t, root):
    """The header's formulas in torch's fp32, operation by operation: the stored codes and scales."""
    b = torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)).view(-1, BLOCK)
    scale = b.abs().amax(1) * torch.tensor(1.0 / TOP, device=DEV)
    c = b / torch.where(scale > 0, scale, 1.0)[:, None]
    if root:
        c = torch.where(c > 0, c.clamp(LEAST, TOP), 0.0)
    return c.clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(-1)[:t.numel()], scale


@pytest.mark.parametrize("n", [256 * 3000, 100003])
def test_codes_are_those_of_the_formulas_in_fp32(n):
    """Next to a border between two codes a sum contracted into one rounding would choose the other one."""
    params, grads = tensors([n], torch.bfloat16, torch.bfloat16)
    state = filled(llp.adamw_state(params, 8), grads)
    f = [state[k][0].float() * state[k + "_scale"][0].repeat_interleave(BLOCK)[:n] for k in ("exp_avg", "exp_avg_sq")]
    g = grads[0].float()
    b1, b2 = HYPER["betas"]
    m = f[0] * b1 + g * (1.0 - b1)
    v = f[1] * f[1]
    v = v * b2 + (g * g) * (1.0 - b2)
    llp.adamw_step(params, grads, **state, step=3, **HYPER)
    for key, t, root in (("exp_avg", m, False), ("exp_avg_sq", torch.sqrt(v), True)):
        code, scale = codes_in_fp32(t, root)
        assert torch.equal(state[key + "_scale"][0], scale)
        assert torch.equal(state[key][0].float(), code.float())


def test_tensors_made_under_inference_mode():
    with torch.inference_mode():
        params, grads = tensors([300], torch.float32, torch.float32)
        state = llp.adamw_state(params)
        kept = params[0].clone()
        llp.adamw_step(params, grads, **state, step=1, **HYPER)
        assert not torch.equal(params[0], kept)


def test_refusals():
    params, grads = tensors([64, 32], torch.bfloat16, torch.bfloat16)
    s = llp.adamw_state(params)
    s8 = llp.adamw_state(params, 8)
    kept = [p.clone() for p in params]

    def call(params=params, grads=grads, state=s, **over):
        llp.adamw_step(params, grads, **{**state, "step": 1, **over})

    for bad, error in ((dict(params=[params[0], params[0]], grads=[grads[0]] * 2), ValueError),
                       (dict(params=[params[0], params[0][:32]]), ValueError),
                       (dict(exp_avg_sq=s["exp_avg"]), ValueError), (dict(state=s8, exp_avg_sq_scale=s8["exp_avg_scale"]), ValueError),
                       (dict(grads=grads[:1]), ValueError), (dict(grads=[grads[0].half(), grads[1]]), TypeError),
                       (dict(grads=[grads[1], grads[0]]), ValueError), (dict(params=[params[0].double(), params[1]]), TypeError),
                       (dict(params=[params[0].cpu(), params[1]]), ValueError),
                       (dict(exp_avg=s["exp_avg"][:1]), ValueError), (dict(exp_avg=s8["exp_avg"]), TypeError),
                       (dict(exp_avg_sq=s["exp_avg"][::-1]), ValueError),
                       (dict(state=s8, exp_avg_scale=s8["exp_avg_scale"][:1]), ValueError),
                       (dict(state=s8, exp_avg_sq_scale=[t.half() for t in s8["exp_avg_sq_scale"]]), TypeError),
                       (dict(masters=[None]), ValueError), (dict(masters=[t.float()[:8] for t in params]), ValueError),
                       (dict(weight_decay=[0.1]), ValueError), (dict(weight_decay=float("nan")), ValueError),
                       (dict(device_step=torch.tensor(1)), ValueError), (dict(device_step=torch.tensor(1.0, device=DEV)), ValueError),
                       (dict(device_lr=torch.ones(2, device=DEV)), ValueError), (dict(step=0), ValueError)):
        with pytest.raises(error):
            call(**bad)
    strided = [torch.randn(16, 8, device=DEV).t(), params[1]]
    with pytest.raises(ValueError):
        call(params=strided, grads=[torch.randn(8, 16, device=DEV), grads[1]])
    assert all(torch.equal(a, b) for a, b in zip(params, kept))
    with pytest.raises(ValueError):
        llp.adamw_state(params, 16)


def test_a_gradient_that_is_written_too_is_refused():
    params, grads = tensors([64, 0, 32, 0], torch.float32, torch.float32)
    state = llp.adamw_state(params)
    kept = [p.clone() for p in params]
    for bad in ([params[0], *grads[1:]], [grads[0], grads[1], params[0][:32], grads[3]],
                [state["exp_avg"][0], *grads[1:]], [*grads[:2], state["exp_avg_sq"][2], grads[3]]):
        with pytest.raises(ValueError, match="gradient"):
            llp.adamw_step(params, bad, **state, step=1)
    assert all(torch.equal(a, b) for a, b in zip(params, kept))
    # one gradient for two parameters is read twice; tensors without elements share no place
    llp.adamw_step([params[0], params[1], params[2]], [grads[0], grads[1], grads[0][:32]],
                   state["exp_avg"][:3], state["exp_avg_sq"][:3], 1)
    assert not torch.equal(params[2], kept[2])
