"""The RMS norms around a block and AdamW where a tensor's last byte is the last of a mapped region of device memory."""
import pytest
import torch

import lm_head_selected_gb300 as llp
from mapped_region import DEV, Region, at_the_end
from test_gpu_adamw import HYPER, filled, tensors
from test_gpu_residual_rms_norm import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def regions():
    return [torch.as_tensor(Region(), device=DEV) for _ in range(2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "columns", "rows"])
@pytest.mark.parametrize("N,D", [(1, 1), (7, 3), (33, 101), (40, 264), (200, 1001), (20, 2688), (9, 8200), (3, 17001)])
def test_norms(regions, N, D, gate, dtype):
    args = inputs(N, D, dtype, dtype, gate, True, True)
    s, h, pr, r = llp.residual_rms_norm_fwd(*args)
    g = torch.Generator().manual_seed(N + D)
    gs, gh = (torch.randn(N, D, generator=g).to(dtype).to(DEV) for _ in range(2))
    want = llp.residual_rms_norm_bwd(gs, gh, s, *args[1:], pr, r)
    for i in range(5):
        if args[i] is None:
            continue
        moved = list(args)
        moved[i] = at_the_end(regions[0], args[i])
        for a, b in zip(llp.residual_rms_norm_fwd(*moved), (s, h, pr, r)):
            assert torch.equal(a, b), i
    every = [gs, gh, s, *args[1:], pr, r]
    for i in range(len(every)):
        j = (i + 1) % len(every)
        if every[i] is None or every[j] is None:
            continue
        moved = list(every)
        moved[i], moved[j] = at_the_end(regions[0], every[i]), at_the_end(regions[1], every[j])
        for a, b in zip(llp.residual_rms_norm_bwd(*moved), want):
            assert (a is None and b is None) or torch.equal(a, b), (i, j)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                     (torch.float32, torch.float32)])
@pytest.mark.parametrize("n", [1, 7, 255, 256, 257, 5000, 16384, 70001])
def test_adamw(regions, n, pdt, gdt, bits):
    params, grads = tensors([n], pdt, gdt)
    state = filled(llp.adamw_state(params, bits, True), grads)
    one = {"p": params[0], "g": grads[0], **{k: v[0] for k, v in state.items() if v[0] is not None}}
    names = list(one)

    def step(t):
        kept = {k: [t[k]] if k in t else [None] for k in state}
        llp.adamw_step([t["p"]], [t["g"]], **kept, step=5, weight_decay=0.1, **HYPER)
        return t

    want = step({k: v.clone() for k, v in one.items()})
    for i, name in enumerate(names):
        other = names[(i + 1) % len(names)]
        t = {k: v.clone() for k, v in one.items()}
        t[name], t[other] = at_the_end(regions[0], one[name]), at_the_end(regions[1], one[other])
        step(t)
        for k in want:
            assert torch.equal(t[k].view(torch.uint8), want[k].view(torch.uint8)), (name, other, k)
