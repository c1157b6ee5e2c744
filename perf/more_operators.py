"""The operators of a model's blocks and of its optimizer, as measured cases: the gated linear layer (two projections,
an activation and a product) and its gradient, the RMS norms before and after a block with the block's gate and residual
scale and their gradient, and the AdamW step over many tensors with states in 32 or 8 bits.

``run`` computes one pass.  With ``own`` false it is the plain form: elementary torch operations in 32 bits, rounded
once at the end.  With ``own`` true it is the call into this package.  ``exact`` is the definition in 64 bits.
Sizes are the ones of this repository's workloads and example (hidden 2688, 4096, 2048 and 512, vocabulary 131072 and
8192; 32, 16384 and 65600 tokens), inner widths of two or four times the hidden size, and generic odd ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5
BETAS, ADAM_EPS, DECAY, RATE = (0.9, 0.95), 1e-8, 0.1, 1e-3
BLOCK = 256    # values of an 8-bit state that share a scale
TOP = 448.0    # largest value of an 8-bit state
LEAST = 2.0 ** -9


def listed():
    return [
        # one token of one sequence through a block's first half at hidden 4096: the weights' stream, latency counts
        {"name": "gated token", "op": "gated_fwd", "N": 1, "D": 4096, "F": 16384, "dtype": "bf16", "act": "silu",
         "keep": False},
        # the tokens of one decoding step of 32 sequences
        {"name": "gated decode", "op": "gated_fwd", "N": 32, "D": 2688, "F": 10752, "dtype": "bf16", "act": "silu",
         "keep": False},
        # a small fp16 model's batch, sizes that no tile divides, both projections kept for the gradient
        {"name": "gated odd", "op": "gated_fwd", "N": 1111, "D": 1000, "F": 2744, "dtype": "fp16", "act": "gelu",
         "keep": True},
        # a training batch
        {"name": "gated batch", "op": "gated_fwd", "N": 16384, "D": 2688, "F": 10752, "dtype": "bf16", "act": "silu",
         "keep": True},
        # the gradient of a training batch
        {"name": "gated grad", "op": "gated_bwd", "N": 16384, "D": 2688, "F": 10752, "dtype": "bf16", "act": "silu"},
        # one decoding step of 32 sequences: a block's end and the next one's start; latency counts
        {"name": "norms decode", "op": "norms_fwd", "N": 32, "D": 2688, "dtype": "bf16", "params": "bf16",
         "gate": "columns", "post": True},
        # the same of a training batch
        {"name": "norms batch", "op": "norms_fwd", "N": 16384, "D": 2688, "dtype": "bf16", "params": "bf16",
         "gate": "columns", "post": True},
        # the gradient in a small fp32 model with an odd hidden size and a gate of its own for every token
        {"name": "norms grad odd", "op": "norms_bwd", "N": 2049, "D": 1001, "dtype": "fp32", "params": "fp32",
         "gate": "rows", "post": True},
        # the gradient of a training batch at hidden 4096
        {"name": "norms grad", "op": "norms_bwd", "N": 16384, "D": 4096, "dtype": "bf16", "params": "bf16",
         "gate": "columns", "post": True},
        # the example's model with gated blocks: few and small tensors, latency counts
        {"name": "adamw small", "op": "adamw", "hidden": 512, "inner": 1024, "layers": 2, "vocab": 8192,
         "dtype": "bf16", "grads": "bf16", "bits": 32, "masters": False},
        # the head's table and a block, in bf16 with fp32 master weights and states
        {"name": "adamw table", "op": "adamw", "hidden": 2688, "inner": 10752, "layers": 1, "vocab": 131072,
         "dtype": "bf16", "grads": "bf16", "bits": 32, "masters": True},
        # blocks of an odd-sized model, states in eight bits
        {"name": "adamw 8-bit", "op": "adamw", "hidden": 2047, "inner": 8191, "layers": 6, "vocab": 32767,
         "dtype": "bf16", "grads": "bf16", "bits": 8, "masters": False},
    ]


MOST = {"gated_fwd": 0.95e12, "gated_bwd": 3.8e12, "norms_fwd": 2.7e8 * 4, "norms_bwd": 1.1e9, "adamw": 1.2e10}


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "norms_fwd", "norms_bwd", "norms_bwd", "adamw", "adamw"])
        if op == "adamw":
            case = {"op": op, "hidden": rng.choice([_spread(rng, 17, 2700) | 1, 8 * _spread(rng, 4, 330)]),
                    "layers": _spread(rng, 1, 12), "vocab": rng.choice([_spread(rng, 100, 65536) | 1, 8192, 32768]),
                    "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "bits": rng.choice([32, 8])}
            case["inner"] = rng.choice([2 * case["hidden"], 4 * case["hidden"], _spread(rng, 64, 8192)])
            case["grads"] = rng.choice([case["dtype"], "fp32"])
            case["masters"] = case["dtype"] != "fp32" and rng.random() < 0.5
        else:
            case = {"op": op, "N": rng.choice([_spread(rng, 1, 65600), _spread(rng, 1, 65600) | 1, 32, 512, 4096, 16384])}
            if op.startswith("gated"):
                case["D"] = rng.choice([8 * _spread(rng, 4, 512), 512, 2048, 2688, 4096])
                case["F"] = rng.choice([8 * _spread(rng, 8, 2048), 2 * case["D"], 4 * case["D"]])
                case["dtype"] = rng.choice(["bf16", "bf16", "fp16"])
                case["act"] = rng.choice(["silu", "gelu", "gelu_tanh"])
                if op == "gated_fwd":
                    case["keep"] = rng.random() < 0.5
            else:
                case["D"] = rng.choice([_spread(rng, 24, 8300), 8 * _spread(rng, 4, 1100), 2048, 2688, 4096])
                case["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
                case["params"] = rng.choice([case["dtype"], "fp32"])
                case["gate"] = rng.choice(["columns", "rows", "none"])
                case["post"] = rng.random() < 0.75
        w = work(case)
        if w["flops" if op.startswith("gated") else "bytes"] <= MOST[op]:
            return case


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------

def _normal(shape, g, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=g.device, dtype=torch.float32) * std).to(dtype)


def _adamw_sizes(case):
    """Elements of the matrices and of the vectors, tensor by tensor."""
    h, f = case["hidden"], case["inner"]
    return [case["vocab"] * h] + [f * h] * (3 * case["layers"]), [h] * (2 * case["layers"] + 1)


def _places(sizes, bits):
    """Where each tensor starts in its flat buffer and how long that is.  Tensors with states in 32 bits follow one
    another at any element; those with states in 8 bits start with a block of their own."""
    at, places = 0, []
    for n in sizes:
        places.append(at)
        at += n if bits == 32 else -(-n // BLOCK) * BLOCK
    return places, at


def _views(flat, sizes, places):
    return [flat[a:a + n] for n, a in zip(sizes, places)]


def _used(sizes, places, total, dev):
    """1 for the elements of a flat buffer that belong to a tensor, 0 for those between two."""
    used = torch.zeros(total, dtype=torch.bool, device=dev)
    for v in _views(used, sizes, places):
        v.fill_(True)
    return used


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if op.startswith("gated"):
        N, D, F = case["N"], case["D"], case["F"]
        s["x"] = _normal((N, D), g, dt)  # a norm's output
        s["w_gate"], s["w_up"] = (_normal((F, D), g, dt, 1.0 / math.sqrt(D)) for _ in range(2))
        if op == "gated_bwd":
            s["grad_y"] = _normal((N, F), g, dt)
            s["pre"] = torch.empty((2, N, F), dtype=dt, device=dev)  # what the forward pass kept
            for k, w in enumerate((s["w_gate"], s["w_up"])):
                s["pre"][k].copy_(s["x"] @ w.t())
    elif op.startswith("norms"):
        N, D = case["N"], case["D"]
        pt = DTYPES[case["params"]]
        # a residual stream: columns of their own offset and width, a few of them far wider than the rest
        wide = torch.where(torch.rand(D, generator=g, device=dev) < 0.01, 20.0, 1.0)
        x = torch.randn((N, D), generator=g, device=dev) * wide + torch.randn(D, generator=g, device=dev)
        s["x"] = x.to(dt)
        s["branch"] = _normal((N, D), g, dt, 0.7)
        s["gate"] = (None if case["gate"] == "none" else _normal((D,), g, pt, 0.5) if case["gate"] == "columns"
                     else torch.sigmoid(torch.randn((N, D), generator=g, device=dev)).to(dt))
        s["post_weight"] = (1.0 + _normal((D,), g, torch.float32, 0.2)).to(pt) if case["post"] else None
        s["weight"] = (1.0 + _normal((D,), g, torch.float32, 0.2)).to(pt)
        s["scale"] = 0.5
        if op == "norms_bwd":
            s["stream"], _, s["post_rstd"], s["rstd"] = _norms_plain(s)  # what the forward pass gave
            del s["x"]
            s["grad_stream"], s["grad_h"] = (_normal((N, D), g, dt) for _ in range(2))
    else:
        # parameters, gradients and states as views of flat buffers, one set for matrices and one for vectors
        s["step"] = 1 + int(seed) % 1000
        s["groups"] = []
        for sizes, p_dt, g_dt, decay in zip(_adamw_sizes(case), (dt, torch.float32), (DTYPES[case["grads"]], torch.float32),
                                            (DECAY, 0.0)):
            places, total = _places(sizes, case["bits"])
            used = _used(sizes, places, total, dev)
            q = {"sizes": sizes, "places": places, "decay": decay}
            p = _normal((total,), g, torch.float32, 0.02).mul_(used)
            q["params"] = p.to(p_dt)
            q["masters"] = p if case["masters"] and p_dt != torch.float32 else None
            del p
            # gradients of blocks of their own size, an exact zero here and there
            size = torch.exp(torch.randn((total // 64 + 1, 1), generator=g, device=dev)) * 1e-3
            size = size.expand(-1, 64).reshape(-1)[:total] * used
            zero = torch.rand(total, generator=g, device=dev) < 1.0 / 64
            q["grads"] = torch.randn(total, generator=g, device=dev).mul_(size).masked_fill_(zero, 0.0).to(g_dt)
            m = torch.randn(total, generator=g, device=dev).mul_(size).mul_(0.25)
            u = torch.rand(total, generator=g, device=dev).add_(0.5).mul_(size)  # root of the second moment
            del size, zero
            if case["bits"] == 8:
                q["m"], q["m_scale"] = _pack_plain(m, False)
                q["v"], q["v_scale"] = _pack_plain(u, True)
            else:
                q["m"], q["v"] = m, u.square_()
            s["groups"].append(q)
        # the lists that a user's program holds
        s["lists"] = {k: [v for q in s["groups"] for v in _views(q[k], q["sizes"], q["places"])]
                      for k in ("params", "grads", "m", "v")}
        s["lists"]["decay"] = [q["decay"] for q in s["groups"] for _ in q["sizes"]]
        s["lists"]["masters"] = ([None if q["masters"] is None else v for q in s["groups"] for v in
                                  _views(q["params"] if q["masters"] is None else q["masters"], q["sizes"], q["places"])]
                                 if case["masters"] else None)
        for k in ("m_scale", "v_scale"):
            s["lists"][k] = ([q[k][a // BLOCK:a // BLOCK + -(-n // BLOCK)] for q in s["groups"]
                              for n, a in zip(q["sizes"], q["places"])] if case["bits"] == 8 else None)
    return s


# ---------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import lm_head_selected_gb300 as llp
    case = s["case"]
    op = case["op"]
    if op == "gated_fwd":
        return llp.gated_linear_fwd(s["x"], s["w_gate"], s["w_up"], case["act"], keep=case["keep"])
    if op == "gated_bwd":
        return llp.gated_linear_bwd(s["grad_y"], s["pre"], s["x"], s["w_gate"], s["w_up"], case["act"])
    if op == "norms_fwd":
        return llp.residual_rms_norm_fwd(s["x"], s["branch"], s["gate"], s["post_weight"], s["weight"],
                                         scale=s["scale"], eps=EPS)
    if op == "norms_bwd":
        return llp.residual_rms_norm_bwd(s["grad_stream"], s["grad_h"], s["stream"], s["branch"], s["gate"],
                                         s["post_weight"], s["weight"], s["post_rstd"], s["rstd"], scale=s["scale"])
    t = s["lists"]
    llp.adamw_step(t["params"], t["grads"], t["m"], t["v"], s["step"], lr=RATE, betas=BETAS, eps=ADAM_EPS,
                   weight_decay=t["decay"], masters=t["masters"], exp_avg_scale=t["m_scale"],
                   exp_avg_sq_scale=t["v_scale"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return [{k: q.get(k) for k in ("params", "masters", "m", "v", "m_scale", "v_scale")} for q in s["groups"]]


def _act_plain(act, z):
    """The activation and its derivative."""
    if act == "silu":
        e = 1.0 / (1.0 + torch.exp(-z))
        return z * e, e * (1.0 + z * (1.0 - e))
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)


def _norms_plain(s):
    dt = s["x"].dtype
    t = s["branch"].float()
    post_rstd = None
    if s["post_weight"] is not None:
        post_rstd = torch.rsqrt(t.square().mean(1) + EPS)
        t = t * post_rstd[:, None] * s["post_weight"].float()
    t = t * s["scale"]
    if s["gate"] is not None:
        t = t * s["gate"].float()
    t = t + s["x"].float()
    rstd = torch.rsqrt(t.square().mean(1) + EPS)
    return t.to(dt), (t * rstd[:, None] * s["weight"].float()).to(dt), post_rstd, rstd


def _norms_grad_plain(s):
    dt, pt = s["stream"].dtype, s["weight"].dtype
    h = s["stream"].float() * s["rstd"][:, None]
    gh = s["grad_h"].float()
    a = gh * s["weight"].float()
    g_weight = (gh * h).sum(0).to(pt)
    gx = (a - h * (a * h).mean(1, keepdim=True)) * s["rstd"][:, None] + s["grad_stream"].float()
    b = s["branch"].float()
    n = b if s["post_weight"] is None else b * s["post_rstd"][:, None]
    t = gx * s["scale"]
    normed = n if s["post_weight"] is None else n * s["post_weight"].float()
    g_gate = None
    if s["gate"] is not None:
        g_gate = t * normed
        g_gate = g_gate.sum(0).to(pt) if s["gate"].dim() == 1 else g_gate.to(dt)
        t = t * s["gate"].float()
    g_post = None
    if s["post_weight"] is not None:
        g_post = (t * n).sum(0).to(pt)
        t = t * s["post_weight"].float()
        t = (t - n * (t * n).mean(1, keepdim=True)) * s["post_rstd"][:, None]
    return gx.to(dt), t.to(dt), g_gate, g_post, g_weight


def _pack_plain(t, root):
    """Values in eight bits (1-4-3, one scale to BLOCK of them); a root above 0 stays above 0."""
    n = t.numel()
    b = torch.nn.functional.pad(t, (0, -n % BLOCK)).view(-1, BLOCK)
    scale = b.abs().amax(1) / TOP
    c = b / torch.where(scale > 0, scale, 1.0)[:, None]
    if root:
        c = torch.where(c > 0, c.clamp(LEAST, TOP), 0.0)
    return c.clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(-1)[:n], scale


def _unpack_plain(code, scale):
    n = code.numel()
    b = torch.nn.functional.pad(code.float(), (0, -n % BLOCK)).view(-1, BLOCK)
    return (b * scale[:, None]).view(-1)[:n]


def _adamw_plain(q, step, bits):
    g = q["grads"].float()
    m, v = (q["m"], q["v"]) if bits == 32 else (_unpack_plain(q["m"], q["m_scale"]),
                                                _unpack_plain(q["v"], q["v_scale"]).square())
    m = m * BETAS[0] + g * (1.0 - BETAS[0])
    v = v * BETAS[1] + (g * g) * (1.0 - BETAS[1])
    p = (q["params"] if q["masters"] is None else q["masters"]).float()
    root = torch.sqrt(v)
    update = m / (root * (1.0 / math.sqrt(1.0 - BETAS[1] ** step)) + ADAM_EPS) * (RATE / (1.0 - BETAS[0] ** step))
    p = p * (1.0 - RATE * q["decay"]) - update
    q["params"].copy_(p)
    if q["masters"] is not None:
        q["masters"].copy_(p)
    if bits == 32:
        q["m"].copy_(m)
        q["v"].copy_(v)
        return
    for key, t in (("m", m), ("v", root)):
        code, scale = _pack_plain(t, key == "v")
        q[key].copy_(code)
        q[key + "_scale"].copy_(scale)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "gated_fwd":
        x = s["x"].float()
        gate, up = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
        y = (_act_plain(case["act"], gate)[0] * up).to(s["x"].dtype)
        return (y, torch.stack([gate, up]).to(s["x"].dtype)) if case["keep"] else y
    if op == "gated_bwd":
        dt = s["x"].dtype
        gate, up, gy = s["pre"][0].float(), s["pre"][1].float(), s["grad_y"].float()
        a, slope = _act_plain(case["act"], gate)
        d_gate, d_up = gy * up * slope, gy * a
        x = s["x"].float()
        gx = d_gate @ s["w_gate"].float() + d_up @ s["w_up"].float()
        return gx.to(dt), (d_gate.t() @ x).to(dt), (d_up.t() @ x).to(dt)
    if op == "norms_fwd":
        return _norms_plain(s)
    if op == "norms_bwd":
        return _norms_grad_plain(s)
    _adamw_plain(s["groups"][0], s["step"], case["bits"])
    _adamw_plain(s["groups"][1], s["step"], case["bits"])
    return _adamw_outputs(s)


# ---------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------

def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op.startswith("gated"):
        N, D, F = case["N"], case["D"], case["F"]
        if op == "gated_fwd":
            return {"bytes": (N * D + 2 * F * D + (3 if case["keep"] else 1) * N * F) * e, "flops": 4 * N * D * F}
        return {"bytes": (3 * N * F + 2 * N * D + 4 * F * D) * e, "flops": 8 * N * D * F}
    if op.startswith("norms"):
        N, D = case["N"], case["D"]
        rows = N * D * e
        vectors = (1 + (case["gate"] == "columns") + case["post"]) * D * BYTES[case["params"]]
        gates = rows if case["gate"] == "rows" else 0
        stats = 4 * N * (1 + case["post"])
        if op == "norms_fwd":
            return {"bytes": 4 * rows + gates + vectors + stats, "flops": 12 * N * D}
        branch = rows if case["post"] or case["gate"] != "none" else 0
        return {"bytes": 5 * rows + branch + 2 * gates + 2 * vectors + stats, "flops": 24 * N * D}
    total = 0.0
    for sizes, p, g in zip(_adamw_sizes(case), (e, 4), (BYTES[case["grads"]], 4)):
        master = 8 if case["masters"] and p != 4 else 0
        param = p if master else 2 * p  # with masters the parameters are only written
        state = 16 if case["bits"] == 32 else 4 + 16.0 / BLOCK
        total += sum(sizes) * (param + master + g + state)
    return {"bytes": total, "flops": 15 * sum(sum(sizes) for sizes in _adamw_sizes(case))}


# ---------------------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _phi(act, z):
    """The activation, in place of z's own values."""
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -(0.5 ** 0.5))
    return z * torch.sigmoid(2.0 * (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))


def _slope(act, z):
    """Its derivative, by automatic differentiation."""
    with torch.enable_grad():
        z = z.detach().requires_grad_(True)
        return torch.autograd.grad(_phi(act, z).sum(), z)[0]


def _round8(x):
    """To the nearest value of one sign, four exponent and three fraction bits, halves to even."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.clamp(a, min=2.0 ** -6)))
    e = e + (a >= torch.exp2(e + 1)).double() - (a < torch.exp2(e)).double() * (e > -6)
    unit = torch.exp2(e - 3)
    return torch.sign(x) * torch.clamp(torch.round(a / unit) * unit, max=TOP)


def _blocks(t):
    out = torch.zeros(-(-t.numel() // BLOCK) * BLOCK, dtype=torch.float64, device=t.device)
    out[:t.numel()] = t
    return out.view(-1, BLOCK)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated_fwd":
        x = s["x"].double()
        pre = torch.stack([torch.einsum("nd,fd->nf", x, s[k].double()) for k in ("w_gate", "w_up")])
        y = _phi(case["act"], pre[0]) * pre[1]
        return (y, pre) if case["keep"] else y
    if op == "gated_bwd":
        gy, gate, up = s["grad_y"].double(), s["pre"][0].double(), s["pre"][1].double()
        up.mul_(gy).mul_(_slope(case["act"], gate))
        gy.mul_(_phi(case["act"], gate))
        del gate
        x = s["x"].double()
        gx = torch.einsum("nf,fd->nd", up, s["w_gate"].double()) + torch.einsum("nf,fd->nd", gy, s["w_up"].double())
        return gx, torch.einsum("nf,nd->fd", up, x), torch.einsum("nf,nd->fd", gy, x)
    if op == "norms_fwd":
        x, b, D = s["x"].double(), s["branch"].double(), case["D"]
        post_rstd = None
        if case["post"]:
            post_rstd = (torch.einsum("nd,nd->n", b, b) / D + EPS) ** -0.5
            b = torch.einsum("nd,n,d->nd", b, post_rstd, s["post_weight"].double())
        if s["gate"] is not None:
            b = b * s["gate"].double()
        x = x + s["scale"] * b
        rstd = (torch.einsum("nd,nd->n", x, x) / D + EPS) ** -0.5
        return x, torch.einsum("nd,n,d->nd", x, rstd, s["weight"].double()), post_rstd, rstd
    if op == "norms_bwd":
        st, b, gh, D = s["stream"].double(), s["branch"].double(), s["grad_h"].double(), case["D"]
        r, w = s["rstd"].double(), s["weight"].double()
        along = torch.einsum("nd,nd,d->n", gh, st, w) * r ** 3 / D
        gx = s["grad_stream"].double() + gh * w * r[:, None] - st * along[:, None]
        g_weight = torch.einsum("nd,nd,n->d", gh, st, r)
        gate = torch.ones((), device=st.device, dtype=torch.float64) if s["gate"] is None else s["gate"].double()
        pr = s["post_rstd"].double() if case["post"] else torch.ones_like(r)
        pw = s["post_weight"].double() if case["post"] else torch.ones_like(w)
        g_gate = None
        if s["gate"] is not None:
            g_gate = gx * b * pr[:, None] * pw * s["scale"]
            g_gate = g_gate if s["gate"].dim() == 2 else g_gate.sum(0)
        gn = gx * gate * s["scale"]
        if not case["post"]:
            return gx, gn, g_gate, None, g_weight
        g_post = torch.einsum("nd,nd,n->d", gn, b, pr)
        gn = gn * pw
        gb = gn * pr[:, None] - b * (torch.einsum("nd,nd->n", gn, b) * pr ** 3 / D)[:, None]
        return gx, gb, g_gate, g_post, g_weight
    out = []
    for q in s["groups"]:
        p = (q["params"] if q["masters"] is None else q["masters"]).double()
        g, n = q["grads"].double(), q["grads"].numel()
        if case["bits"] == 8:
            m = (_blocks(q["m"].double()) * q["m_scale"].double()[:, None]).view(-1)[:n]
            v = (_blocks(q["v"].double()) * q["v_scale"].double()[:, None]).view(-1)[:n] ** 2
        else:
            m, v = q["m"].double(), q["v"].double()
        m = m + (1 - BETAS[0]) * (g - m)
        v = v + (1 - BETAS[1]) * (g * g - v)
        m_hat, v_hat = m / (1 - BETAS[0] ** s["step"]), v / (1 - BETAS[1] ** s["step"])
        p = p - RATE * (m_hat / (v_hat ** 0.5 + ADAM_EPS) + q["decay"] * p)
        r = {"params": p, "masters": None if q["masters"] is None else p, "m": m, "v": v, "m_scale": None,
             "v_scale": None}
        if case["bits"] == 8:
            for key, t in (("m", m), ("v", v ** 0.5)):
                b = _blocks(t)
                r[key + "_scale"] = b.abs().max(1).values / TOP
                c = _round8(b / torch.where(r[key + "_scale"] > 0, r[key + "_scale"], 1.0)[:, None])
                if key == "v":
                    c = torch.where((b > 0) & (c < LEAST), LEAST, c)
                r[key] = c.view(-1)[:n]
        out.append(r)
    return out
