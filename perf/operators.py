"""The operators around the LM head, as measured cases: the embedding lookup and its gradient, layer norm and its
gradient, dropout and its gradient.

``run`` computes one pass.  With ``own`` false it is the plain form: elementary torch operations in 32 bits, rounded
once at the end.  With ``own`` true it is the call into this package.  ``exact`` is the definition in 64 bits.
Sizes are the ones of this repository's workloads (hidden 2688 and vocabulary 131072; hidden 4096 and vocabulary
128256; 32, 16384 and 65600 tokens) and generic odd ones.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def listed():
    return [
        # the tokens of one decoding step of 32 sequences; latency counts
        {"name": "embedding decode", "op": "embedding_fwd", "N": 32, "D": 2688, "V": 131072, "dtype": "bf16",
         "scale": 1.0},
        # a rollout batch's prompt and response tokens, table scaled by sqrt(hidden)
        {"name": "embedding batch", "op": "embedding_fwd", "N": 16384, "D": 2688, "V": 131072, "dtype": "bf16",
         "scale": math.sqrt(2688.0)},
        # a small fp32 model with an odd hidden size: rows start at any 4-byte boundary
        {"name": "embedding grad odd", "op": "embedding_bwd", "N": 2049, "D": 1001, "V": 50257, "dtype": "fp32",
         "scale": 1.0, "accumulate": False},
        # the training batch's untied table: every row of the gradient is written
        {"name": "embedding grad", "op": "embedding_bwd", "N": 16384, "D": 2688, "V": 131072, "dtype": "bf16",
         "scale": math.sqrt(2688.0), "accumulate": False},
        # a table tied to the LM head: the head's gradient is there already, and the tokens' rows are added to it
        {"name": "embedding grad tied", "op": "embedding_bwd", "N": 16384, "D": 4096, "V": 128256, "dtype": "bf16",
         "scale": 1.0, "accumulate": True},
        # the final norm of one decoding step of 32 sequences; latency counts
        {"name": "norm decode", "op": "layer_norm_fwd", "N": 32, "D": 2688, "dtype": "bf16", "params": "bf16"},
        # the final norm of a training batch
        {"name": "norm batch", "op": "layer_norm_fwd", "N": 16384, "D": 2688, "dtype": "bf16", "params": "bf16"},
        # a small batch in fp16 with fp32 parameters
        {"name": "norm grad small", "op": "layer_norm_bwd", "N": 257, "D": 1000, "dtype": "fp16", "params": "fp32"},
        # the training batch at hidden 4096
        {"name": "norm grad", "op": "layer_norm_bwd", "N": 16384, "D": 4096, "dtype": "bf16", "params": "bf16"},
        # a long-context batch with fp32 parameters
        {"name": "norm grad long", "op": "layer_norm_bwd", "N": 65600, "D": 2688, "dtype": "bf16", "params": "fp32"},
        # a residual branch of a training batch: residual + dropout(branch)
        {"name": "dropout residual", "op": "dropout_fwd", "N": 16384, "D": 2688, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # the gradient through dropout in a small fp32 model with an odd hidden size
        {"name": "dropout grad odd", "op": "dropout_bwd", "N": 1111, "D": 1001, "dtype": "fp32", "p": 0.25,
         "residual": False},
    ]


MOST_BYTES = 1.1e9  # of a drawn case: the long layer norm gradient's


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["embedding_fwd", "embedding_bwd", "embedding_bwd", "layer_norm_fwd", "layer_norm_bwd",
                         "dropout_fwd", "dropout_bwd"])
        case = {"op": op,
                "N": rng.choice([_spread(rng, 1, 65600) | 1, _spread(rng, 1, 65600) | 1, 32, 512, 4096, 16384]),
                "D": rng.choice([_spread(rng, 24, 3000), 8 * _spread(rng, 4, 380), 2048, 2688, 4096]),
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
        if op.startswith("embedding"):
            case["V"] = rng.choice([_spread(rng, 100, 131072) | 1, 32768, 50257, 131072])
            case["scale"] = rng.choice([1.0, math.sqrt(case["D"])])
        if op == "embedding_bwd":
            case["accumulate"] = rng.random() < 0.5
        if op.startswith("layer_norm"):
            case["params"] = rng.choice([case["dtype"], "fp32"])
        if op.startswith("dropout"):
            case["p"] = rng.choice([0.05, 0.1, 0.25, 0.5])
            case["residual"] = op == "dropout_fwd" and rng.random() < 0.5
        if work(case)["bytes"] <= MOST_BYTES:
            return case


# ---------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------

def _tokens(case, g, dev):
    """Token ids whose frequency falls as 1 / (id + 1), as merge-ordered vocabularies have it; one in 64 is padding."""
    u = torch.rand(case["N"], generator=g, device=dev, dtype=torch.float64)
    t = (torch.exp(u * math.log(case["V"] + 1.0)).long() - 1).clamp_(0, case["V"] - 1)
    pad = torch.rand(case["N"], generator=g, device=dev) < 1.0 / 64
    return torch.where(pad, torch.full_like(t, IGNORE), t)


def _normal(shape, g, dev, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op, N, D = case["op"], case["N"], case["D"]
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if op.startswith("embedding"):
        s["tokens"] = _tokens(case, g, dev)
        if op == "embedding_fwd":
            s["weight"] = _normal((case["V"], D), g, dev, dt, 0.02)
        else:
            s["grad_out"] = _normal((N, D), g, dev, dt)
            if case["accumulate"]:
                s["grad_weight"] = _normal((case["V"], D), g, dev, dt)
    elif op.startswith("layer_norm"):
        # hidden states: columns of their own offset and width, a few of them far wider than the rest
        wide = torch.where(torch.rand(D, generator=g, device=dev) < 0.01, 20.0, 1.0)
        x = torch.randn((N, D), generator=g, device=dev) * wide + torch.randn(D, generator=g, device=dev) + 0.25
        s["x"] = x.to(dt)
        s["weight"] = (1.0 + _normal((D,), g, dev, torch.float32, 0.2)).to(DTYPES[case["params"]])
        s["bias"] = _normal((D,), g, dev, DTYPES[case["params"]], 0.2)
        if op == "layer_norm_bwd":
            s["grad_y"] = _normal((N, D), g, dev, dt)
            xf = s["x"].float()  # the statistics that the forward pass kept
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
    else:
        s["x"] = _normal((N, D), g, dev, dt)
        s["residual"] = _normal((N, D), g, dev, dt) if case["residual"] else None
        s["seed"] = int(seed) * 0x9E3779B97F4A7C15 % (1 << 63)
        s["offset"] = int(seed) % 1000
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
    if op == "embedding_fwd":
        return llp.embedding_fwd(s["tokens"], s["weight"], case["scale"], IGNORE)
    if op == "embedding_bwd":
        if case["accumulate"]:
            return llp.embedding_bwd(s["grad_out"], s["tokens"], case["V"], case["scale"], IGNORE,
                                     out=s["grad_weight"], accumulate=True)
        return llp.embedding_bwd(s["grad_out"], s["tokens"], case["V"], case["scale"], IGNORE)
    if op == "layer_norm_fwd":
        return llp.layer_norm_fwd(s["x"], s["weight"], s["bias"], EPS)
    if op == "layer_norm_bwd":
        return llp.layer_norm_bwd(s["grad_y"], s["x"], s["mean"], s["rstd"], s["weight"])
    if op == "dropout_fwd":
        return llp.dropout_fwd(s["x"], case["p"], s["seed"], s["offset"], residual=s["residual"])
    return llp.dropout_bwd(s["x"], case["p"], s["seed"], s["offset"])


def _keep_plain(n, p, seed, offset, dev):
    """Whether each of n elements is kept: 16-bit lanes of Philox4x32-10 blocks, eight elements to a block.  Products
    of two 32-bit numbers wrap in int64; their high halves are right all the same."""
    lo32 = 0xFFFFFFFF
    block = torch.arange((n + 7) // 8, device=dev, dtype=torch.int64)
    c0, c1 = block & lo32, block >> 32
    c2, c3 = torch.full_like(block, offset & lo32), torch.full_like(block, offset >> 32)
    k0, k1 = seed & lo32, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & lo32) ^ c1 ^ k0, b & lo32, ((a >> 32) & lo32) ^ c3 ^ k1, a & lo32
        k0, k1 = (k0 + 0x9E3779B9) & lo32, (k1 + 0xBB67AE85) & lo32
    words = torch.stack([c0, c1, c2, c3], 1)
    lanes = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    return lanes >= _threshold(p)


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op.startswith("embedding"):
        t, V = s["tokens"], case["V"]
        ok = (t != IGNORE) & (t >= 0) & (t < V)
        at = torch.where(ok, t, torch.zeros_like(t))
        if op == "embedding_fwd":
            return torch.where(ok[:, None], s["weight"][at].float() * case["scale"], 0.0).to(dt)
        g = torch.where(ok[:, None], s["grad_out"].float() * case["scale"], 0.0)
        if not case["accumulate"]:
            return torch.zeros((V, case["D"]), device=t.device).index_add_(0, at, g).to(dt)
        s["grad_weight"].copy_(s["grad_weight"].float().index_add_(0, at, g))
        return s["grad_weight"]
    if op == "layer_norm_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = torch.rsqrt(c.square().mean(1) + EPS)
        y = c * rstd[:, None] * s["weight"].float() + s["bias"].float()
        return y.to(dt), mean, rstd
    if op == "layer_norm_bwd":
        pt = DTYPES[case["params"]]
        g = s["grad_y"].float()
        h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        a = g * s["weight"].float()
        gx = (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True)) * s["rstd"][:, None]
        return gx.to(dt), (g * h).sum(0).to(pt), g.sum(0).to(pt)
    x = s["x"].float()
    keep = _keep_plain(x.numel(), case["p"], s["seed"], s["offset"], x.device).view_as(x)
    y = torch.where(keep, x * (65536.0 / (65536 - _threshold(case["p"]))), 0.0)
    if case["residual"]:
        y = y + s["residual"].float()
    return y.to(dt)


# ---------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------

def _distinct(N, V):
    """Expected number of distinct valid ids among N of _tokens()."""
    v = torch.arange(1, V + 1, dtype=torch.float64)
    p = torch.log1p(1.0 / v) / math.log(V + 1.0) * (63.0 / 64)
    return float((-torch.expm1(N * torch.log1p(-p.clamp(max=1.0 - 1e-12)))).sum())


def work(case):
    op, N, D, e = case["op"], case["N"], case["D"], BYTES[case["dtype"]]
    rows = N * D * e
    if op == "embedding_fwd":
        return {"bytes": 8 * N + _distinct(N, case["V"]) * D * e + rows, "flops": N * D}
    if op == "embedding_bwd":
        out = 2 * _distinct(N, case["V"]) * D * e if case["accumulate"] else case["V"] * D * e
        return {"bytes": 8 * N + rows + out, "flops": 2 * N * D}
    if op == "layer_norm_fwd":
        return {"bytes": 2 * rows + 8 * N + 2 * D * BYTES[case["params"]], "flops": 8 * N * D}
    if op == "layer_norm_bwd":
        return {"bytes": 3 * rows + 8 * N + 3 * D * BYTES[case["params"]], "flops": 14 * N * D}
    return {"bytes": (3 if case["residual"] else 2) * rows, "flops": 2 * N * D}


# ---------------------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _kept_exact(n, p, seed, offset):
    """The kept elements by Philox4x32-10 in numpy's unsigned 64-bit arithmetic."""
    import numpy as np
    m, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    i = np.arange(-(-n // 8), dtype=np.uint64)
    c = [i & m, i >> sh, np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for r in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        ka = np.uint64((key[0] + r * 0x9E3779B9) % (1 << 32))
        kb = np.uint64((key[1] + r * 0xBB67AE85) % (1 << 32))
        c = [(p1 >> sh) ^ c[1] ^ ka, p1 & m, (p0 >> sh) ^ c[3] ^ kb, p0 & m]
    lanes = np.empty((i.size, 8), dtype=np.int64)
    for w in range(4):
        lanes[:, 2 * w] = (c[w] & np.uint64(0xFFFF)).astype(np.int64)
        lanes[:, 2 * w + 1] = (c[w] >> np.uint64(16)).astype(np.int64)
    return torch.from_numpy(lanes.reshape(-1)[:n] >= math.floor(p * 65536 + 0.5))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embedding_fwd":
        t = s["tokens"]
        out = torch.zeros((case["N"], case["D"]), dtype=torch.float64, device=t.device)
        ok = torch.nonzero((t >= 0) & (t < case["V"]) & (t != IGNORE)).flatten()
        out[ok] = s["weight"].index_select(0, t[ok]).double() * case["scale"]
        return out
    if op == "embedding_bwd":
        # running sums over the tokens in sorted order; a row is the difference at its segment's two ends
        t = s["tokens"]
        ok = torch.nonzero((t >= 0) & (t < case["V"]) & (t != IGNORE)).flatten()
        order = ok[torch.sort(t[ok], stable=True).indices]
        run_sum = torch.zeros((order.numel() + 1, case["D"]), dtype=torch.float64, device=t.device)
        torch.cumsum(s["grad_out"][order].double() * case["scale"], 0, out=run_sum[1:])
        ids, counts = torch.unique_consecutive(t[order], return_counts=True)
        end = torch.cumsum(counts, 0)
        out = (s["grad_weight"].double() if case["accumulate"]
               else torch.zeros((case["V"], case["D"]), dtype=torch.float64, device=t.device))
        out[ids] += run_sum[end] - run_sum[end - counts]
        return out
    if op == "layer_norm_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        return ((x - mean[:, None]) * rstd[:, None] * s["weight"].double() + s["bias"].double(), mean, rstd)
    if op == "layer_norm_bwd":
        x, g, D = s["x"].double(), s["grad_y"].double(), case["D"]
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        x.sub_(mean[:, None]).mul_(rstd[:, None])
        gw, gb = torch.einsum("nd,nd->d", g, x), torch.einsum("nd->d", g)
        g.mul_(s["weight"].double())
        along = torch.einsum("nd,nd->n", g, x) / D
        g.sub_(torch.einsum("nd->n", g)[:, None] / D).sub_(x.mul_(along[:, None])).mul_(rstd[:, None])
        return g, gw, gb
    x = s["x"].double()
    keep = _kept_exact(x.numel(), case["p"], s["seed"], s["offset"]).to(x.device).view_as(x)
    y = x * keep * (1.0 / (1.0 - math.floor(case["p"] * 65536 + 0.5) / 65536.0))
    return y + s["residual"].double() if case["residual"] else y
