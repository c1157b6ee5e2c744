"""One training step of a small language model with a tied table, end to end through this package:

    tokens -> embedding (scaled) -> dropout -> blocks of x + dropout(mlp(layer_norm(x)))
           -> layer_norm -> linear_logp -> loss

The table [V, D] is the embedding at the input and the LM head at the output.  Its gradient is
written once, by the head's backward, and the embedding's is added to the rows that the tokens
name (``embedding_bwd(..., accumulate=True)``): no second [V, D] gradient is formed or summed.
Dropout masks are numbered by (seed, offset) and never stored.

    python examples/tied_lm_step.py [--tokens 4096] [--hidden 512] [--vocab 8192] [--steps 30]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lm_head_selected_gb300 as llp  # noqa: E402


class TiedLM:
    def __init__(self, vocab: int, hidden: int, layers: int = 2, p: float = 0.1, seed: int = 0,
                 dtype: torch.dtype = torch.bfloat16, device: str = "cuda"):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(device=device, dtype=dtype)

        self.V, self.D, self.p, self.seed = vocab, hidden, p, seed
        self.scale = math.sqrt(hidden)
        self.table = normal(vocab, hidden, std=1.0 / math.sqrt(hidden))
        self.blocks = [{"w": torch.ones(hidden, device=device), "b": torch.zeros(hidden, device=device),
                        "up": normal(hidden, 2 * hidden, std=1.0 / math.sqrt(hidden)),
                        "down": normal(2 * hidden, hidden, std=0.5 / math.sqrt(2 * hidden))} for _ in range(layers)]
        self.norm = {"w": torch.ones(hidden, device=device), "b": torch.zeros(hidden, device=device)}
        for t in self._inner():
            t.requires_grad_(True)

    def _inner(self):
        """Every parameter but the table."""
        return [t for blk in self.blocks + [self.norm] for t in blk.values()]

    def body(self, x: torch.Tensor, step: int) -> torch.Tensor:
        """Embedded tokens [N, D] -> the head's input; masks are numbered from step and layer."""
        offset = step * (len(self.blocks) + 1)
        h = llp.dropout(x, self.p, self.seed, offset)
        for i, blk in enumerate(self.blocks):
            up = llp.layer_norm(h, blk["w"], blk["b"]) @ blk["up"]
            h = llp.dropout(torch.nn.functional.gelu(up) @ blk["down"], self.p, self.seed, offset + 1 + i, residual=h)
        return llp.layer_norm(h, self.norm["w"], self.norm["b"])

    def gradients(self, tokens: torch.Tensor, targets: torch.Tensor, step: int):
        """(loss, gradient of the table, gradients of the other parameters)."""
        x = llp.embedding_fwd(tokens, self.table, self.scale).requires_grad_(True)
        y = self.body(x, step)
        with torch.no_grad():
            logp, lse = llp.linear_logp_fwd(y, self.table, targets)
            valid = torch.isfinite(lse)
            n = valid.sum().clamp(min=1)
            loss = -logp.sum() / n
            grad_logp = torch.where(valid, -1.0 / n, 0.0).float()
            gy, g_table, _ = llp.linear_logp_bwd(grad_logp, lse, y, self.table, targets)
        inner = self._inner()
        grads = torch.autograd.grad(y, [x] + inner, gy)
        llp.embedding_bwd(grads[0], tokens, self.V, self.scale, out=g_table, accumulate=True)
        return loss, g_table, list(zip(inner, grads[1:]))

    def step(self, tokens: torch.Tensor, targets: torch.Tensor, step: int, lr: float) -> torch.Tensor:
        loss, g_table, inner = self.gradients(tokens, targets, step)
        with torch.no_grad():
            self.table.sub_(lr * g_table)
            for p, g in inner:
                p.sub_(lr * g)
        return loss


def batch(n: int, vocab: int, seed: int, device: str = "cuda"):
    """Tokens whose successor is a fixed function of the token; one target in 32 is ignored."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, vocab, (n,), generator=g)
    nxt = (t * 5 + 7) % vocab
    nxt[torch.rand(n, generator=g) < 1 / 32] = llp.IGNORE_INDEX
    return t.to(device), nxt.to(device)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--lr", type=float, default=2.0)
    a = ap.parse_args()
    model = TiedLM(a.vocab, a.hidden)
    tokens, targets = batch(a.tokens, a.vocab, seed=1)
    for i in range(a.steps):
        loss = model.step(tokens, targets, i, a.lr)
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  loss {float(loss):.4f}")
    if llp.device_status() != 0:
        raise RuntimeError("a kernel gave up on a bounded wait")


if __name__ == "__main__":
    main()
