"""A small language model trained with DP-SGD-RC on the library's operators.

    python -m randomized_norm_clipping_gb300.example_lm [--steps 60] [--dtype bf16]

Embedding (scaled) -> residual MLP blocks (normalisation, up map with GELU and
bias, down map with bias, dropout and the residual in its epilogue) -> head.
Each step: forward, per-sample losses, `RandomizedClippingStep` (per-sample
norms of the embedding, the biases and the linear weights; clip factors; the
clipped gradient sum; noise), an SGD update.  The data is a synthetic Markov
chain, so the loss has something to learn; no dataset is needed.
"""

from __future__ import annotations

import argparse

import torch

from .layers import Embedding, Linear
from .step import RandomizedClippingStep


class Block(torch.nn.Module):
    def __init__(self, width, hidden, p, seed, dtype):
        super().__init__()
        self.norm = torch.nn.LayerNorm(width, elementwise_affine=False, dtype=dtype)
        self.up = Linear(width, hidden, bias=True, act="gelu", dtype=dtype)
        self.down = Linear(hidden, width, bias=True, p=p, seed=seed, dtype=dtype)

    def forward(self, x):
        return self.down(self.up(self.norm(x)), residual=x)


class TinyLM(torch.nn.Module):
    """Next-token model over the current token and the one before it."""

    def __init__(self, vocab=256, width=128, hidden=512, blocks=2, p=0.1, dtype=torch.bfloat16):
        super().__init__()
        self.embed = Embedding(vocab, width, scale=width ** -0.5, dtype=dtype)
        self.blocks = torch.nn.ModuleList(
            Block(width, hidden, p, 1000 + i, dtype) for i in range(blocks))
        self.norm = torch.nn.LayerNorm(width, elementwise_affine=False, dtype=dtype)
        self.head = Linear(width, vocab, dtype=dtype)

    def forward(self, tokens):
        x = self.embed(tokens)
        x = x + torch.nn.functional.pad(x, (0, 0, 1, -1))  # the token before
        for block in self.blocks:
            x = block(x)
        return self.head(self.norm(x))


def markov_batch(generator, B, T, vocab):
    """Each token is, nine times in ten, a fixed function of the one before."""
    t = torch.randint(0, vocab, (B, T + 1), generator=generator)
    follow = torch.rand(B, T, generator=generator) < 0.9
    for i in range(T):
        t[:, i + 1] = torch.where(follow[:, i], (5 * t[:, i] + 7) % vocab, t[:, i + 1])
    return t


def train(steps=60, B=16, T=64, vocab=256, C=1.0, sigma=0.05, lr=4.0, dtype=torch.bfloat16,
          seed=0, device="cuda"):
    """The mean loss of every step."""
    torch.manual_seed(seed)
    model = TinyLM(vocab, dtype=dtype).to(device)
    step = RandomizedClippingStep(model, C=C, sigma=sigma, k=32, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    history = []
    for it in range(steps):
        t = markov_batch(g, B, T, vocab).to(device)
        logits = model(t[:, :-1])
        losses = torch.nn.functional.cross_entropy(
            logits.float().transpose(1, 2), t[:, 1:], reduction="none").mean(1)
        step(losses, step=it)
        with torch.no_grad():
            for prm in step.parameters():
                prm -= (lr / B) * prm.grad
        history.append(losses.detach().mean())
    step.close()
    return [float(x) for x in history]


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    loss = train(a.steps, dtype=torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    for i in range(0, len(loss), 10):
        print(f"step {i:4d}  mean loss {loss[i]:.4f}")
    print(f"last       mean loss {loss[-1]:.4f}")


if __name__ == "__main__":
    main()
