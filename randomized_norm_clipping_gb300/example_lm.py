"""A small language model trained with DP-SGD-RC on the library's operators.

    python -m randomized_norm_clipping_gb300.example_lm [--steps 60] [--dtype bf16] [--heads 4]

Embedding (scaled) -> residual MLP blocks (normalisation, up map with GELU and
bias, down map with bias, dropout and the residual in its epilogue) -> head.  With
heads, a block begins with attention (trained normalisation, one map to queries, keys and
values, rotary positions, causal attention, a map back onto the residual).
Each step: forward, per-sample losses, `RandomizedClippingStep` (per-sample
norms of the embedding, the biases and the linear weights; clip factors; the
clipped gradient sum; noise), an SGD update.  The data is a synthetic Markov
chain, so the loss has something to learn; no dataset is needed.
"""

from __future__ import annotations

import argparse

import torch

from . import binding as rnc
from .layers import Attention, Embedding, LayerNorm, Linear, rotary_freqs
from .step import RandomizedClippingStep


class Mixer(torch.nn.Module):
    """Attention onto the residual: `heads` heads of queries, half as many of keys."""

    def __init__(self, width, heads, p, seed, dtype):
        super().__init__()
        kv, d = max(1, heads // 2), width // heads
        self.norm = LayerNorm(width, center=False, bias=False, dtype=dtype)
        self.rows = Linear(width, (heads + 2 * kv) * d, dtype=dtype)
        self.attention = Attention(heads, kv, d, freqs=rotary_freqs(d // 2))
        self.back = Linear(heads * d, width, p=p, seed=seed, dtype=dtype)

    def forward(self, x, docs=None):
        return self.back(self.attention(self.rows(self.norm(x)), docs=docs), residual=x)

    def cache(self, B, T, device):
        """Room for the keys and values of T tokens."""
        a = self.attention
        shape = (2, B, T, a.kv_heads, a.width)
        return torch.zeros(shape, dtype=self.rows.weight.dtype, device=device)

    @torch.no_grad()
    def extend(self, x, cache, at):
        """The new tokens x [B][n][width], which stand at positions at [B] and on, over the
        cache and themselves; their keys and values are put into it."""
        a = self.attention
        B, n, _ = x.shape
        H, Hkv = a.heads, a.kv_heads
        rows = self.rows(self.norm(x)).view(B, n, H + 2 * Hkv, a.width)
        pos = at[:, None] + torch.arange(n, dtype=torch.int32, device=x.device)
        qk = rnc.dprc_rotary(rows[:, :, :H + Hkv], pos, a.freqs)
        b = torch.arange(B, device=x.device)[:, None]
        cache[0, b, pos.long()] = qk[:, :, H:]
        cache[1, b, pos.long()] = rows[:, :, H + Hkv:]
        out = rnc.dprc_attention(qk[:, :, :H], cache[0], cache[1], lengths=at + n, first=at)
        return self.back(out.view(B, n, -1), residual=x)


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

    def __init__(self, vocab=256, width=128, hidden=512, blocks=2, p=0.1, dtype=torch.bfloat16,
                 heads=0):
        super().__init__()
        self.embed = Embedding(vocab, width, scale=width ** -0.5, dtype=dtype)
        self.blocks = torch.nn.ModuleList(
            Block(width, hidden, p, 1000 + i, dtype) for i in range(blocks))
        self.mixers = torch.nn.ModuleList(
            Mixer(width, heads, p, 2000 + i, dtype) for i in range(blocks if heads else 0))
        self.norm = torch.nn.LayerNorm(width, elementwise_affine=False, dtype=dtype)
        self.head = Linear(width, vocab, dtype=dtype)

    def forward(self, tokens, docs=None):
        x = self.embed(tokens)
        if not self.mixers:
            x = x + torch.nn.functional.pad(x, (0, 0, 1, -1))  # the token before
        for i, block in enumerate(self.blocks):
            if self.mixers:
                x = self.mixers[i](x, docs)
            x = block(x)
        return self.head(self.norm(x))

    @torch.no_grad()
    def generate(self, tokens, n):
        """n tokens behind tokens [B][T], the likeliest each time, over a cache of keys and
        values (a model with heads, out of training)."""
        B, T = tokens.shape
        caches = [m.cache(B, T + n, tokens.device) for m in self.mixers]
        new, out = tokens, []
        at = torch.zeros(B, dtype=torch.int32, device=tokens.device)
        for _ in range(n):
            x = self.embed(new)
            for mixer, block, cache in zip(self.mixers, self.blocks, caches):
                x = block(mixer.extend(x, cache, at))
            at = at + new.shape[1]
            new = self.head(self.norm(x[:, -1:])).argmax(-1)
            out.append(new)
        return torch.cat(out, 1)


def markov_batch(generator, B, T, vocab):
    """Each token is, nine times in ten, a fixed function of the one before."""
    t = torch.randint(0, vocab, (B, T + 1), generator=generator)
    follow = torch.rand(B, T, generator=generator) < 0.9
    for i in range(T):
        t[:, i + 1] = torch.where(follow[:, i], (5 * t[:, i] + 7) % vocab, t[:, i + 1])
    return t


def train(steps=60, B=16, T=64, vocab=256, C=1.0, sigma=0.05, lr=4.0, dtype=torch.bfloat16,
          seed=0, device="cuda", heads=0):
    """The mean loss of every step."""
    torch.manual_seed(seed)
    model = TinyLM(vocab, dtype=dtype, heads=heads).to(device)
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
    ap.add_argument("--heads", type=int, default=0)
    a = ap.parse_args()
    loss = train(a.steps, dtype=torch.bfloat16 if a.dtype == "bf16" else torch.float32,
                 heads=a.heads)
    for i in range(0, len(loss), 10):
        print(f"step {i:4d}  mean loss {loss[i]:.4f}")
    print(f"last       mean loss {loss[-1]:.4f}")


if __name__ == "__main__":
    main()
