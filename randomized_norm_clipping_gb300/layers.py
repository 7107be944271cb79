"""torch.nn modules over the operators around the norm path.

`Embedding`, `Linear` (bias, activation, dropout and residual in one call),
`Dropout`, `LayerNorm` (also its RMS form) and `Attention` (with rotary positions)
run on libdprc (dprc_embed_*, dprc_linear*, dprc_dropout, dprc_layernorm*,
dprc_rotary, dprc_attention*) in both directions, and `RandomizedClippingStep` takes
their parameters: the embedding, the biases and the normalisations by their exact
per-sample norms, the linear weights by the estimates.  Device tensors of float32 or
bfloat16 only; the library raises on
anything else.  Gradients can be taken once; a gradient of a gradient raises.

Dropout masks come from the library's Philox stream under (seed, step): `seed`
is the module's (one of its own, in copies too, where none is given), `step` counts
its training forward passes (set `step` to repeat a run; a module with dropout has
both in its state_dict, so that a restored run goes on).  A mask is not stored: the backward passes of one
forward pass, a clipping step has two, draw it again, and so does a forward pass
that activation checkpointing repeats (preserve_rng_state, its default, is needed:
a training forward pass with dropout draws once from torch's CPU generator, by
which its repetition is known).
"""

from __future__ import annotations

import copy
import itertools
import math

import torch
from torch.autograd.function import once_differentiable

from . import binding as rnc


def _dense(t):
    """t as the library takes it: contiguous, from a 16-byte boundary on."""
    if t is None:
        return None
    t = t.detach().contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _in_backward():
    """Whether this runs inside a backward pass (as activation checkpointing's
    repeated forward passes do)."""
    return torch._C._current_graph_task_id() != -1


class _Lookup(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale):
        tokens = _dense(tokens)
        ctx.save_for_backward(tokens)
        ctx.scale, ctx.shape, ctx.dtype = scale, weight.shape, weight.dtype
        return rnc.dprc_embed_lookup(_dense(weight), tokens, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        (tokens,) = ctx.saved_tensors
        V, d = ctx.shape
        flat = tokens.reshape(1, -1)
        plan = rnc.dprc_embed_plan(flat, V)
        dW = torch.empty((V, d), dtype=ctx.dtype, device=grad.device)
        G = _dense(grad.to(ctx.dtype)).view(1, -1, d)
        return None, rnc.dprc_embed_grad(G, plan, dW, scale=ctx.scale), None


class Embedding(torch.nn.Module):
    """Rows of `weight` [num_embeddings][embedding_dim] times `scale`; a
    negative token gives a zero row and has no gradient."""

    def __init__(self, num_embeddings, embedding_dim, scale=1.0, device=None, dtype=None):
        super().__init__()
        self.num_embeddings, self.embedding_dim = int(num_embeddings), int(embedding_dim)
        self.scale = float(scale)
        self.weight = torch.nn.Parameter(
            torch.randn(num_embeddings, embedding_dim, device=device, dtype=dtype))

    def forward(self, tokens):
        return _Lookup.apply(tokens, self.weight, self.scale)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, step):
        ctx.args = (p, seed, step)
        return rnc.dprc_dropout(_dense(x), p, seed, step, residual=_dense(residual))

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        dx = rnc.dprc_dropout(_dense(grad), *ctx.args) if ctx.needs_input_grad[0] else None
        return dx, grad if ctx.needs_input_grad[1] else None, None, None, None


_PASSES_KEPT = 1024
_MASK_KEY = "mask_seed_step"
_modules_built = itertools.count(1)


def _own_seed():
    """A seed that no other module of the process got, from torch's initial seed and
    the number of modules built (Steele, Lea and Flood's splitmix64 of the two)."""
    m = (1 << 64) - 1
    h = (torch.initial_seed() + next(_modules_built) * 0x9E3779B97F4A7C15) & m
    h = ((h ^ (h >> 30)) * 0xBF58476D1CE4E5B9) & m
    h = ((h ^ (h >> 27)) * 0x94D049BB133111EB) & m
    return (h ^ (h >> 31)) >> 1


class _Masked(torch.nn.Module):
    """A module with a dropout mask of its own in every training forward pass."""

    def __init__(self, p, seed):
        super().__init__()
        self.p, self.step = float(p), 0
        self.seed = _own_seed() if seed is None else int(seed)
        self._seed_given = seed is not None
        self._passes = {}

    def __setstate__(self, state):
        super().__setstate__(state)
        self.__dict__.setdefault("_seed_given", True)  # (pickled without these two)
        self.__dict__.setdefault("_passes", {})

    def __deepcopy__(self, memo):
        """A copy, which gets a seed of its own where this module has one."""
        new = self.__class__.__new__(self.__class__)
        memo[id(self)] = new
        new.__dict__.update(copy.deepcopy(self.__dict__, memo))
        if not self._seed_given:
            new.seed = _own_seed()
        return new

    def _save_to_state_dict(self, destination, prefix, keep_vars):
        super()._save_to_state_dict(destination, prefix, keep_vars)
        if self.p > 0.0:  # (else the keys of the plain module)
            signed = (self.seed + (1 << 63)) % (1 << 64) - (1 << 63)
            destination[prefix + _MASK_KEY] = torch.tensor([signed, self.step], device="cpu")

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys,
                              unexpected_keys, error_msgs):
        super()._load_from_state_dict(state_dict, prefix, local_metadata, strict, missing_keys,
                                      unexpected_keys, error_msgs)
        key = prefix + _MASK_KEY
        if key in state_dict:
            seed, self.step = (int(v) for v in state_dict[key])
            self.seed = seed % (1 << 64)
            if key in unexpected_keys:
                unexpected_keys.remove(key)

    def _next_step(self):
        """The step of a training forward pass.  Activation checkpointing runs a pass
        again inside the backward pass, after it has put torch's generators back
        where they were: each pass draws a ticket from the CPU's, and a pass that
        is run again finds its step by that."""
        ticket = int(torch.randint(1 << 62, (), device="cpu"))
        if _in_backward():
            if ticket not in self._passes:
                raise RuntimeError(
                    "a training forward pass inside a backward pass repeats none of the last "
                    f"{_PASSES_KEPT}, so that its dropout mask is unknown; activation checkpointing "
                    "needs preserve_rng_state=True")
            return self._passes[ticket]
        self.step += 1
        self._passes.pop(ticket, None)
        self._passes[ticket] = self.step
        if len(self._passes) > _PASSES_KEPT:
            del self._passes[next(iter(self._passes))]
        return self.step


class Dropout(_Masked):
    """residual + dropout(x); the identity (plus the residual) outside training."""

    def __init__(self, p=0.1, seed=None):
        super().__init__(p, seed)

    def forward(self, x, residual=None):
        if not self.training or self.p == 0.0:
            return x if residual is None else x + residual
        return _Dropout.apply(x, residual, self.p, self.seed, self._next_step())


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, module, p, step, keep):
        x, w = _dense(x), _dense(weight)
        z = None
        if keep and module.act != "none":
            z = torch.empty((*x.shape[:-1], w.shape[0]), dtype=x.dtype, device=x.device)
        ctx.save_for_backward(x, w, z)
        # the module may change before the backward pass: what it was is kept
        ctx.module = module
        ctx.args = dict(act=module.act, p=p, seed=module.seed, step=step)
        if not _in_backward():  # (a repeated pass has its place already)
            module._last = (z, ctx.args)
        return rnc.dprc_linear(x, w, bias=_dense(bias), residual=_dense(residual), Z=z, **ctx.args)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, w, z = ctx.saved_tensors
        last = ctx.module._last
        if last is not None and last[1] is ctx.args:  # Z is kept by the graph alone from here on
            ctx.module._last = None
        grad = _dense(grad)
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        if ctx.module.norm_pass:  # the clipping step's first backward: no weight gradients
            need_w = need_b = False
        dx = torch.empty_like(x) if need_x else None
        dw = torch.empty_like(w) if need_w else None
        db = torch.empty(w.shape[0], dtype=w.dtype, device=w.device) if need_b else None
        if need_x or need_w or need_b:
            rnc.dprc_linear_grad(grad, x, w, Z=z, dX=dx, dW=dw, db=db, **ctx.args)
        return dx, dw, db, grad if need_r else None, None, None, None, None


class Linear(_Masked):
    """residual + dropout(act(x W^T + bias)), in one call."""

    def __init__(self, in_features, out_features, bias=False, act="none", p=0.0, seed=None,
                 device=None, dtype=None):
        super().__init__(p, seed)
        if act not in rnc.DPRC_ACTS:
            raise ValueError(f"act must be one of {sorted(rnc.DPRC_ACTS)}")
        self.in_features, self.out_features = int(in_features), int(out_features)
        self.act = act
        self.norm_pass = False
        self._last = None
        self.weight = torch.nn.Parameter(
            torch.randn(out_features, in_features, device=device, dtype=dtype)
            / math.sqrt(in_features))
        self.bias = (torch.nn.Parameter(torch.zeros(out_features, device=device, dtype=dtype))
                     if bias else None)

    def forward(self, x, residual=None):
        p = self.p if self.training else 0.0
        step = self._next_step() if p > 0.0 else self.step
        return _Linear.apply(x, self.weight, self.bias, residual, self, p, step,
                             torch.is_grad_enabled())

    def preactivation_grad(self, dy, last):
        """The gradient with respect to x W^T + bias, from that with respect to
        the output: what the norm estimates take as G.  `last` is what the
        forward pass left in `_last`."""
        z, args = last
        if args["act"] == "none" and args["p"] == 0.0:
            return dy
        g = torch.empty_like(dy)
        rnc.dprc_linear_grad(dy, None, _dense(self.weight), Z=z, dZ=g, **args)
        return g


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, module, keep):
        x, w = _dense(x), _dense(weight)
        stats = None
        if keep:
            stats = torch.empty((*x.shape[:-1], 2), dtype=torch.float32, device=x.device)
        ctx.save_for_backward(x, w, stats)
        ctx.module, ctx.center = module, module.center
        if not _in_backward():  # (a repeated pass has its place already)
            module._last = stats
        return rnc.dprc_layernorm(x, w, _dense(bias), eps=module.eps, center=module.center,
                                  stats=stats)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, w, stats = ctx.saved_tensors
        if ctx.module._last is stats:  # kept by the graph alone from here on
            ctx.module._last = None
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        if ctx.module.norm_pass:  # the clipping step's first backward: no parameter gradients
            need_w = need_b = False
        grad = _dense(grad)
        dx = torch.empty_like(x) if need_x else None
        dw = torch.empty(x.shape[-1], dtype=x.dtype, device=x.device) if need_w else None
        db = torch.empty(x.shape[-1], dtype=x.dtype, device=x.device) if need_b else None
        if need_x or need_w or need_b:
            rnc.dprc_layernorm_grad(grad, x, stats, w, center=ctx.center, dX=dx, dW=dw, db=db)
        return dx, dw, db, None, None


class LayerNorm(torch.nn.Module):
    """Layer normalisation of the last axis, or with center=False RMS normalisation."""

    def __init__(self, width, eps=1e-5, center=True, weight=True, bias=True, device=None,
                 dtype=None):
        super().__init__()
        self.width, self.eps, self.center = int(width), float(eps), bool(center)
        self.norm_pass = False
        self._last = None
        new = lambda f: torch.nn.Parameter(f(width, device=device, dtype=dtype))  # noqa: E731
        self.weight = new(torch.ones) if weight else None
        self.bias = new(torch.zeros) if bias else None

    def forward(self, x):
        return _LayerNorm.apply(x, self.weight, self.bias, self, torch.is_grad_enabled())


def _heads(t):
    """t as the library takes [B][T][H][D]: any strides, a head's elements together."""
    t = t.detach()
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, freqs, sections, interleaved):
        ctx.save_for_backward(positions, freqs)
        ctx.args = dict(sections=sections, interleaved=interleaved)
        return rnc.dprc_rotary(_heads(x), positions, freqs, **ctx.args)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        positions, freqs = ctx.saved_tensors
        dx = rnc.dprc_rotary(_heads(grad), positions, freqs, inverse=True, **ctx.args)
        return dx, None, None, None, None


def rotary(x, positions, freqs, sections=None, interleaved=False):
    """dprc_rotary with its gradient (by x)."""
    return _Rotary.apply(x, _dense(positions), _dense(freqs), sections, interleaved)


def rotary_freqs(pairs, base=10000.0, sections=None):
    """base^(-p / n) for the pairs p of each section of n (one of them all, if none given)."""
    return torch.cat([base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
                      for n in (sections or [pairs])])


def _plain(mask):
    """The arguments of a mask, dense; the library's types are the caller's to give."""
    for name, t in mask.items():
        if isinstance(t, torch.Tensor):
            if t.requires_grad:
                raise ValueError(f"{name} has no gradient here")
            mask[name] = _dense(t)
    return mask


_MASKS = ("slopes", "docs", "prefix", "lengths", "first")


def _saved(args):
    """The masks among the arguments, which the graph saves (one that changes before the backward
    pass then raises there), and the others."""
    return [args.get(n) for n in _MASKS], {n: v for n, v in args.items() if n not in _MASKS}


class _Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, args, keep):
        q, k, v = _heads(q), _heads(k), _heads(v)
        lse = None
        if keep:
            lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32,
                              device=q.device)
        out = rnc.dprc_attention(q, k, v, lse=lse, **args)
        masks, ctx.args = _saved(args)
        ctx.save_for_backward(q, k, v, out, lse, *masks)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        q, k, v, out, lse, *masks = ctx.saved_tensors
        d = [torch.empty(t.shape, dtype=t.dtype, device=t.device) if need else None
             for t, need in zip((q, k, v), ctx.needs_input_grad)]
        if any(t is not None for t in d):
            rnc.dprc_attention_grad(_heads(grad), q, k, v, out, lse, dQ=d[0], dK=d[1], dV=d[2],
                                    **dict(zip(_MASKS, masks)), **ctx.args)
        return *d, None, None


def attend(q, k, v, scale=None, causal=True, cap=0.0, slopes=None, docs=None, prefix=None,
           lengths=None, first=None):
    """dprc_attention of q [B][Tq][H][D] over k, v [B][Tk][Hkv][D], with its gradient."""
    args = _plain(dict(scale=scale, causal=causal, cap=cap, slopes=slopes, docs=docs,
                       prefix=prefix, lengths=lengths, first=first))
    return _Attend.apply(q, k, v, args, torch.is_grad_enabled())


class _SelfAttend(torch.autograd.Function):
    """Attention from the rows [q | k | v] of one product, with rotary positions: the
    gradient is written in place into rows of the same form."""

    @staticmethod
    def forward(ctx, rows, positions, freqs, heads, turn, args, keep):
        H, Hkv, D = heads
        B, T, _ = rows.shape
        rows = _dense(rows).view(B, T, H + 2 * Hkv, D)
        qk, v = rows[:, :, :H + Hkv], rows[:, :, H + Hkv:]
        if freqs is not None:
            qk = rnc.dprc_rotary(qk, positions, freqs, **turn)
        q, k = qk[:, :, :H], qk[:, :, H:]
        lse = torch.empty((B, H, T), dtype=torch.float32, device=rows.device) if keep else None
        out = rnc.dprc_attention(q, k, v, lse=lse, **args)
        masks, ctx.args = _saved(args)
        ctx.save_for_backward(q, k, v, out, lse, positions, freqs, *masks)
        ctx.heads, ctx.turn = heads, turn
        return out.view(B, T, H * D)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        q, k, v, out, lse, positions, freqs, *masks = ctx.saved_tensors
        H, Hkv, D = ctx.heads
        B, T = q.shape[:2]
        d = torch.empty((B, T, H + 2 * Hkv, D), dtype=q.dtype, device=q.device)
        dqk = d[:, :, :H + Hkv]
        rnc.dprc_attention_grad(_dense(grad).view(B, T, H, D), q, k, v, out, lse, dQ=d[:, :, :H],
                                dK=dqk[:, :, H:], dV=d[:, :, H + Hkv:],
                                **dict(zip(_MASKS, masks)), **ctx.args)
        if freqs is not None:
            rnc.dprc_rotary(dqk, positions, freqs, inverse=True, out=dqk, **ctx.turn)
        return d.view(B, T, (H + 2 * Hkv) * D), None, None, None, None, None, None


class Attention(torch.nn.Module):
    """Self-attention of rows [q | k | v] (heads, key heads, key heads, of `width` each),
    as one product gives them, to [B][T][heads width].  With `freqs` (radians of the
    pairs, rotary_freqs), queries and keys are turned by their positions [B][T] (or
    [B][T][axes] with the pairs of each axis in sections; None: 0, 1, 2, ..)."""

    def __init__(self, heads, kv_heads, width, causal=True, cap=0.0, slopes=None, scale=None,
                 freqs=None, sections=None, interleaved=False):
        super().__init__()
        if heads % kv_heads != 0:
            raise ValueError(f"{heads} heads are no multiple of {kv_heads} heads of keys")
        self.heads, self.kv_heads, self.width = int(heads), int(kv_heads), int(width)
        self.causal, self.cap, self.scale = bool(causal), float(cap), scale
        self.sections, self.interleaved = sections, bool(interleaved)
        # (kept in their own types when the module's parameters change theirs)
        self.freqs = None if freqs is None else freqs.detach().double()
        self.slopes = None if slopes is None else slopes.detach().float()

    def _apply(self, fn, recurse=True):
        super()._apply(fn, recurse)
        for name, dtype in (("freqs", torch.float64), ("slopes", torch.float32)):
            t = getattr(self, name)
            if t is not None:
                setattr(self, name, t.to(fn(torch.empty(0, device=t.device)).device, dtype))
        return self

    def positions(self, B, T, device):
        return torch.arange(T, device=device).expand(B, T).contiguous()

    def forward(self, rows, positions=None, docs=None, prefix=None, lengths=None):
        B, T, n = rows.shape
        if n != (self.heads + 2 * self.kv_heads) * self.width:
            raise ValueError(f"rows of {n} are not [q | k | v] of {self.heads}, {self.kv_heads} and "
                             f"{self.kv_heads} heads of {self.width}")
        if self.freqs is None:
            positions = None
        elif positions is None:
            positions = self.positions(B, T, rows.device)
        args = _plain(dict(scale=self.scale, causal=self.causal, cap=self.cap, slopes=self.slopes,
                           docs=docs, prefix=prefix, lengths=lengths))
        turn = dict(sections=self.sections, interleaved=self.interleaved)
        return _SelfAttend.apply(rows, _dense(positions), self.freqs,
                                 (self.heads, self.kv_heads, self.width), turn, args,
                                 torch.is_grad_enabled())
