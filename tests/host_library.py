"""The library's calls that layers.py and step.py make, on host tensors from the
float64 oracle, so that the modules and the clipping step can be tested without
a GPU.  `install` puts them in the place of the binding's."""

import numpy as np
import torch

import randomized_norm_clipping_gb300.binding as binding
from oracle import operators as ops


def _np(t):
    return None if t is None else t.detach().double().numpy()


def _to(x, like):
    return torch.from_numpy(np.ascontiguousarray(x)).to(like.dtype)


class Plan:
    def __init__(self, tokens, V):
        self.tokens, self.V = tokens.clone(), V
        self.buf = torch.zeros(1, dtype=torch.uint8)


def embed_plan(tokens, V, buf=None, stream=None):
    return Plan(tokens, V)


def embed_lookup(W, tokens, scale=1.0, out=None, stream=None):
    return _to(ops.embed_lookup(_np(W), tokens.numpy(), scale), W)


def embed_norm(G, plan, n, scale=1.0, accumulate=False, ws=None, stream=None):
    v = _to(ops.embed_norm(_np(G), plan.tokens.numpy(), plan.V, scale), n)
    n.copy_(n + v if accumulate else v)
    return n


def embed_grad(G, plan, dW, c=None, scale=1.0, accumulate=False, ws=None, stream=None):
    v = _to(ops.embed_grad(_np(G), plan.tokens.numpy(), plan.V, _np(c), scale), dW)
    dW.copy_(dW + v if accumulate else v)
    return dW


def dropout(x, p, seed, step, residual=None, first_element=0, out=None, stream=None):
    return _to(ops.dropout(_np(x), p, seed, step, _np(residual), first_element), x)


def linear(X, W, bias=None, act="none", p=0.0, seed=0, step=0, residual=None, Z=None, out=None,
           ws=None, stream=None):
    rows = X.reshape(-1, X.shape[-1])
    shape = (*X.shape[:-1], W.shape[0])
    res = None if residual is None else _np(residual).reshape(-1, W.shape[0])
    y, z = ops.linear(_np(rows), _np(W), _np(bias), act, p, seed, step, res)
    if Z is not None:
        Z.copy_(_to(z.reshape(shape), X))
    return _to(y.reshape(shape), X)


def linear_grad(dY, X, W, Z=None, act="none", p=0.0, seed=0, step=0, dX=None, dW=None, db=None,
                dZ=None, ws=None, stream=None):
    N, K = W.shape
    x = np.zeros((dY.numel() // N, K)) if X is None else _np(X).reshape(-1, K)
    z = None if Z is None else _np(Z).reshape(-1, N)
    got = ops.linear_grad(_np(dY).reshape(-1, N), x, _np(W), z, act, p, seed, step)
    for t, v in zip((dX, dW, db, dZ), got):
        if t is not None:
            t.copy_(_to(v, t).reshape(t.shape))


def norm_hutch(A, G, P, n, accumulate=False, ws=None, stream=None):
    M = torch.einsum("btd,btk->bdk", A.double(), G.double() @ P.double())
    v = (M ** 2).sum((1, 2)).to(n.dtype)
    n.copy_(n + v if accumulate else v)


def clip_factors(n, C, c, stream=None):
    c.copy_(torch.clamp(C / torch.sqrt(n), max=1.0))


def norm_hutch_clip(A, G, P, n, C, c, accumulate=False, ws=None, stream=None):
    norm_hutch(A, G, P, n, accumulate)
    clip_factors(n, C, c)


def norm_hutch_layers(As, Gs, Ps, n, accumulate=False, ws=None, C=None, c=None, stream=None):
    for j, (A, G, P) in enumerate(zip(As, Gs, Ps)):
        norm_hutch(A, G, P, n, accumulate or j > 0)
    clip_factors(n, C, c)


def install(monkeypatch):
    for name, f in dict(embed_plan=embed_plan, embed_lookup=embed_lookup, embed_norm=embed_norm,
                        embed_grad=embed_grad, dropout=dropout, linear=linear,
                        linear_grad=linear_grad, norm_hutch=norm_hutch,
                        norm_hutch_clip=norm_hutch_clip, norm_hutch_layers=norm_hutch_layers,
                        clip_factors=clip_factors).items():
        monkeypatch.setattr(binding, "dprc_" + name, f)
