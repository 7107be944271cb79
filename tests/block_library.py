"""The library's calls of a transformer block (normalisation, rotary positions, attention)
on host tensors from the float64 oracle, beside those of host_library."""

import numpy as np
import torch

import host_library
import randomized_norm_clipping_gb300.binding as binding
from oracle import block


def _np(t):
    return t.detach().double().numpy() if isinstance(t, torch.Tensor) else t


def _put(out, value, like):
    t = torch.from_numpy(np.ascontiguousarray(value)).to(like.dtype)
    if out is None:
        return t
    out.copy_(t)
    return out


def layernorm(X, weight=None, bias=None, eps=1e-5, center=True, out=None, stats=None, stream=None):
    y, mu, r = block.layernorm(_np(X), _np(weight), _np(bias), eps, center)
    if stats is not None:
        _put(stats, np.stack((mu, r), -1), stats)
    return _put(out, y, X)


def layernorm_grad(dY, X, stats, weight=None, center=True, dX=None, dW=None, db=None, n=None,
                   norm_of_bias=False, accumulate=False, c=None, ws=None, stream=None):
    d = X.shape[-1]
    B = X.shape[0] if X.dim() > 1 else 1
    st = _np(stats).reshape(B, -1, 2)
    x, dy = _np(X).reshape(B, -1, d), _np(dY).reshape(B, -1, d)
    xh = (x - st[..., :1]) * st[..., 1:]
    g = dy if weight is None else dy * _np(weight)
    dx = g - xh * (g * xh).mean(-1, keepdims=True) - (g.mean(-1, keepdims=True) if center else 0.0)
    W, b = (dy * xh).sum(1), dy.sum(1)
    f = np.ones((B, 1)) if c is None else _np(c)[:, None]
    if dX is not None:
        _put(dX, (dx * st[..., 1:]).reshape(dX.shape), dX)
    if dW is not None:
        _put(dW, (f * W).sum(0), dW)
    if db is not None:
        _put(db, (f * b).sum(0), db)
    if n is not None:
        v = (W ** 2).sum(1) + ((b ** 2).sum(1) if norm_of_bias else 0.0)
        _put(n, _np(n) + v if accumulate else v, n)


def rotary(X, positions, freqs, sections=None, interleaved=False, inverse=False, out=None,
           stream=None):
    return _put(out, block.rotary(_np(X), positions.numpy(), _np(freqs), sections, interleaved,
                                  inverse), X)


def attention(Q, K, V, scale=None, causal=True, cap=0.0, slopes=None, docs=None, prefix=None,
              lengths=None, first=None, out=None, lse=None, ws=None, stream=None):
    o, l = block.attention(_np(Q), _np(K), _np(V), scale, causal, cap, _np(slopes), _np(docs),
                           _np(prefix), _np(lengths), _np(first))
    if lse is not None:
        _put(lse, l, lse)
    return _put(out, o, Q)


def attention_grad(dO, Q, K, V, O, lse, scale=None, causal=True, cap=0.0, slopes=None, docs=None,
                   prefix=None, lengths=None, first=None, dQ=None, dK=None, dV=None, ws=None,
                   stream=None):
    got = block.attention(_np(Q), _np(K), _np(V), scale, causal, cap, _np(slopes), _np(docs),
                          _np(prefix), _np(lengths), _np(first), dO=_np(dO))
    for t, v in zip((dQ, dK, dV), got[2:5]):
        if t is not None:
            _put(t, v, t)


def install(monkeypatch):
    host_library.install(monkeypatch)
    for name, f in dict(layernorm=layernorm, layernorm_grad=layernorm_grad, rotary=rotary,
                        attention=attention, attention_grad=attention_grad).items():
        monkeypatch.setattr(binding, "dprc_" + name, f)
