"""Oracle for the operators around the norm path: embedding, dropout, linear map.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Float64 numpy, from the
definitions in include/dprc.h, position by position:

  lookup    out[j] = s W[tok_j], a zero row where tok_j is no token
  norm      n_i = s^2 sum_v || sum_{t: tok_it = v} G_it ||^2
  gradient  dW[v] = s sum_i c_i sum_{t: tok_it = v} G_it
  dropout   element e is dropped when half (e & 7) of Philox block e >> 3 is
            below floor(65536 p + 1/2); the rest times 65536 / (65536 - that)
  linear    z = X W^T + b, y = r + drop(act(z)), and its gradient
"""

from __future__ import annotations

import math

import numpy as np

from .philox import philox_words


def embed_lookup(W, tokens, scale=1.0):
    W = np.asarray(W, dtype=np.float64)
    tok = np.asarray(tokens)
    out = np.zeros((*tok.shape, W.shape[1]))
    ok = (tok >= 0) & (tok < W.shape[0])
    out[ok] = scale * W[tok[ok]]
    return out


def embed_rows(G_i, tok_i, V):
    """The per-sample gradient rows {v: sum_t G_t} of one sample (before the scale)."""
    rows = {}
    for t, v in enumerate(tok_i):
        v = int(v)
        if 0 <= v < V:
            rows[v] = rows.get(v, 0.0) + np.asarray(G_i[t], dtype=np.float64)
    return rows


def embed_norm(G, tokens, V, scale=1.0):
    return np.array([scale ** 2 * sum(float(np.dot(r, r)) for r in embed_rows(g, t, V).values())
                     for g, t in zip(G, tokens)])


def embed_grad(G, tokens, V, c=None, scale=1.0):
    dW = np.zeros((V, G.shape[2]))
    for i in range(G.shape[0]):
        f = scale * (1.0 if c is None else float(c[i]))
        for v, r in embed_rows(G[i], tokens[i], V).items():
            dW[v] += f * r
    return dW


def dropout_threshold(p):
    return min(65536, int(math.floor(65536.0 * p + 0.5)))


def dropout_factor(n, p, seed, step, first_element=0):
    """0 for a dropped element, 65536 / (65536 - t) for a kept one."""
    if n == 0:
        return np.zeros(0)
    thr = dropout_threshold(p)
    e0 = int(first_element)
    b0, b1 = e0 >> 3, (e0 + n - 1) >> 3
    w = philox_words(seed, step, b0, b1 - b0 + 1).astype(np.uint64)
    halves = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], axis=2).reshape(-1)
    h = halves[e0 - 8 * b0: e0 - 8 * b0 + n]
    keep = 0.0 if thr >= 65536 else 65536.0 / (65536 - thr)
    return np.where(h < thr, 0.0, keep)


def dropout(x, p, seed, step, residual=None, first_element=0):
    x = np.asarray(x, dtype=np.float64)
    f = dropout_factor(x.size, p, seed, step, first_element).reshape(x.shape)
    y = np.where(f == 0.0, 0.0, x * f)
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        t = np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
        return (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * math.sqrt(2.0 / math.pi)
                * (1.0 + 3.0 * 0.044715 * z * z))
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def linear(X, W, bias=None, name="none", p=0.0, seed=0, step=0, residual=None):
    """(y, z)."""
    z = np.asarray(X, np.float64) @ np.asarray(W, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = act(z, name)
    if dropout_threshold(p) > 0:
        y = dropout(y, p, seed, step)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y, z


def linear_grad(dY, X, W, Z=None, name="none", p=0.0, seed=0, step=0):
    """(dX, dW, db, dZ)."""
    dz = np.asarray(dY, np.float64)
    if dropout_threshold(p) > 0:
        dz = dropout(dz, p, seed, step)
    if name != "none":
        dz = dz * act_slope(np.asarray(Z, np.float64), name)
    return dz @ np.asarray(W, np.float64), dz.T @ np.asarray(X, np.float64), dz.sum(0), dz
