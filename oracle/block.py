"""Oracle for the operators of a transformer block: normalisation, rotary positions,
attention.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Float64 numpy, from the
definitions in include/dprc.h:

  layernorm  xh = (x - mu) r, y = w xh + b; per sample W_i = sum_t dy xh, b_i = sum_t dy
  rotary     the pair (a, b) as the complex number a + i b, times exp(i pos freq)
  attention  s = cap tanh(q k scale / cap) - slope |i - j|, softmax over the keys that a
             query sees, and its gradient
"""

from __future__ import annotations

import numpy as np


def layernorm(X, w=None, b=None, eps=1e-5, center=True):
    """(y, mu, r)."""
    X = np.asarray(X, np.float64)
    mu = X.mean(-1) if center else np.zeros(X.shape[:-1])
    r = 1.0 / np.sqrt(((X - mu[..., None]) ** 2).mean(-1) + eps)
    y = (X - mu[..., None]) * r[..., None]
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mu, r


def layernorm_grad(dY, X, w=None, eps=1e-5, center=True):
    """(dX, W [B][d], b [B][d]) of X [B][T][d]; the sums by sample."""
    dY, X = np.asarray(dY, np.float64), np.asarray(X, np.float64)
    xh, _, r = layernorm(X, None, None, eps, center)
    g = dY if w is None else dY * w
    dX = g - xh * (g * xh).mean(-1, keepdims=True)
    if center:
        dX = dX - g.mean(-1, keepdims=True)
    return dX * r[..., None], (dY * xh).sum(1), dY.sum(1)


def rotary(X, positions, freqs, sections=None, interleaved=False, inverse=False):
    """X [B][T][H][D], positions [B][T][axes]."""
    X = np.array(X, np.float64)
    positions = np.asarray(positions)
    if positions.ndim == 2:
        positions = positions[..., None]
    P = len(freqs)
    sections = [P] if sections is None else sections
    first = 0
    for a, n in enumerate(sections):
        p = np.arange(first, first + n)
        re, im = (2 * p, 2 * p + 1) if interleaved else (p, P + p)
        angle = positions[..., a, None].astype(np.float64) * np.asarray(freqs)[p]
        z = (X[..., re] + 1j * X[..., im]) * np.exp(1j * (-angle if inverse else angle))[:, :, None]
        X[..., re], X[..., im] = z.real, z.imag
        first += n
    return X


def sees(b, Tq, Tk, causal=True, docs=None, prefix=None, lengths=None, first=None):
    """Which keys the queries of sample b see, and the queries' positions."""
    at = (Tk - Tq if first is None else int(first[b])) + np.arange(Tq)
    j = np.arange(Tk)
    s = np.ones((Tq, Tk), bool)
    if causal:
        s = j[None] <= at[:, None]
        if prefix is not None:
            s = s | (j < int(prefix[b]))[None]
    if lengths is not None:
        s = s & (j < int(lengths[b]))[None]
    if docs is not None:
        d = np.asarray(docs[b])
        inside = (at >= 0) & (at < Tk)
        dq = np.where(inside, d[np.clip(at, 0, max(Tk - 1, 0))], -1) if Tk else np.full(Tq, -1)
        s = s & (dq[:, None] == d[None]) & (dq[:, None] >= 0)
    return s, at


def attention(Q, K, V, scale=None, causal=True, cap=0.0, slopes=None, docs=None, prefix=None,
              lengths=None, first=None, dO=None):
    """(out, lse), or with dO (out, lse, dQ, dK, dV, and the sums of the sizes of the terms
    of which dQ and dK are differences: p (|dp| + |delta|) |scale k|)."""
    Q, K, V = (np.asarray(x, np.float64) for x in (Q, K, V))
    B, Tq, H, D = Q.shape
    Tk, Hkv = K.shape[1], K.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros(Q.shape), np.full((B, H, Tq), -np.inf)
    dQ, dK, dV = np.zeros(Q.shape), np.zeros(K.shape), np.zeros(V.shape)
    tQ, tK = np.zeros(Q.shape), np.zeros(K.shape)
    for b in range(B):
        see, at = sees(b, Tq, Tk, causal, docs, prefix, lengths, first)
        used = see.any(0)  # other keys may hold anything
        for h in range(H):
            q = np.where(see.any(1)[:, None], Q[b, :, h], 0.0)
            k = np.where(used[:, None], K[b, :, h * Hkv // H], 0.0)
            v = np.where(used[:, None], V[b, :, h * Hkv // H], 0.0)
            z = q @ k.T * scale
            t = np.zeros_like(z)
            if cap > 0:
                t = np.tanh(z / cap)
                z = cap * t
            if slopes is not None:
                z = z - float(slopes[h]) * np.abs(at[:, None] - np.arange(Tk)[None])
            z = np.where(see, z, -np.inf)
            m = z.max(1, initial=-np.inf)
            e = np.exp(z - np.where(np.isinf(m), 0.0, m)[:, None])
            l = e.sum(1)
            p = e / np.where(l == 0, 1.0, l)[:, None]
            out[b, :, h] = p @ v
            with np.errstate(divide="ignore"):
                lse[b, h] = m + np.log(l)
            if dO is None:
                continue
            do = np.where(see.any(1)[:, None], np.asarray(dO[b, :, h], np.float64), 0.0)
            dp = do @ v.T
            size = p * (np.abs(dp) + np.abs(do * out[b, :, h]).sum(1)[:, None]) * (1 - t * t) * abs(scale)
            tQ[b, :, h] = size @ np.abs(k)
            tK[b, :, h * Hkv // H] += size.T @ np.abs(q)
            ds = p * (dp - (do * out[b, :, h]).sum(1)[:, None]) * (1 - t * t) * scale
            dQ[b, :, h] = ds @ k
            dK[b, :, h * Hkv // H] += ds.T @ q
            dV[b, :, h * Hkv // H] += p.T @ do
    return (out, lse) if dO is None else (out, lse, dQ, dK, dV, tQ, tK)
