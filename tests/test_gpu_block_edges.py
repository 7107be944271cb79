"""Normalisation and attention at the borders of their ranges, against the float64 oracle, with the
tolerances of test_gpu_block_operators.py.
"""

import numpy as np
import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from oracle import block
from randomized_norm_clipping_gb300 import layers as lay
from test_gpu_block_operators import ATT, ATT_GRAD, CANCEL, NORM, _mask, _near, _np, _randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    torch.cuda.synchronize()
    assert rnc.dprc_device_error(reset=True) == 0


def _check(dtype, Q, K, V, dO, kw, off=0.0, grad=True, dev=None):
    """Forward and gradient of host tensors (dev: the same on the device, if strided) against the
    oracle.  off: what the scores' size adds to the relative error of a weight, and
    so to the lse, to delta (of its terms) and, twice, to a gradient."""
    on = {n: x.to(DEV) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    host = {n: _np(x) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    q, k, v = (t.to(DEV) for t in (Q, K, V)) if dev is None else dev
    do = dO.to(DEV)
    lse = torch.empty(Q.shape[0], Q.shape[2], Q.shape[1], device=DEV)
    out = rnc.dprc_attention(q, k, v, lse=lse, **on)
    ref = block.attention(_np(Q), _np(K), _np(V), dO=_np(dO), **host)
    _near(out, ref[0], ATT[dtype] + off, "out")
    got, want = _np(lse), ref[1]
    none = np.isinf(want)
    assert (got[none] == -np.inf).all()
    assert np.abs(got[~none] - want[~none]).max(initial=0.0) <= \
        1e-5 * (1 + np.abs(want[~none]).max(initial=0.0)) + off
    if not grad:
        return
    dq, dk, dv = (torch.full(t.shape, 7.0, dtype=dtype, device=DEV) for t in (Q, K, V))
    rnc.dprc_attention_grad(do, q, k, v, out, lse, dQ=dq, dK=dk, dV=dv, **on)
    for name, a, b, terms in (("dQ", dq, ref[2], ref[5]), ("dK", dk, ref[3], ref[6]),
                              ("dV", dv, ref[4], 0.0)):
        _near(a, b, ATT_GRAD[dtype] + 2 * off, name, (CANCEL[dtype] + off) * np.linalg.norm(terms))


def _heads(dtype, B, Tq, Tk, H, Hkv, D, seed=0):
    return (_randn((B, Tq, H, D), dtype, seed + 1), _randn((B, Tk, Hkv, D), dtype, seed + 2),
            _randn((B, Tk, Hkv, D), dtype, seed + 3), _randn((B, Tq, H, D), dtype, seed + 4))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mask", ["causal", "full", "documents"])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("T,H,Hkv,D", [(300, 4, 2, 64), (130, 6, 2, 128), (200, 1, 1, 64)])
def test_attention_of_rising_biases(dtype, mask, cap, T, H, Hkv, D):
    """Slopes below zero: scores rise with the distance, also beside a last tile of rows that is not
    full.  A score of size s is rounded some eight times (the bias, the lse and its units)."""
    slopes = -0.6 * torch.ones(H)
    slopes[H // 2:] = -1.25
    kw = dict(_mask(mask, 1, T, T), slopes=slopes, cap=cap)
    _check(dtype, *_heads(dtype, 1, T, T, H, Hkv, D), kw, off=8 * 2.0 ** -24 * 1.25 * T)


@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128), (BF16, 33)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_of_documents_behind_the_length(dtype, D, causal, bad):
    """A document that lies behind its sample's length as a whole: its queries see nothing, although
    their position does, and may hold anything, as may their output's gradient."""
    B, T, H, Hkv = 2, 300, 4, 2
    lengths = torch.tensor([130, 290], dtype=torch.int32)
    docs = torch.zeros(B, T, dtype=torch.int32)
    docs[0, 150:], docs[1, 295:] = 1, 3
    Q, K, V, dO = _heads(dtype, B, T, T, H, Hkv, D)
    gone = torch.arange(T)[None] >= lengths[:, None]
    K[gone], V[gone] = bad, bad
    Q[docs > 0], dO[docs > 0] = bad, bad
    _check(dtype, Q, K, V, dO, dict(causal=causal, docs=docs, lengths=lengths))


def _terms(dY, X, W, mu, r):
    """The sizes of the terms of which dX is the sum."""
    g = np.abs(_np(dY) * _np(W))
    xh = np.abs((_np(X) - mu[..., None]) * r[..., None])
    return (g + g.mean(-1, keepdims=True) + xh * (g * xh).mean(-1, keepdims=True)) * r[..., None]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 321, 2048, 4104, 5003])
@pytest.mark.parametrize("size,eps", [(1e17, 1e-5), (1e15, 1e-5), (1e13, 1e-5), (1e-2, 1e-5), (1.0, 0.5),
                                      (1e-13, 0.0)])
def test_normalisation_of_any_size(size, eps, d, dtype):
    """Rows whose deviation's square, or its reciprocal's, is far from 1; sums of squares stay below
    2^127 (5003 1e34)."""
    for center in (True, False):
        X, dY = _randn((2, 9, d), F32, d).mul(size).to(dtype), _randn((2, 9, d), dtype, d + 1)
        W = (1 + _randn((d,), F32, d + 2, 0.2)).to(dtype)
        y, mu, r = block.layernorm(_np(X), _np(W), None, eps, center)
        x, w, stats = X.to(DEV), W.to(DEV), torch.empty(2, 9, 2, device=DEV)
        _near(rnc.dprc_layernorm(x, w, eps=eps, center=center, stats=stats), y, NORM[dtype], "y")
        _near(stats[..., 1], r, 64 * 2.0 ** -24, "r")
        dX, Ws, bs = block.layernorm_grad(_np(dY), _np(X), _np(W), eps, center)
        dx, dw, db, n = (torch.empty(s, device=DEV, dtype=t) for s, t in
                         ((X.shape, dtype), ((d,), dtype), ((d,), dtype), ((2,), F32)))
        rnc.dprc_layernorm_grad(dY.to(DEV), x, stats, w, center=center, dX=dx, dW=dw, db=db, n=n)
        # (relative to 1 / size, so that no square of the test's own norms leaves the range)
        terms = np.linalg.norm(_terms(dY, X, W, mu, r) * size)
        _near(_np(dx) * size, dX * size, NORM[dtype], "dX", 8 * 2.0 ** -24 * terms)
        _near(dw, Ws.sum(0), NORM[dtype], "dW")
        _near(db, bs.sum(0), NORM[dtype], "db")
        _near(n, (Ws ** 2).sum(1), 64 * 2.0 ** -24, "n")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_normalisation_of_rows_without_an_axis_of_samples(dtype):
    """More rows in the first axis than there may be samples."""
    N, d = 70001, 24
    X, u = _randn((N, d), dtype, 1), _randn((N, d), dtype, 2)
    m = lay.LayerNorm(d, device=DEV, dtype=dtype)
    x = X.to(DEV).requires_grad_()
    (m(x) * u.to(DEV)).sum().backward()
    dX, Ws, bs = block.layernorm_grad(_np(u)[None], _np(X)[None])
    # (dX: a sum of three terms of the size of u, r being near 1)
    _near(x.grad, dX[0], NORM[dtype], "dX", 8 * 2.0 ** -24 * np.linalg.norm(_np(u)) * 3)
    _near(m.weight.grad, Ws[0], NORM[dtype], "dW")
    _near(m.bias.grad, bs[0], NORM[dtype], "db")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T", [(0, 0), (0, 5), (2, 0)])
def test_modules_on_batches_of_nothing(dtype, B, T):
    norm = lay.LayerNorm(48, device=DEV, dtype=dtype)
    att = lay.Attention(4, 2, 6, freqs=lay.rotary_freqs(3)).to(DEV)
    x = torch.zeros(B, T, 48, device=DEV, dtype=dtype, requires_grad=True)
    y = att(norm(x))
    assert y.shape == (B, T, 24)
    y.sum().backward()
    assert x.grad.shape == x.shape
    for p in (norm.weight, norm.bias):
        assert p.grad.shape == p.shape and (p.grad == 0).all()
    plain = lay.LayerNorm(48, weight=False, bias=False)
    (g,) = torch.autograd.grad(plain(x).sum(), x)
    assert g.shape == x.shape
    q, kv = x.detach().view(B, T, 8, 6).requires_grad_(), torch.zeros(B, 9, 2, 6, device=DEV, dtype=dtype)
    lay.attend(q, kv, kv).sum().backward()
    assert q.grad.shape == q.shape
    kv.requires_grad_()
    for t in torch.autograd.grad(lay.attend(q, kv, kv).sum(), (q, kv)):
        assert (t == 0).all()
