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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mask", ["documents", "lengths"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 0.5])
@pytest.mark.parametrize("cap,slope", [(0.0, 0.0), (4.0, 0.0), (0.0, 0.1)])
@pytest.mark.parametrize("Tq,T,H,Hkv,D", [(150, 150, 6, 2, 64), (2, 700, 8, 2, 64), (40, 200, 4, 1, 128)])
def test_attention_of_any_scale(dtype, mask, scale, cap, slope, Tq, T, H, Hkv, D):
    """A scale below zero turns the order of the products; one of zero takes all alike."""
    kw = dict(_mask(mask, 2, Tq, T), scale=scale, cap=cap)
    if slope:
        kw["slopes"] = torch.full((H,), slope)
    _check(dtype, *_heads(dtype, 2, Tq, T, H, Hkv, D), kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Tq", [200, 3])
def test_attention_of_expanded_keys(dtype, Tq):
    """One prompt's keys and values for all samples, and one head's for all heads."""
    Q, K, V, dO = _heads(dtype, 3, Tq, 200, 4, 2, 64)
    for axis in (0, 2):
        k, v = (t.narrow(axis, 0, 1) for t in (K, V))
        dev = [Q.to(DEV)] + [t.to(DEV).expand(K.shape) for t in (k, v)]
        assert dev[1].stride(axis) == 0
        _check(dtype, Q, k.expand(K.shape), v.expand(V.shape), dO, {}, dev=dev)


@pytest.mark.parametrize("Tq,T,H,Hkv,D", [(640, 640, 8, 2, 64), (600, 777, 4, 4, 64), (500, 500, 4, 1, 128)])
def test_attention_to_the_roundings_of_its_parts(Tq, T, H, Hkv, D):
    """bf16, all keys, independent inputs: the errors of the many terms of a sum do not add up
    but in the mean square.  A rounding to bf16 is off by 2^-8 at most, spread evenly over that,
    2^-8 / sqrt(3) in the mean square; a result has up to three in a row (the weights P or dS,
    delta's output, itself): 2^-8 together, in the 2-norm of 10^5 values.  A term that is wrong
    by one part in a hundred of the result shows."""
    Q, K, V, dO = _heads(BF16, 2, Tq, T, H, Hkv, D)
    ref = block.attention(_np(Q), _np(K), _np(V), causal=False, dO=_np(dO))
    q, k, v, do = (t.to(DEV) for t in (Q, K, V, dO))
    lse = torch.empty(2, H, Tq, device=DEV)
    out = rnc.dprc_attention(q, k, v, causal=False, lse=lse)
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    rnc.dprc_attention_grad(do, q, k, v, out, lse, causal=False, dQ=dq, dK=dk, dV=dv)
    for name, a, b in (("out", out, ref[0]), ("dQ", dq, ref[2]), ("dK", dk, ref[3]), ("dV", dv, ref[4])):
        _near(a, b, 2.0 ** -8, name)


@pytest.mark.parametrize("mask", ["causal", "all", "full documents"])
@pytest.mark.parametrize("Tq,T,H,Hkv,D", [(37, 37, 128, 1, 64), (90, 90, 100, 1, 128), (50, 50, 96, 2, 72),
                                          (1, 500, 128, 1, 64), (2, 300, 32, 2, 64), (9, 300, 3, 1, 40)])
def test_attention_of_wide_groups(mask, Tq, T, H, Hkv, D):
    """Groups of heads that fill a tile of rows by themselves, or leave part of it; all masks at once
    over few tokens."""
    _check(BF16, *_heads(BF16, 2, Tq, T, H, Hkv, D), _mask(mask, 2, Tq, T))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [7, 64, 1027, 2048, 5003, 16383])
def test_normalisation_in_place(dtype, d):
    x = _randn((3, 41, d), dtype, d).to(DEV)
    w = _randn((d,), dtype, d + 1).to(DEV)
    y = rnc.dprc_layernorm(x, w)
    assert rnc.dprc_layernorm(x, w, out=x) is x and torch.equal(x, y)
