"""The operators around the norm path, without a GPU: the float64 oracle of
oracle/operators.py pinned to brute force, differences and automatic
differentiation, mistakes planted in it that the pins must catch, and the C
entry points' refusals (no kernel runs)."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import operators as ops
from oracle.philox import philox4x32_10


def _rng(seed):
    return np.random.default_rng(seed)


# ---- embedding -------------------------------------------------------------
def _dense_grads(G, tok, V, scale):
    """Every sample's dense [V][d] gradient, through a one-hot product."""
    out = []
    for g, t in zip(G, tok):
        hot = np.zeros((len(t), V))
        for j, v in enumerate(t):
            if 0 <= v < V:
                hot[j, v] = 1.0
        out.append(scale * hot.T @ g)
    return np.stack(out)


@pytest.mark.parametrize("B,T,V,d", [(1, 1, 1, 1), (3, 7, 5, 4), (2, 40, 3, 6), (4, 9, 50, 2)])
def test_embedding_oracle_matches_dense_gradients(B, T, V, d):
    r = _rng(B * 100 + T)
    G = r.standard_normal((B, T, d))
    tok = r.integers(-1, V, (B, T))
    c = r.uniform(0.1, 1.0, B)
    dense = _dense_grads(G, tok, V, 1.7)
    assert np.allclose(ops.embed_norm(G, tok, V, 1.7), (dense ** 2).sum((1, 2)), rtol=1e-12)
    assert np.allclose(ops.embed_grad(G, tok, V, c, 1.7), np.tensordot(c, dense, 1), atol=1e-12)
    W = r.standard_normal((V, d))
    hot = np.zeros((B, T, V))
    for i in range(B):
        for t in range(T):
            if tok[i, t] >= 0:
                hot[i, t, tok[i, t]] = 1.0
    assert np.allclose(ops.embed_lookup(W, tok, 0.3), 0.3 * hot @ W, atol=1e-12)


def test_embedding_gradient_is_the_lookups_derivative():
    r = _rng(3)
    V, d, tok = 6, 3, np.array([[0, 2, 2, -1, 5]])
    W, G = r.standard_normal((V, d)), r.standard_normal((1, 5, d))
    dW = ops.embed_grad(G, tok, V, None, 2.5)
    h = 1e-6
    for v in range(V):
        for k in range(d):
            E = np.zeros_like(W)
            E[v, k] = h
            diff = ((ops.embed_lookup(W + E, tok, 2.5) - ops.embed_lookup(W - E, tok, 2.5)) * G)
            assert abs(diff.sum() / (2 * h) - dW[v, k]) < 1e-8


def test_bias_is_an_embedding_of_one_row():
    r = _rng(4)
    G = r.standard_normal((3, 11, 5))
    tok = np.zeros((3, 11), dtype=np.int64)
    assert np.allclose(ops.embed_norm(G, tok, 1), (G.sum(1) ** 2).sum(1), rtol=1e-12)


@pytest.mark.parametrize("mistake", ["square first", "no scale", "padding counted"])
def test_planted_embedding_mistakes_are_caught(mistake):
    r = _rng(5)
    G = r.standard_normal((2, 12, 4))
    tok = r.integers(-1, 4, (2, 12))
    ref = (_dense_grads(G, tok, 4, 1.5) ** 2).sum((1, 2))
    if mistake == "square first":  # sums of squares instead of squares of sums
        bad = np.array([1.5 ** 2 * (g[t >= 0] ** 2).sum() for g, t in zip(G, tok)])
    elif mistake == "no scale":
        bad = ops.embed_norm(G, tok, 4, 1.0)
    else:
        bad = ops.embed_norm(G, np.where(tok < 0, 0, tok), 4, 1.5)
    assert not np.allclose(bad, ref, rtol=1e-3)


# ---- dropout ---------------------------------------------------------------
def test_dropout_halves_follow_the_stream():
    seed, step, p = 0x1234567890ABCDEF, 7, 0.3
    f = ops.dropout_factor(64, p, seed, step, first_element=8 * 5 + 3)
    thr = math.floor(65536 * p + 0.5)
    for i in range(64):
        e = 8 * 5 + 3 + i
        w = [int(x) for x in philox4x32_10(e >> 3, 0, step, 0, seed & 0xFFFFFFFF, seed >> 32)]
        half = (w[(e & 7) >> 1] >> (16 * (e & 1))) & 0xFFFF
        assert f[i] == (0.0 if half < thr else 65536.0 / (65536 - thr))


def test_dropout_rate_and_mean():
    n, p = 1 << 20, 0.37
    f = ops.dropout_factor(n, p, 11, 2)
    q = ops.dropout_threshold(p) / 65536.0
    assert abs(q - p) <= 2.0 ** -17
    dropped = (f == 0).mean()
    assert abs(dropped - q) < 5 * math.sqrt(q * (1 - q) / n)  # five standard errors
    assert abs(f.mean() - 1.0) < 5 * math.sqrt(q / (1 - q) / n)
    # neighbouring elements (halves of a word, words, blocks) are uncorrelated
    z = (f == 0) - q
    for lag in (1, 2, 4, 8, 16):
        r = (z[lag:] * z[:-lag]).mean() / (q * (1 - q))
        assert abs(r) < 5 / math.sqrt(n)


@pytest.mark.parametrize("p", [0.0, 1.0, 1e-6])
def test_dropout_ends(p):
    f = ops.dropout_factor(1000, p, 1, 1)
    assert (f == (0.0 if p == 1.0 else 1.0)).all()


def test_dropout_piece_is_the_whole_tensors_piece():
    whole = ops.dropout_factor(1000, 0.4, 3, 4)
    for a, b in ((0, 1), (5, 21), (8, 16), (13, 1000)):
        assert (ops.dropout_factor(b - a, 0.4, 3, 4, first_element=a) == whole[a:b]).all()


# ---- linear map ------------------------------------------------------------
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_linear_gradient_matches_autograd_and_differences(name, p):
    r = _rng(9)
    M, K, N = 5, 4, 6
    X, W, b = r.standard_normal((M, K)), r.standard_normal((N, K)), r.standard_normal(N)
    res, dY = r.standard_normal((M, N)), r.standard_normal((M, N))
    y, z = ops.linear(X, W, b, name, p, 21, 3, res)
    dX, dW, db, dZ = ops.linear_grad(dY, X, W, z, name, p, 21, 3)
    # automatic differentiation of torch's own activations
    tX, tW, tb = (torch.tensor(v, requires_grad=True) for v in (X, W, b))
    tz = tX @ tW.t() + tb
    f = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name]
    factor = ops.dropout_factor(M * N, p, 21, 3).reshape(M, N) if p else np.ones((M, N))
    ty = f(tz) * torch.tensor(factor) + torch.tensor(res)
    assert np.allclose(ty.detach().numpy(), y, atol=1e-12)
    g = torch.autograd.grad((ty * torch.tensor(dY)).sum(), (tX, tW, tb))
    for ours, theirs in zip((dX, dW, db), g):
        assert np.allclose(ours, theirs.numpy(), atol=1e-11)
    # differences in one direction
    h, D = 1e-6, r.standard_normal((M, K))
    up = (ops.linear(X + h * D, W, b, name, p, 21, 3, res)[0] * dY).sum()
    dn = (ops.linear(X - h * D, W, b, name, p, 21, 3, res)[0] * dY).sum()
    assert abs((up - dn) / (2 * h) - (dX * D).sum()) < 1e-6


@pytest.mark.parametrize("mistake", ["mask after residual", "slope at y", "no rescale"])
def test_planted_linear_mistakes_are_caught(mistake):
    r = _rng(10)
    X, W = r.standard_normal((6, 4)), r.standard_normal((8, 4))
    res = r.standard_normal((6, 8))
    y, z = ops.linear(X, W, None, "silu", 0.5, 1, 2, res)
    if mistake == "mask after residual":
        bad = ops.dropout(ops.act(z, "silu") + res, 0.5, 1, 2)
    elif mistake == "no rescale":
        bad = np.where(ops.dropout_factor(48, 0.5, 1, 2).reshape(6, 8) > 0,
                       ops.act(z, "silu"), 0.0) + res
    else:
        dY = r.standard_normal((6, 8))
        good = ops.linear_grad(dY, X, W, z, "silu")[3]
        bad = dY * ops.act_slope(ops.act(z, "silu"), "silu")
        assert not np.allclose(bad, good, rtol=1e-3)
        return
    assert not np.allclose(bad, y, rtol=1e-3)


# ---- refusals of the C entry points ----------------------------------------
@pytest.fixture(scope="module")
def lib():
    import os

    from randomized_norm_clipping_gb300 import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


P = 0x10000  # aligned, never dereferenced: every call below fails its checks first
BIG = 1 << 40
INF = float("inf")
NAN = float("nan")


def test_embed_refusals(lib):
    f = lib.dprc_embed_lookup
    assert f(None, 1, P, 8, 4, 10, 8, 1.0, P, None) == 1
    assert f(P, 1, None, 8, 4, 10, 8, 1.0, P, None) == 1
    assert f(P, 5, P, 8, 4, 10, 8, 1.0, P, None) == 3
    assert f(P, 1, P, 2, 4, 10, 8, 1.0, P, None) == 3  # token size
    assert f(P, 1, P, 8, -1, 10, 8, 1.0, P, None) == 2
    assert f(P, 1, P, 8, 4, 0, 8, 1.0, P, None) == 2
    assert f(P, 1, P, 8, 4, 10, 0, 1.0, P, None) == 2
    assert f(P, 1, P, 8, 4, 10, 8, INF, P, None) == 2
    assert f(P, 1, P, 8, 4, 10, 8, NAN, P, None) == 2
    assert f(P, 1, P, 8, 4, (1 << 30) + 1, 8, 1.0, P, None) == 2
    assert f(P + 2, 1, P, 8, 4, 10, 8, 1.0, P, None) == 4
    assert f(P, 1, P + 8, 8, 4, 10, 8, 1.0, P, None) == 4
    assert f(P, 1, None, 8, 0, 10, 8, 1.0, None, None) == 0  # no tokens: nothing to do
    g = lib.dprc_embed_plan
    need = lib.dprc_embed_plan_bytes(100, 50)
    assert need > 0
    assert g(P, 8, 100, 50, None, BIG, None) == 5
    assert g(P, 8, 100, 50, P, need - 1, None) == 5
    assert g(None, 8, 100, 50, P, need, None) == 1
    assert g(P, 3, 100, 50, P, need, None) == 3
    assert g(P, 8, 100, 50, P + 4, need, None) == 4
    assert g(P, 8, -5, 50, P, need, None) == 2
    assert g(None, 8, 0, 50, P, need, None) == 0
    for bad in ((-1, 5), (5, 0), ((1 << 30) + 1, 5), (5, (1 << 30) + 1)):
        assert lib.dprc_embed_plan_bytes(*bad) == 0
    ws = lib.dprc_embed_workspace_bytes(1, 2, 50, 16)
    assert ws > 0
    for bad in ((7, 2, 50, 16), (1, 0, 50, 16), (1, 2, -1, 16), (1, 2, 50, 0),
                (1, 65536, 50, 16), (1, 2, 1 << 30, 16)):
        assert lib.dprc_embed_workspace_bytes(*bad) == 0
    n = lib.dprc_embed_norm
    ok = [P, 1, 2, 50, 50, 16, 1.0, P, need, P, 0, P, ws, None]

    def norm(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return n(*a)

    assert norm(_0=None) == 1 and norm(_9=None) == 1
    assert norm(_1=9) == 3
    assert norm(_2=0) == 2 and norm(_3=-1) == 2 and norm(_4=0) == 2 and norm(_5=0) == 2
    assert norm(_6=NAN) == 2
    assert norm(_7=None) == 5 and norm(_8=need - 1) == 5
    assert norm(_11=None) == 5 and norm(_12=ws - 1) == 5
    assert norm(_0=P + 4) == 4 and norm(_9=P + 4) == 4 and norm(_11=P + 4) == 4
    gr = lib.dprc_embed_grad
    okg = [P, 1, P, 2, 50, 50, 16, 1.0, P, need, P, 0, P, ws, None]
    for i, v, code in ((0, None, 1), (10, None, 1), (1, 4, 3), (3, 0, 2), (2, P + 4, 4),
                       (8, None, 5), (13, 0, 5), (10, P + 2, 4)):
        a = list(okg)
        a[i] = v
        assert gr(*a) == code, i


def test_dropout_refusals(lib):
    f = lib.dprc_dropout
    assert f(P, None, 1, 8, 0, 0.1, 1, 1, None, None) == 1
    assert f(None, None, 1, 8, 0, 0.1, 1, 1, P, None) == 1
    assert f(P, None, 3, 8, 0, 0.1, 1, 1, P, None) == 3
    for p in (-0.1, 1.1, NAN):
        assert f(P, None, 1, 8, 0, p, 1, 1, P, None) == 2
    assert f(P, None, 1, -8, 0, 0.1, 1, 1, P, None) == 2
    assert f(P, None, 1, 8, 2 ** 64 - 4, 0.1, 1, 1, P, None) == 2  # the range wraps
    assert f(P + 2, None, 1, 8, 0, 0.1, 1, 1, P, None) == 4
    assert f(P, P + 8, 1, 8, 0, 0.1, 1, 1, P, None) == 4
    assert f(None, None, 1, 0, 0, 0.1, 1, 1, None, None) == 0


def test_linear_refusals(lib):
    b = lib.dprc_linear_workspace_bytes
    ws = b(1, 10, 16, 24, 0)
    wg = b(1, 10, 16, 24, 1)
    assert ws > 0 and wg > 0
    for bad in ((2, 10, 16, 24), (1, -1, 16, 24), (1, 10, 0, 24), (1, 10, 16, 0),
                (1, 10, (1 << 20) + 1, 24)):
        assert b(*bad, 0) == 0 and b(*bad, 1) == 0
    f = lib.dprc_linear
    ok = [P, P, P, P, 1, 10, 16, 24, 3, 0.1, 1, 1, P, P, P, ws, None]

    def lin(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)

    assert lin(0, None) == 1 and lin(1, None) == 1 and lin(13, None) == 1
    assert lin(4, 2) == 3
    assert lin(5, -1) == 2 and lin(6, 0) == 2 and lin(7, 0) == 2
    assert lin(8, 4) == 2 and lin(8, -1) == 2
    assert lin(9, -0.5) == 2 and lin(9, NAN) == 2
    assert lin(14, None) == 5 and lin(15, ws - 1) == 5
    for i in (0, 1, 2, 3, 12, 13, 14):
        assert lin(i, P + 2) == 4, i
    g = lib.dprc_linear_grad
    okg = [P, P, P, P, 1, 10, 16, 24, 3, 0.1, 1, 1, P, P, P, P, P, wg, None]

    def grad(**kw):
        a = list(okg)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return g(*a)

    assert grad(_12=None, _13=None, _14=None, _15=None) == 1  # nothing asked for
    assert grad(_0=None) == 1 and grad(_1=None) == 1 and grad(_2=None) == 1
    assert grad(_3=None) == 1  # an activation's gradient needs Z
    assert grad(_4=2) == 3 and grad(_5=-2) == 2 and grad(_8=9) == 2
    assert grad(_17=wg - 1) == 5
    for i in (0, 1, 2, 3, 12, 13, 14, 15, 16):
        assert grad(**{f"_{i}": P + 2}) == 4, i


def test_binding_refuses_before_the_library():
    import randomized_norm_clipping_gb300 as rnc
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        rnc.dprc_dropout(x, 0.1, 1, 1)  # a host tensor
    with pytest.raises(ValueError):
        rnc.dprc_linear(x, torch.zeros(3, 7))  # widths differ
    with pytest.raises(TypeError):
        rnc.dprc_embed_plan(torch.zeros(2, 3), 5, buf=torch.zeros(1, dtype=torch.uint8))
    assert ctypes.sizeof(ctypes.c_void_p) == 8
