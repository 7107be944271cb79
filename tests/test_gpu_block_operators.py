"""Normalisation, rotary positions and attention against the float64 oracle, through the
C ABI.

Tolerances (relative to the 2-norm of a result, unless said otherwise) count roundings:
half a step is 2^-24 for fp32 and 2^-8 for bf16.  fp32 results are sums of n
terms in fp32, whose errors grow as sqrt(n) half steps of the terms' 2-norm, with a factor
for the few operations of a term.  bf16 results are rounded once (at most 2^-8, in the
2-norm of many values below 2^-8.5); attention's also come from weights rounded to bf16.
"""

import numpy as np
import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    torch.cuda.synchronize()
    assert rnc.dprc_device_error(reset=True) == 0


def _np(t):
    return t.detach().double().cpu().numpy()


def _randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _near(got, ref, tol, what="", terms=0.0):
    """terms: an absolute part, the roundings of terms that cancel."""
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape
    assert np.isfinite(got[np.isfinite(ref)]).all(), what
    off = np.linalg.norm((got - ref).ravel())
    size = np.linalg.norm(ref.ravel())
    assert off <= tol * size + terms + 1e-30, (what, off / max(size, 1e-300), tol, terms)


# ---------------------------------------------------------------------------
# normalisation
# ---------------------------------------------------------------------------
# fp32: x - mu, its square's mean (sqrt(16384) = 128 half steps at worst by the walk of a
# sum, relative to a sum of positive terms: below 8 half steps for pairwise-like
# trees of threads), 1 / sqrt, two products and a sum: 32 half steps.
NORM = {F32: 32 * 2.0 ** -24, BF16: 2.0 ** -8}
WIDTHS = [1, 2, 7, 8, 9, 12, 64, 100, 122, 256, 321, 1000, 2048, 2049, 2052, 4095, 4096, 4104, 8200, 12290,
          16383, 16384]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layernorm(d, dtype):
    for center, w, b, rows in ((True, True, True, (2, 3)), (False, True, False, (5,)),
                               (True, False, False, (1, 1))):
        X = _randn((*rows, d), dtype, d, 1.5) + (3.0 if center else 0.0)
        W = (1 + _randn((d,), F32, d + 1, 0.2)).to(dtype) if w else None
        Bv = _randn((d,), dtype, d + 2, 0.3) if b else None
        ref, mu, r = block.layernorm(_np(X), None if W is None else _np(W),
                                     None if Bv is None else _np(Bv), 1e-5, center)
        stats = torch.empty(*rows, 2, device=DEV)
        y = rnc.dprc_layernorm(X.to(DEV), None if W is None else W.to(DEV),
                               None if Bv is None else Bv.to(DEV), center=center, stats=stats)
        # (d = 1 with the mean taken out: x - mu is 0 exactly, and so is y without a bias)
        _near(y, ref, NORM[dtype])
        # the mean relative to the values' size, whose sum it is
        assert np.abs(_np(stats)[..., 0] - mu).max() <= 8 * 2.0 ** -24 * np.abs(_np(X)).max()
        # r: the variance's relative error is that of (x - mu)^2, i.e. mu's error against
        # the deviation: at most 8 half steps of |x| over a deviation that d values have
        if d > 8 or not center:
            _near(stats[..., 1], r, 64 * 2.0 ** -24)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layernorm_grad(d, dtype):
    for center, B, T, w in ((True, 3, 37, True), (False, 1, 130, True), (True, 70, 2, False),
                            (False, 2, 1, False)):
        if d > 4200 and B == 70:
            B = 65
        X = _randn((B, T, d), dtype, d, 1.5) + (0.5 if center else 0.0)
        dY = _randn((B, T, d), dtype, d + 1)
        W = (1 + _randn((d,), F32, d + 2, 0.2)).to(dtype) if w else None
        if center and d < 8:  # (a deviation near 0 magnifies the roundings of x - mu)
            continue
        dX, Ws, bs = block.layernorm_grad(_np(dY), _np(X), None if W is None else _np(W),
                                          center=center)
        _, mu, r = block.layernorm(_np(X), center=center)
        stats = torch.from_numpy(np.stack((mu, r), -1)).float().to(DEV)
        args = dict(weight=None if W is None else W.to(DEV), center=center)
        x, dy = X.to(DEV), dY.to(DEV)
        dx, dw, db = torch.empty_like(x), torch.empty(d, device=DEV, dtype=dtype), None
        db = torch.empty(d, device=DEV, dtype=dtype)
        c = torch.rand(B, generator=torch.Generator().manual_seed(d))
        cn = c.double().numpy()[:, None]
        n = torch.full((B,), 2.0, device=DEV)
        rnc.dprc_layernorm_grad(dy, x, stats, dX=dx, dW=dw, db=db, n=n, norm_of_bias=True,
                                accumulate=True, c=c.to(DEV), **args)
        # dX is a difference of g, its mean and xh mean(g xh) (of one element without the
        # mean: r g (1 - xh^2), which is near 0), each to 8 half steps of fp32
        g = np.abs(_np(dY) * (1.0 if W is None else _np(W)))
        xh = np.abs((_np(X) - mu[..., None]) * r[..., None])
        size = (g + g.mean(-1, keepdims=True) + xh * (g * xh).mean(-1, keepdims=True)) * r[..., None]
        _near(dx, dX, NORM[dtype], "dX", 8 * 2.0 ** -24 * np.linalg.norm(size))
        _near(dw, (cn * Ws).sum(0), NORM[dtype], "dW")
        _near(db, (cn * bs).sum(0), NORM[dtype], "db")
        _near(n, 2.0 + (Ws ** 2).sum(1) + (bs ** 2).sum(1), 64 * 2.0 ** -24, "n")
        # the same without the norms (the samples' factors are taken by row), alone, and
        # n of the weight alone
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        rnc.dprc_layernorm_grad(dy, x, stats, dW=dw2, db=db2, c=c.to(DEV), **args)
        _near(dw2, (cn * Ws).sum(0), NORM[dtype], "dW alone")
        _near(db2, (cn * bs).sum(0), NORM[dtype], "db alone")
        dx2 = torch.empty_like(dx)
        rnc.dprc_layernorm_grad(dy, x, stats, dX=dx2, **args)
        assert torch.equal(dx2, dx)
        rnc.dprc_layernorm_grad(dy, x, stats, n=n, **args)
        _near(n, (Ws ** 2).sum(1), 64 * 2.0 ** -24, "n of the weight")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,d", [(3, 333, 5), (1, 1001, 31), (5, 77, 129), (2, 500, 257), (2, 701, 1023),
                                   (1, 400, 3001), (1, 130, 5003)])
def test_layernorm_grad_of_many_odd_rows(B, T, d, dtype):
    """Blocks of rows that start at every element of 16 bytes and end with the tensor; the
    gradient in the place of dY."""
    X, dY = _randn((B, T, d), dtype, d, 1.5), _randn((B, T, d), dtype, d + 1)
    W = (1 + _randn((d,), F32, d + 2, 0.2)).to(dtype)
    dX, Ws, bs = block.layernorm_grad(_np(dY), _np(X), _np(W), center=False)
    _, mu, r = block.layernorm(_np(X), center=False)
    stats = torch.from_numpy(np.stack((mu, r), -1)).float().to(DEV)
    g = dY.to(DEV)
    dw, db, n = (torch.empty(k, device=DEV, dtype=t) for k, t in ((d, dtype), (d, dtype), (B, F32)))
    rnc.dprc_layernorm_grad(g, X.to(DEV), stats, W.to(DEV), center=False, dX=g, dW=dw, db=db, n=n,
                            norm_of_bias=True)
    _near(g, dX, NORM[dtype])
    _near(dw, Ws.sum(0), NORM[dtype])
    _near(db, bs.sum(0), NORM[dtype])
    _near(n, (Ws ** 2).sum(1) + (bs ** 2).sum(1), 64 * 2.0 ** -24)


def test_layernorm_large_mean_and_empty():
    """A mean of 1000 deviations: the variance is summed of differences."""
    X = _randn((4, 5, 512), F32, 3) + 1000.0
    y = rnc.dprc_layernorm(X.to(DEV))
    ref, _, _ = block.layernorm(_np(X))
    # the mean's half steps (8 of 1000 2^-24 = 5e-4 of a deviation at worst)
    _near(y, ref, 8 * 1000 * 2.0 ** -24)
    e = rnc.dprc_layernorm(torch.empty(2, 0, 16, device=DEV))
    assert e.shape == (2, 0, 16)
    n, dw = torch.full((2,), 7.0, device=DEV), torch.full((16,), 7.0, device=DEV)
    z = torch.empty(2, 0, 16, device=DEV)
    rnc.dprc_layernorm_grad(z, z, torch.empty(2, 0, 2, device=DEV), dW=dw, n=n)
    assert (n == 0).all() and (dw == 0).all()


def test_layernorm_grad_against_differences():
    """fp64 differences of the loss sum(y u) along a direction."""
    X, u = _randn((2, 9, 48), F32, 1, 2.0), _randn((2, 9, 48), F32, 2)
    w, v = 1 + _randn((48,), F32, 3, 0.2), _randn((2, 9, 48), F32, 4)
    stats = torch.empty(2, 9, 2, device=DEV)
    rnc.dprc_layernorm(X.to(DEV), w.to(DEV), stats=stats)
    dx, dw = torch.empty(2, 9, 48, device=DEV), torch.empty(48, device=DEV)
    rnc.dprc_layernorm_grad(u.to(DEV), X.to(DEV), stats, w.to(DEV), dX=dx, dW=dw)
    f = lambda x, ww: float((block.layernorm(x, ww)[0] * _np(u)).sum())  # noqa: E731
    h = 1e-5
    for got, diff in ((float((_np(dx) * _np(v)).sum()),
                       (f(_np(X) + h * _np(v), _np(w)) - f(_np(X) - h * _np(v), _np(w))) / (2 * h)),
                      (float((_np(dw) * _np(v)[0, 0]).sum()),
                       (f(_np(X), _np(w) + h * _np(v)[0, 0]) - f(_np(X), _np(w) - h * _np(v)[0, 0])) / (2 * h))):
        assert abs(got - diff) <= 1e-5 * max(1.0, abs(diff))


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
# fp32: the angle's part of a turn to half a step (2^-25 of a turn, 3.8e-7 rad at
# most half a turn away), the sine's two steps, two products and a sum: 8 half steps
ROT = {F32: 8 * 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,H,D,sections", [
    (1, 1, 1, 2, [1]), (2, 5, 3, 8, [4]), (2, 33, 5, 64, [32]), (1, 7, 2, 44, [7, 7, 7]),
    (3, 4, 40, 80, [16, 0, 24]), (2, 9, 3, 40, [12]), (1, 300, 2, 128, [20, 22, 22]),
    (1, 3, 1, 4096, [2048]), (1, 2, 65, 13, [5]), (4, 1, 8, 64, [32])])
def test_rotary(dtype, interleaved, B, T, H, D, sections):
    P, axes = sum(sections), len(sections)
    X = _randn((B, T, H + 1, D), dtype, D + T)
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(-1000, 1 << 20, (B, T, axes), generator=g)
    if axes == 1:
        pos = pos[..., 0]
    freqs = 10000.0 ** (-torch.arange(P, dtype=torch.float64) / P)
    x = X.to(DEV)[:, :, :H]  # (a stride that is not H D)
    for inverse, ids in ((False, pos), (True, pos.int())):
        ref = block.rotary(_np(X)[:, :, :H], pos.numpy(), freqs.numpy(), sections, interleaved,
                           inverse)
        y = rnc.dprc_rotary(x, ids.to(DEV), freqs.to(DEV), sections, interleaved, inverse)
        _near(y, ref, ROT[dtype])
    keep = X.to(DEV)
    rnc.dprc_rotary(keep[:, :, :H], pos.to(DEV), freqs.to(DEV), sections, interleaved, True,
                    out=keep[:, :, :H])
    assert torch.equal(keep[:, :, :H], y) and torch.equal(keep[:, :, H].cpu(), X[:, :, H])


def test_rotary_far_positions():
    """Angles of positions near 2^31 and 2^40 keep fp64's reduction: 2^40 turns of 2^-53."""
    for far, tol in ((2 ** 31 - 5, 1e-6), (2 ** 40, 2.0 ** -10)):
        X = _randn((1, 4, 2, 16), F32, 1)
        pos = torch.arange(4)[None] + far
        freqs = 10000.0 ** (-torch.arange(8, dtype=torch.float64) / 8)
        y = rnc.dprc_rotary(X.to(DEV), pos.to(DEV), freqs.to(DEV))
        _near(y, block.rotary(_np(X), pos.numpy(), freqs.numpy()), tol)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
# fp32: a score is a sum of D products (sqrt(D) half steps of |q||k| scale, up to some 40
# with these inputs: 40 * 11 * 2^-24 = 3e-5 absolute in the exponent at the very worst, near
# 2e-6 as it is met), the tanh and exp two steps each: 1e-5.  bf16: weights rounded to
# 2^-8 at most, 2^-9.2 in the mean square, the output once more: 2^-7; the gradients of the
# scores are differences of two terms of which each rounds, delta from a rounded output:
# 2^-6.
ATT = {F32: 1e-5, BF16: 2.0 ** -7}
ATT_GRAD = {F32: 2e-5, BF16: 2.0 ** -6}
# dS is p (dP - delta): of a query that sees one key, the difference of two equal sums of D
# products, whose half steps remain (sqrt(128) of them, 12; 16 with the sums' products), and
# for bf16 delta's, which is formed of the rounded output: 2^-8 of its terms.  So dQ and dK
# may be off by that share of the terms' sizes, which the oracle sums too.
CANCEL = {F32: 16 * 2.0 ** -24, BF16: 2.0 ** -8}


def _mask(kind, B, Tq, Tk, seed=0):
    g = torch.Generator().manual_seed(seed + Tk)
    r = lambda lo, hi: torch.randint(lo, max(hi, lo + 1), (B,), generator=g).int()  # noqa: E731
    m = {}
    if kind == "full":
        m["causal"] = False
    elif kind == "prefix":
        m["prefix"] = r(0, Tk + 1)
    elif kind == "documents":  # runs, padding at the end, one id that comes back
        d = torch.sort(torch.randint(0, 4, (B, Tk), generator=g), 1).values.int()
        d[:, Tk - Tk // 5:] = -1
        if Tk > 40:
            d[:, 20:25] = 9
            d[0, -3:] = 9
        m["docs"] = d
    elif kind == "lengths":  # some samples empty, queries in the middle
        m["lengths"] = r(0, Tk + 1)
        m["lengths"][0] = 0
        m["first"] = r(-3, Tk)
    elif kind == "all":
        m = _mask("documents", B, Tq, Tk, seed)
        m["prefix"] = r(0, Tk // 2 + 1)
        m["lengths"] = r(Tk // 2, Tk + 1)
    elif kind == "full documents":
        m = _mask("documents", B, Tq, Tk, seed)
        m["causal"] = False
    return m


def _attend(dtype, B, Tq, Tk, H, Hkv, D, mask, cap=0.0, slopes=False, gain=1.0, strided=False,
            grad=True, seed=0):
    if strided and Tq == Tk:
        rows = _randn((B, Tk, H + 2 * Hkv, D), dtype, seed + 1, gain)
        Q, K, V = rows[:, :, :H], rows[:, :, H:H + Hkv], rows[:, :, H + Hkv:]
        dev = rows.to(DEV)
        q, k, v = dev[:, :, :H], dev[:, :, H:H + Hkv], dev[:, :, H + Hkv:]
    else:
        Q = _randn((B, Tq, H, D), dtype, seed + 1, gain)
        K, V = _randn((B, Tk, Hkv, D), dtype, seed + 2), _randn((B, Tk, Hkv, D), dtype, seed + 3)
        q, k, v = Q.to(DEV), K.to(DEV), V.to(DEV)
        if strided:  # heads before tokens
            q, k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v))
    kw = dict(cap=cap)
    if slopes:
        kw["slopes"] = torch.exp2(-8.0 * (torch.arange(H) + 1.0) / H)
    kw.update(mask)
    on = {n: x.to(DEV) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    host = {n: _np(x) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    lse = torch.full((B, H, Tq), 7.0, device=DEV)
    out = rnc.dprc_attention(q, k, v, lse=lse, **on)
    dO = _randn((B, Tq, H, D), dtype, seed + 4)
    ref = block.attention(_np(Q), _np(K), _np(V), dO=_np(dO), **host)
    _near(out, ref[0], ATT[dtype], "out")
    got, want = _np(lse), ref[1]
    none = np.isinf(want)
    assert (got[none] == -np.inf).all()
    # lse is a logarithm: 1e-5 absolute per unit of the scores' size
    assert np.abs(got[~none] - want[~none]).max(initial=0.0) <= 1e-5 * (1 + np.abs(want[~none]).max(initial=0.0))
    if not grad:
        return
    if strided and Tq == Tk:
        g = torch.full((B, Tk, H + 2 * Hkv, D), 7.0, dtype=dtype, device=DEV)
        dq, dk, dv = g[:, :, :H], g[:, :, H:H + Hkv], g[:, :, H + Hkv:]
    else:
        dq, dk, dv = (torch.full(t.shape, 7.0, dtype=dtype, device=DEV) for t in (q, k, v))
    do = dO.to(DEV)
    if strided:  # heads before tokens
        out, do = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (out, do))
    rnc.dprc_attention_grad(do, q, k, v, out, lse, dQ=dq, dK=dk, dV=dv, **on)
    for name, a, b, terms in (("dQ", dq, ref[2], ref[5]), ("dK", dk, ref[3], ref[6]),
                              ("dV", dv, ref[4], 0.0)):
        _near(a, b, ATT_GRAD[dtype], name, CANCEL[dtype] * np.linalg.norm(terms))
    a, b = torch.empty_like(dq), torch.empty_like(dk)
    rnc.dprc_attention_grad(do, q, k, v, out, lse, dQ=a, dK=b, **on)
    assert torch.equal(a, dq) and torch.equal(b, dk)  # (and again, bitwise)
    b = torch.empty_like(dv)
    rnc.dprc_attention_grad(do, q, k, v, out, lse, dV=b, **on)
    assert torch.equal(b, dv)


MASKS = ["causal", "full", "prefix", "documents", "lengths", "all", "full documents"]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("B,T,H,Hkv,D", [
    (1, 1, 1, 1, 8), (2, 2, 2, 1, 16), (2, 63, 4, 2, 64), (1, 64, 3, 3, 32), (2, 65, 4, 1, 40),
    (1, 128, 2, 2, 128), (2, 129, 7, 1, 72), (1, 200, 12, 4, 64), (1, 300, 8, 8, 80),
    (1, 513, 4, 1, 128), (1, 777, 2, 2, 64)])
def test_attention_of_a_sequence(dtype, mask, B, T, H, Hkv, D):
    _attend(dtype, B, T, T, H, Hkv, D, _mask(mask, B, T, T), strided=T % 2 == 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("cap,slopes", [(15.0, False), (0.0, True), (5.0, True)])
def test_attention_caps_and_slopes(dtype, mask, cap, slopes):
    for T, D in ((150, 64), (270, 104)):
        _attend(dtype, 2, T, T, 6, 2, D, _mask(mask, 2, T, T), cap, slopes, gain=3.0 if cap else 1.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mask", ["causal", "full", "prefix", "documents", "lengths"])
@pytest.mark.parametrize("B,Tq,Tk,H,Hkv,D", [
    (3, 1, 1, 2, 1, 64), (2, 1, 100, 32, 8, 64), (4, 1, 1000, 8, 1, 128), (1, 1, 5000, 4, 4, 64),
    (2, 3, 700, 6, 2, 80), (1, 16, 2000, 8, 2, 64), (1, 40, 1500, 4, 1, 64), (2, 5, 3, 4, 2, 64),
    (1, 1, 260, 130, 1, 32)])
def test_attention_of_few_tokens(dtype, mask, B, Tq, Tk, H, Hkv, D):
    _attend(dtype, B, Tq, Tk, H, Hkv, D, _mask(mask, B, Tq, Tk), cap=20.0 if Tq == 3 else 0.0,
            slopes=Tq == 16, strided=Tk % 2 == 1, grad=Tk < 1200)


@pytest.mark.parametrize("D", [1, 3, 17, 33, 65, 100, 127])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_odd_widths(dtype, D):
    _attend(dtype, 2, 70, 70, 4, 2, D, _mask("documents", 2, 70, 70))
    _attend(dtype, 2, 70, 70, 4, 2, D, {}, strided=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [1, 47, 127])
@pytest.mark.parametrize("T", [943, 200, 450])
def test_attention_of_few_tokens_of_odd_widths(dtype, D, T):
    """Shares of odd numbers of odd rows, whose statistics lie at whole 8 bytes."""
    _attend(dtype, 3, 5, T, 3, 3, D, _mask("lengths", 3, 5, T), slopes=True, grad=False)
    _attend(dtype, 1, 1, T, 3, 1, D, {}, grad=False)


def test_attention_of_nothing():
    for dtype in (F32, BF16):
        q, kv = _randn((2, 3, 4, 64), dtype, 1).to(DEV), torch.empty(2, 0, 2, 64, device=DEV, dtype=dtype)
        lse = torch.zeros(2, 4, 3, device=DEV)
        out = rnc.dprc_attention(q, kv, kv, lse=lse)
        assert (out == 0).all() and (lse == -np.inf).all()
        dq = torch.ones_like(q)
        rnc.dprc_attention_grad(q, q, kv, kv, out, lse, dQ=dq, dK=torch.empty_like(kv))
        assert (dq == 0).all()
        e = q[:, :0]
        assert rnc.dprc_attention(e, q, q).shape == (2, 0, 4, 64)
        dk = torch.ones_like(q)
        rnc.dprc_attention_grad(e, e, q, q, e, lse[:, :, :0].contiguous(), dK=dk)
        assert (dk == 0).all()


@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128), (BF16, 33)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_ignores_what_nobody_sees(dtype, D, bad):
    """Keys behind the lengths, padding, and rows that see nothing may hold anything."""
    B, T = 2, 200
    lengths = torch.tensor([77, 130], dtype=torch.int32)
    docs = torch.zeros(B, T, dtype=torch.int32)
    docs[0, 40:] = 1
    docs[:, 60:66] = -1
    for mask, empty in ((dict(lengths=lengths), None), (dict(docs=docs), docs < 0)):
        Q, K, V, dO = (_randn((B, T, 4, D), dtype, i) for i in range(4))
        hidden = (torch.arange(T)[None] >= lengths[:, None]) if empty is None else empty
        K[hidden], V[hidden] = bad, bad
        if empty is not None:
            Q[hidden], dO[hidden] = bad, bad
        on = {n: x.to(DEV) for n, x in mask.items()}
        q, k, v, do = (t.to(DEV) for t in (Q, K, V, dO))
        lse = torch.empty(B, 4, T, device=DEV)
        out = rnc.dprc_attention(q, k, v, lse=lse, **on)
        ref = block.attention(_np(Q), _np(K), _np(V), dO=_np(dO), **{n: _np(x) for n, x in mask.items()})
        _near(out, ref[0], ATT[dtype])
        dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
        rnc.dprc_attention_grad(do, q, k, v, out, lse, dQ=dq, dK=dk, dV=dv, **on)
        for a, b in ((dq, ref[2]), (dk, ref[3]), (dv, ref[4])):
            _near(a, b, ATT_GRAD[dtype])


def test_attention_grad_against_differences():
    Q, K, V, u, d = (_randn((1, 20, h, 16), F32, i) for i, h in enumerate((4, 2, 2, 4, 4)))
    kw = dict(cap=3.0, slopes=torch.tensor([0.5, 0.1, 0.02, 0.0]), prefix=torch.tensor([5]).int())
    on = {n: x.to(DEV) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    host = {n: _np(x) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    lse = torch.empty(1, 4, 20, device=DEV)
    q, k, v = Q.to(DEV), K.to(DEV), V.to(DEV)
    out = rnc.dprc_attention(q, k, v, lse=lse, **on)
    g = [torch.empty_like(t) for t in (q, k, v)]
    rnc.dprc_attention_grad(u.to(DEV), q, k, v, out, lse, dQ=g[0], dK=g[1], dV=g[2], **on)
    h = 1e-5
    for i in range(3):
        step = _np(d) if i == 0 else _np(d)[:, :, :2]
        f = []
        for sgn in (1, -1):
            args = [_np(Q), _np(K), _np(V)]
            args[i] = args[i] + sgn * h * step
            f.append(float((block.attention(*args, **host)[0] * _np(u)).sum()))
        diff = (f[0] - f[1]) / (2 * h)
        assert abs(float((_np(g[i]) * step).sum()) - diff) <= 1e-4 * max(1.0, abs(diff)), i


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cap", [1e-30, 300.0, 4000.0, 1e5, 1e17, 3e38])
def test_attention_of_any_cap(dtype, cap):
    """A score is off by at most 2^-22 of a cap up to 4096 (bf16, an exponential's tanh), else
    by a few half steps of itself; the weights, lse and delta by as much."""
    off = cap * 2.0 ** -22 if dtype is BF16 and cap <= 4096 else 0.0
    for Tq, T in ((150, 150), (3, 500)):
        Q, K, V, dO = (_randn((2, t, h, 64), dtype, i, g) for i, (t, h, g) in
                       enumerate(((Tq, 4, 3.0), (T, 2, 1.0), (T, 2, 1.0), (Tq, 4, 1.0))))
        q, k, v, do = (t.to(DEV) for t in (Q, K, V, dO))
        lse = torch.empty(2, 4, Tq, device=DEV)
        out = rnc.dprc_attention(q, k, v, cap=cap, lse=lse)
        ref = block.attention(_np(Q), _np(K), _np(V), cap=cap, dO=_np(dO))
        _near(out, ref[0], ATT[dtype] + off)
        assert np.abs(_np(lse) - ref[1]).max() <= 1e-5 * (1 + np.abs(ref[1]).max()) + off
        dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
        rnc.dprc_attention_grad(do, q, k, v, out, lse, cap=cap, dQ=dq, dK=dk, dV=dv)
        # Where t is near 1 (a tiny cap's slope is 0), 1 - t^2 is off by the reciprocal's half
        # steps: 12 of them.  A row's weights add up to 1 and |dp|, |delta| <= |do| max |v|,
        # so dS is off by 24 half steps of that at most, and dQ, dK by the sums of it.
        size = lambda t: np.linalg.norm(_np(t), axis=-1).max()  # noqa: E731
        lost = 32 * 2.0 ** -24 * 64 ** -0.5 * np.linalg.norm(_np(dO)) * size(V)
        for name, a, b, terms, by in (("dQ", dq, ref[2], ref[5], size(K)),
                                      ("dK", dk, ref[3], ref[6], np.linalg.norm(_np(Q))),
                                      ("dV", dv, ref[4], 0.0, 0.0)):
            _near(a, b, ATT_GRAD[dtype] + 2 * off, name,
                  CANCEL[dtype] * np.linalg.norm(terms) + lost * by)


@pytest.mark.parametrize("H,Hkv,D", [(32, 8, 64), (8, 2, 128)])
@pytest.mark.parametrize("mask", ["documents", "causal", "full"])
def test_attention_whose_values_come_late(mask, H, Hkv, D):
    """Many CTAs at a time, whose groups of rows get ahead of the copies of the values: every wait
    ends (the fixture reads the error word), and a sample's head is right."""
    B, T = 4, 4096
    m = _mask(mask, B, T, T)
    rows = _randn((B, T, H + 2 * Hkv, D), BF16, 1)
    dev = rows.to(DEV)
    on = {n: x.to(DEV) if isinstance(x, torch.Tensor) else x for n, x in m.items()}
    outs = [rnc.dprc_attention(dev[:, :, :H], dev[:, :, H:H + Hkv], dev[:, :, H + Hkv:], **on)
            for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    one = {n: _np(x[B - 1:]) if isinstance(x, torch.Tensor) else x for n, x in m.items()}
    ref = block.attention(_np(rows[B - 1:, :, H - 1:H]), _np(rows[B - 1:, :, H + Hkv - 1:H + Hkv]),
                          _np(rows[B - 1:, :, H + 2 * Hkv - 1:]), **one)[0]
    _near(outs[0][B - 1:, :, H - 1:], ref, ATT[BF16])
