"""The operators around the norm path against the float64 oracle
(oracle/operators.py): embedding lookup, order, per-sample norm and clipped
gradient, dropout, the linear map with its epilogue and its gradient.

Tolerances are derived, element by element:
  - a bf16 result is rounded once: 2^-8 |y| covers half an ulp (2^-9) with room
    for the fp32 value's own error;
  - a sum of n fp32 terms errs by at most n 2^-23 sum |terms| (each addition
    rounds or truncates by at most one ulp of a partial sum);
  - a tensor-core sum adds 16 products per step: K / 16 such additions, plus
    a few for the shares' sum and the epilogue; for fp32 inputs there are six
    plane products per step, and the products left out are below 2^-22 of a
    term;
  - an activation is Lipschitz with a constant below 1.2 and its own evaluation
    errs by less than 2^-18 (1 + |z|) (bf16: hardware exponential) or 2^-21
    (1 + |z|) (fp32);
  - a bf16 gradient's dZ enters its products rounded: 2^-9 of each term, twice
    that as the bound.
"""

import numpy as np
import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from oracle import operators as ops
from randomized_norm_clipping_gb300.workloads import to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ULP = 2.0 ** -23


def _gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def _randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * scale).to(DT[dtype])


def _round(dtype, y):
    """The rounding of a result to its type."""
    return (2.0 ** -8 if dtype == "bf16" else 2.0 ** -23) * np.abs(y)


def _close(got, ref, bound):
    got = to_f64(got)
    assert got.shape == ref.shape
    assert np.isfinite(got).all()
    excess = np.abs(got - ref) - bound
    i = np.unravel_index(np.argmax(excess), excess.shape) if excess.size else None
    assert excess.size == 0 or excess[i] <= 0, (
        f"at {i}: got {got[i]}, want {ref[i]}, bound {bound[i]}")


@pytest.fixture(autouse=True)
def _no_device_error():
    rnc.dprc_device_error(reset=True)
    yield
    torch.cuda.synchronize()
    assert rnc.dprc_device_error(reset=True) == 0


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
def _tokens(kind, B, T, V, seed):
    g = _gen(seed)
    if kind == "one":
        return torch.zeros(B, T, dtype=torch.int64)
    if kind == "none":
        return torch.full((B, T), -1, dtype=torch.int64)
    if kind == "uniform":
        return torch.randint(0, V, (B, T), generator=g)
    if kind == "runs":  # a few tokens, each many times, in stretches; some padding
        t = torch.randint(0, max(1, V // 8), (B, T), generator=g) * min(8, V) % V
        t[:, T // 3: T // 2] = V - 1
        t[torch.rand(B, T, generator=g) < 0.1] = -1
        return t
    t = (torch.exp(torch.rand(B, T, generator=g) * np.log(V + 1.0)) - 1).long().clamp(0, V - 1)
    t[:, T - T // 5:] = -1
    return t


EMBED = [
    # kind, B, T, V, d, dtype
    ("zipf", 1, 1, 1, 1, "bf16"),
    ("zipf", 4, 128, 1000, 64, "f32"),
    ("one", 3, 200, 1, 40, "bf16"),
    ("one", 2, 5000, 7, 264, "bf16"),
    ("none", 2, 50, 9, 16, "f32"),
    ("runs", 3, 777, 40, 96, "bf16"),
    ("runs", 2, 2100, 17, 33, "f32"),
    ("uniform", 5, 33, 2000, 520, "bf16"),
    ("zipf", 2, 3000, 3000, 1025, "bf16"),
    ("zipf", 7, 31, 100, 2050, "bf16"),
    ("zipf", 1, 6001, 70000, 12, "bf16"),
    ("uniform", 16, 1, 3, 321, "f32"),
    ("zipf", 2, 33, 128, 130, "f32"),
    ("zipf", 1, 4097, 1024, 24, "f32"),
]


@pytest.mark.parametrize("kind,B,T,V,d,dtype", EMBED)
@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_lookup(kind, B, T, V, d, dtype, ids):
    tok = _tokens(kind, B, T, V, 1)
    W = _randn((V, d), dtype, 2)
    out = rnc.dprc_embed_lookup(W.to(DEV), tok.to(ids).to(DEV), scale=1.7)
    ref = ops.embed_lookup(to_f64(W), tok.numpy(), np.float64(np.float32(1.7)))
    assert out.dtype == W.dtype and out.shape == (B, T, d)
    _close(out, ref, _round(dtype, ref))
    assert (to_f64(out)[tok.numpy() < 0] == 0).all()


@pytest.mark.parametrize("N,V", [(1, 1), (2, 3), (31, 1000), (33, 5), (1024, 1023), (1025, 1024),
                                 (4096, 200000), (4097, 70000), (20001, 2), (70000, 128256),
                                 (9000, (1 << 20) + 5), (300, 1 << 30)])
def test_plan_is_the_stable_order(N, V):
    g = _gen(N)
    tok = torch.randint(-2, V, (1, N), generator=g)
    if V > 4:
        tok[0, ::3] = torch.randint(0, 4, (tok[0, ::3].numel(),), generator=g)
    plan = rnc.dprc_embed_plan(tok.to(DEV), V)
    torch.cuda.synchronize()
    key = np.where(tok[0].numpy() < 0, V, tok[0].numpy())
    order = np.argsort(key, kind="stable")
    step = (4 * N + 255) // 256 * 256
    raw = plan.buf.cpu().numpy()
    assert (raw[:4 * N].view(np.uint32) == key[order]).all()
    assert (raw[step:step + 4 * N].view(np.int32) == order).all()


def _longest_run(tok):
    return max([int(np.unique(t[t >= 0], return_counts=True)[1].max()) for t in tok
                if (t >= 0).any()] or [0])


@pytest.mark.parametrize("kind,B,T,V,d,dtype", EMBED)
def test_norm_and_gradient(kind, B, T, V, d, dtype):
    tok = _tokens(kind, B, T, V, 3)
    G = _randn((B, T, d), dtype, 4, 0.1)
    # what stands at positions without a token is not read
    G[tok < 0] = float("nan")
    clean = torch.where((tok >= 0)[..., None], G, torch.zeros((), dtype=G.dtype))
    g64, t = to_f64(clean), tok.numpy()
    scale = 1.25
    plan = rnc.dprc_embed_plan(tok.to(DEV), V)
    Gd = G.to(DEV)

    ref = ops.embed_norm(g64, t, V, scale)
    size = ops.embed_norm(np.abs(g64), t, V, scale)  # sum over tokens of (sum |g|)^2
    run = _longest_run(t)
    bound = (2 * (run + 2) + 40 + np.log2(T * d + 1)) * ULP * size
    n = torch.full((B,), 7.0, device=DEV)
    assert rnc.dprc_embed_norm(Gd, plan, n, scale=scale) is n
    _close(n, ref, bound)
    again = torch.empty_like(n)
    rnc.dprc_embed_norm(Gd, plan, again, scale=scale)
    assert torch.equal(n, again)
    rnc.dprc_embed_norm(Gd, plan, n, scale=scale, accumulate=True)
    _close(n, 2 * ref, 2 * bound + 2 * ULP * ref)

    c = torch.rand(B, generator=_gen(5)) + 0.1
    for factors in (None, c):
        f = None if factors is None else factors.double().numpy()
        dref = ops.embed_grad(g64, t, V, f, scale)
        dsize = ops.embed_grad(np.abs(g64), t, V, f, scale)
        total = np.unique(t[t >= 0], return_counts=True)[1].max() if (t >= 0).any() else 0
        dbound = _round(dtype, dref) + (total + 6) * ULP * dsize
        cd = None if factors is None else factors.to(DEV)
        dW = torch.full((V, d), float("nan"), dtype=G.dtype, device=DEV)
        rnc.dprc_embed_grad(Gd, plan, dW, c=cd, scale=scale)
        _close(dW, dref, dbound)
        # on top of what is there; rows without a token stay as they are
        base = _randn((V, d), dtype, 6)
        acc = base.to(DEV)
        rnc.dprc_embed_grad(Gd, plan, acc, c=cd, scale=scale, accumulate=True)
        aref = to_f64(base) + dref
        _close(acc, aref, _round(dtype, aref) + (total + 6) * ULP * dsize)
        absent = np.setdiff1d(np.arange(V), t[t >= 0])
        assert torch.equal(acc.cpu()[absent], base[absent])


def test_embedding_without_tokens():
    plan = rnc.dprc_embed_plan(torch.empty((2, 0), dtype=torch.int64, device=DEV), 5)
    G = torch.empty((2, 0, 8), device=DEV)
    n = torch.ones(2, device=DEV)
    rnc.dprc_embed_norm(G, plan, n, accumulate=True)
    assert (n.cpu() == 1).all()
    rnc.dprc_embed_norm(G, plan, n)
    assert (n.cpu() == 0).all()
    dW = torch.ones((5, 8), device=DEV)
    rnc.dprc_embed_grad(G, plan, dW, accumulate=True)
    assert (dW.cpu() == 1).all()
    rnc.dprc_embed_grad(G, plan, dW)
    assert (dW.cpu() == 0).all()
    out = rnc.dprc_embed_lookup(torch.ones((5, 8), device=DEV),
                                torch.empty((0,), dtype=torch.int64, device=DEV))
    assert out.shape == (0, 8)


def test_tokens_out_of_range_are_recorded_and_read_nothing():
    W = torch.ones((5, 8), device=DEV)
    out = rnc.dprc_embed_lookup(W, torch.tensor([0, 5, 2 ** 40, -3], device=DEV))
    assert (out.cpu().sum(1) == torch.tensor([8.0, 0.0, 0.0, 0.0])).all()
    assert rnc.dprc_device_error(reset=True) == 8
    tok = torch.tensor([[0, 9, 0, -1]], device=DEV)
    plan = rnc.dprc_embed_plan(tok, 5)
    n = torch.empty(1, device=DEV)
    rnc.dprc_embed_norm(torch.ones((1, 4, 8), device=DEV), plan, n)
    assert n.item() == 2 * 2 * 8
    assert rnc.dprc_device_error(reset=True) == 8


def test_norm_shows_a_non_finite_gradient():
    tok = torch.tensor([[1, 1, 2], [0, 0, 0]], device=DEV)
    G = torch.ones((2, 3, 8), device=DEV)
    G[0, 1, 3] = float("inf")
    n = torch.empty(2, device=DEV)
    rnc.dprc_embed_norm(G, rnc.dprc_embed_plan(tok, 3), n)
    assert not torch.isfinite(n[0]) and n[1].item() == 9 * 8


def test_bias_norm_by_the_one_row_embedding():
    G = _randn((3, 1000, 72), "bf16", 8)
    plan = rnc.dprc_embed_plan(torch.zeros((3, 1000), dtype=torch.int32, device=DEV), 1)
    n = torch.empty(3, device=DEV)
    rnc.dprc_embed_norm(G.to(DEV), plan, n)
    ref = (to_f64(G).sum(1) ** 2).sum(1)
    size = (np.abs(to_f64(G)).sum(1) ** 2).sum(1)
    _close(n, ref, 2100 * ULP * size)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("N", [0, 1, 7, 8, 9, 1003, 100003, 1 << 20])
@pytest.mark.parametrize("first", [0, 5, 8 * 7, (1 << 40) + 3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("res", [False, True])
def test_dropout(N, first, dtype, res):
    x = _randn((N,), dtype, 1)
    r = _randn((N,), dtype, 2) if res else None
    y = rnc.dprc_dropout(x.to(DEV), 0.3, 99, 5, residual=None if r is None else r.to(DEV),
                         first_element=first)
    ref = ops.dropout(to_f64(x), 0.3, 99, 5, None if r is None else to_f64(r), first)
    _close(y, ref, _round(dtype, ref) + 3 * ULP * (2 * np.abs(to_f64(x)) + 1))
    if not res:
        keep = ops.dropout_factor(N, 0.3, 99, 5, first) > 0
        assert ((to_f64(y) != 0) == (keep & (to_f64(x) != 0))).all()


@pytest.mark.parametrize("p", [0.0, 1.0, 0.5])
def test_dropout_ends_and_masked_values(p):
    x = _randn((4000,), "f32", 3)
    f = ops.dropout_factor(4000, p, 1, 2)
    x[torch.from_numpy(f == 0)] = float("nan")  # a dropped element is 0, whatever it held
    y = rnc.dprc_dropout(x.to(DEV), p, 1, 2)
    ref = np.where(f == 0, 0.0, to_f64(torch.nan_to_num(x)) * f)
    _close(y, ref, 2 * ULP * np.abs(ref))


def test_dropout_in_place_and_its_gradient():
    x = _randn((1003,), "f32", 4).to(DEV)
    r = _randn((1003,), "f32", 5).to(DEV)
    y = rnc.dprc_dropout(x, 0.4, 7, 7, residual=r)
    acc = r.clone()
    rnc.dprc_dropout(x, 0.4, 7, 7, residual=acc, out=acc)
    assert torch.equal(acc, y)
    same = x.clone()
    rnc.dprc_dropout(same, 0.4, 7, 7, out=same)
    assert torch.equal(same, rnc.dprc_dropout(x, 0.4, 7, 7))
    # linear in x: the gradient is the same call; a difference shows it
    g = torch.ones_like(x)
    dx = rnc.dprc_dropout(g, 0.4, 7, 7)
    d = (rnc.dprc_dropout(x + 0.5, 0.4, 7, 7) - rnc.dprc_dropout(x - 0.5, 0.4, 7, 7))
    assert torch.allclose(d, dx, atol=4e-6)


# ---------------------------------------------------------------------------
# linear map
# ---------------------------------------------------------------------------
LINEAR = [
    # M, K, N
    (1, 16, 16),
    (1, 2048, 512),
    (8, 1000, 264),
    (17, 72, 1032),
    (33, 200, 130),
    (64, 520, 96),
    (65, 64, 64),
    (128, 128, 256),
    (200, 1, 1),
    (130, 7, 9),
    (257, 333, 515),
    (1000, 520, 264),
    (700, 2112, 136),
    (2500, 40, 700),
]


def _linear_bounds(dtype, X, W, b, z, name):
    """Bounds of z and of act(z) before their rounding."""
    size = np.abs(X) @ np.abs(W).T + (0 if b is None else np.abs(b))
    steps = X.shape[1] / 16 * (6 if dtype == "f32" else 1) + 80
    ez = (steps + (4 if dtype == "f32" else 0)) * ULP * size
    ea = ez if name == "none" else (
        1.2 * ez + (2.0 ** -18 if dtype == "bf16" else 2.0 ** -21) * (1 + np.abs(z)))
    return ez, ea


@pytest.mark.parametrize("M,K,N", LINEAR)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name,bias,res,p", [("none", False, False, 0.0), ("silu", True, False, 0.0),
                                             ("gelu", True, True, 0.2), ("relu", False, True, 0.0)])
def test_linear(M, K, N, dtype, name, bias, res, p):
    X, W = _randn((M, K), dtype, 1), _randn((N, K), dtype, 2, K ** -0.5)
    b = _randn((N,), dtype, 3) if bias else None
    r = _randn((M, N), dtype, 4) if res else None
    dev = [None if t is None else t.to(DEV) for t in (X, W, b, r)]
    f = [None if t is None else to_f64(t) for t in (X, W, b, r)]
    y, z = ops.linear(f[0], f[1], f[2], name, p, 31, 2, f[3])
    ez, ea = _linear_bounds(dtype, f[0], f[1], f[2], z, name)
    Z = torch.full((M, N), float("nan"), dtype=X.dtype, device=DEV)
    out = rnc.dprc_linear(dev[0], dev[1], bias=dev[2], act=name, p=p, seed=31, step=2,
                          residual=dev[3], Z=Z)
    _close(Z, z, _round(dtype, z) + ez)
    _close(out, y, _round(dtype, y) + ea / (1 - p) + 3 * ULP * np.abs(y - 0))
    again = rnc.dprc_linear(dev[0], dev[1], bias=dev[2], act=name, p=p, seed=31, step=2,
                            residual=dev[3])
    assert torch.equal(out, again)  # bitwise, and the same without Z
    if p > 0 and not res:
        assert ((to_f64(out) == 0) == (ops.dropout_factor(M * N, p, 31, 2).reshape(M, N) == 0)).all()


@pytest.mark.parametrize("M,K,N", LINEAR)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name,p", [("none", 0.0), ("silu", 0.0), ("gelu", 0.2), ("relu", 0.3)])
def test_linear_grad(M, K, N, dtype, name, p):
    X, W = _randn((M, K), dtype, 1), _randn((N, K), dtype, 2, K ** -0.5)
    dY, Z = _randn((M, N), dtype, 3, 0.1), _randn((M, N), dtype, 4)
    f = [to_f64(t) for t in (dY, X, W, Z)]
    dX, dW, db, dz = ops.linear_grad(*f, name, p, 31, 2)
    # dZ itself, before and after its rounding for the products
    slope_err = 0.0 if name in ("none", "relu") else (2.0 ** -17 if dtype == "bf16" else 2.0 ** -20)
    edz = 4 * ULP * np.abs(dz) + slope_err * np.abs(f[0]) * (1 + np.abs(f[3])) / (1 - p)
    same = name == "none" and p == 0
    rdz = edz + (0.0 if dtype == "f32" or same else 2.0 ** -8) * np.abs(dz)
    steps = 6 if dtype == "f32" else 1
    aX, aW = np.abs(f[1]), np.abs(f[2])
    bX = _round(dtype, dX) + rdz @ aW + (steps * N / 16 + 84) * ULP * (np.abs(dz) @ aW)
    bW = _round(dtype, dW) + rdz.T @ aX + (steps * M / 16 + 84) * ULP * (np.abs(dz).T @ aX)
    bb = _round(dtype, db) + edz.sum(0) + (M / 8 + 80) * ULP * np.abs(dz).sum(0)
    t = dict(dX=torch.empty_like(X), dW=torch.empty_like(W), db=torch.empty(N, dtype=X.dtype),
             dZ=torch.empty_like(dY))
    t = {k: v.to(DEV) for k, v in t.items()}
    dev = [v.to(DEV) for v in (dY, X, W, Z)]
    kw = dict(Z=None if name == "none" else dev[3], act=name, p=p, seed=31, step=2)
    rnc.dprc_linear_grad(*dev[:3], **kw, **t)
    _close(t["dZ"], dz, _round(dtype, dz) + edz)
    _close(t["dX"], dX, bX)
    _close(t["dW"], dW, bW)
    _close(t["db"], db, bb)
    # each output asked for alone is the same, bit for bit
    for k in t:
        one = torch.empty_like(t[k])
        rnc.dprc_linear_grad(*dev[:3], **kw, **{k: one})
        assert torch.equal(one, t[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_without_tokens(dtype):
    X, W = torch.empty((0, 24), dtype=DT[dtype], device=DEV), _randn((8, 24), dtype, 1).to(DEV)
    assert rnc.dprc_linear(X, W).shape == (0, 8)
    dW, db = torch.ones_like(W), torch.ones(8, dtype=DT[dtype], device=DEV)
    rnc.dprc_linear_grad(torch.empty((0, 8), dtype=DT[dtype], device=DEV), X, W, dW=dW, db=db,
                         dX=torch.empty_like(X))
    assert (dW.float().cpu() == 0).all() and (db.float().cpu() == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 300])
def test_non_finite_rows_stay_in_their_rows(dtype, M):
    X, W = _randn((M, 136), dtype, 1), _randn((72, 136), dtype, 2)
    X[1, 5] = float("nan")
    X[2, 7] = float("inf")
    y = rnc.dprc_linear(X.to(DEV), W.to(DEV)).cpu().float()
    assert not torch.isfinite(y[1]).any() and not torch.isfinite(y[2]).any()
    rest = [i for i in range(M) if i not in (1, 2)]
    assert torch.isfinite(y[rest]).all()


def test_linear_in_place_residual_and_leading_axes():
    X, W = _randn((2, 70, 64), "bf16", 1).to(DEV), _randn((64, 64), "bf16", 2, 0.1).to(DEV)
    r = _randn((2, 70, 64), "bf16", 3).to(DEV)
    y = rnc.dprc_linear(X, W, residual=r, act="silu", p=0.1, seed=1, step=1)
    acc = r.clone()
    rnc.dprc_linear(X, W, residual=acc, act="silu", p=0.1, seed=1, step=1, out=acc)
    assert y.shape == (2, 70, 64) and torch.equal(acc, y)


def test_linear_gradient_against_differences():
    """fp32, one direction per operand, through the library's own forward."""
    M, K, N = 90, 48, 56
    X, W = _randn((M, K), "f32", 1), _randn((N, K), "f32", 2, 0.2)
    b, dY = _randn((N,), "f32", 3), _randn((M, N), "f32", 4)
    kw = dict(act="gelu", p=0.2, seed=3, step=3)
    d = [t.to(DEV) for t in (X, W, b, dY)]
    Z = torch.empty((M, N), device=DEV)
    rnc.dprc_linear(d[0], d[1], bias=d[2], Z=Z, **kw)
    out = dict(dX=torch.empty_like(d[0]), dW=torch.empty_like(d[1]), db=torch.empty_like(d[2]))
    rnc.dprc_linear_grad(d[3], d[0], d[1], Z=Z, **kw, **out)
    h = 2.0 ** -6
    for i, k in enumerate(("dX", "dW", "db")):
        D = torch.randn(d[i].shape, generator=_gen(10 + i)).to(DEV)
        up, dn = list(d), list(d)
        up[i], dn[i] = d[i] + h * D, d[i] - h * D
        f = [(rnc.dprc_linear(v[0], v[1], bias=v[2], **kw).double() * d[3].double()).sum().item()
             for v in (up, dn)]
        slope = (out[k].double() * D.double()).sum().item()
        # central difference: h^2 / 6 of a third derivative (below 3 per term),
        # and the forward's rounding over 2 h
        terms = (d[3].abs().double().sum() * 1.25).item()
        third = {"dX": K * 0.2, "dW": K, "db": 1.0}[k] ** 1.5
        assert abs((f[0] - f[1]) / (2 * h) - slope) < terms * (h * h * third + 60 * ULP / h), k


def test_operators_on_another_stream():
    """Inputs made on the stream the call is given, and read there."""
    s = torch.cuda.Stream()
    tok = torch.randint(0, 50, (2, 300), device=DEV)
    W = torch.randn(50, 64, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out = rnc.dprc_embed_lookup(W, tok)
        plan = rnc.dprc_embed_plan(tok, 50)
        n = torch.empty(2, device=DEV)
        rnc.dprc_embed_norm(out, plan, n)
        y = rnc.dprc_linear(out, W[:48].contiguous())
        z = rnc.dprc_dropout(y, 0.1, 1, 1)
    s.synchronize()
    ref = ops.embed_lookup(to_f64(W), tok.cpu().numpy())
    assert np.allclose(to_f64(out), ref)
    nref = ops.embed_norm(ref, tok.cpu().numpy(), 50)
    assert np.allclose(to_f64(n), nref, rtol=1e-4)
    assert np.allclose(to_f64(z), ops.dropout(to_f64(y), 0.1, 1, 1), rtol=1e-6)


def test_calls_on_a_given_stream_allocate_there():
    """out, plan and workspace left to the binding, the stream given by handle."""
    s = torch.cuda.Stream()
    x = torch.randn(300, 64, device=DEV)
    W = torch.randn(40, 64, device=DEV)
    tok = torch.randint(0, 40, (3, 100), device=DEV)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        y = rnc.dprc_linear(x, W, act="gelu", stream=stream)
        e = rnc.dprc_embed_lookup(W, tok, stream=stream)
        plan = rnc.dprc_embed_plan(tok, 40, stream=stream)
        n = torch.zeros(3, device=DEV)
        torch.cuda.synchronize()
        rnc.dprc_embed_norm(e, plan, n, stream=stream)
        d = rnc.dprc_dropout(y, 0.5, 1, 2, stream=stream)
        s.synchronize()
        ref = ops.linear(to_f64(x), to_f64(W), None, "gelu")[0]
        assert np.allclose(to_f64(y), ref, rtol=1e-4, atol=1e-4)
        assert np.allclose(to_f64(d), ops.dropout(to_f64(y), 0.5, 1, 2), rtol=1e-6)
        assert np.allclose(to_f64(n), ops.embed_norm(to_f64(e), tok.cpu().numpy(), 40), rtol=1e-5)


@pytest.mark.parametrize("B,T", [(300, 40), (1500, 17)])
def test_many_samples_with_long_runs(B, T):
    """More than 16 equal tokens in every sample, many samples."""
    tok = torch.randint(0, 2, (B, T), generator=_gen(1)) * 3
    tok[::3] = 1
    G = _randn((B, T, 300), "bf16", 2)
    n = torch.empty(B, device=DEV)
    rnc.dprc_embed_norm(G.to(DEV), rnc.dprc_embed_plan(tok.to(DEV), 5), n)
    ref = ops.embed_norm(to_f64(G), tok.numpy(), 5)
    size = ops.embed_norm(np.abs(to_f64(G)), tok.numpy(), 5)
    _close(n, ref, (2 * (T + 2) + 40 + np.log2(T * 300)) * ULP * size)


def test_values_at_the_ends_of_the_range():
    """fp32 maps of values next to the largest, and the slopes of large z."""
    X = torch.zeros(70, 64)
    X[:, 0] = 3.4e38
    X[:, 1] = 1.0
    W = torch.zeros(8, 64)
    W[:, 0], W[:, 1] = 0.5, 2.0
    for rows in (4, 70):  # both paths
        y = rnc.dprc_linear(X[:rows].to(DEV), W.to(DEV))
        assert torch.isfinite(y).all()
        ref = to_f64(X[:rows]) @ to_f64(W).T
        _close(y, ref, 8 * ULP * np.abs(ref))
    Z = torch.tensor([[3e19, -3e19, 1e30, -1e30, 0.0, 80.0, -80.0, 5.0]] * 3)
    dZ = torch.empty(3, 8, device=DEV)
    rnc.dprc_linear_grad(torch.ones(3, 8, device=DEV), None, torch.zeros(8, 16, device=DEV),
                         Z=Z.to(DEV), act="gelu", dZ=dZ)
    assert np.allclose(dZ.cpu().numpy()[:, :7], [1, 0, 1, 0, 0.5, 1, 0], atol=1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_back_to_back_on_one_workspace(dtype):
    """Kernels of a call run side by side and its successor starts while it
    ends: calls on one workspace in turn give what each gives alone."""
    sizes = [(1001, 517, 263), (40, 264, 136), (300, 128, 776), (5, 1000, 333), (513, 96, 72)]
    problems, ws_bytes = [], 1
    for j, (M, K, N) in enumerate(sizes):
        dY, X = _randn((M, N), dtype, 10 * j).to(DEV), _randn((M, K), dtype, 10 * j + 1).to(DEV)
        W, Z = _randn((N, K), dtype, 10 * j + 2).to(DEV), _randn((M, N), dtype, 10 * j + 3).to(DEV)
        outs = [torch.empty_like(t) for t in (X, W, W[:, 0].contiguous(), dY)]
        problems.append((dY, X, W, Z, outs))
        ws_bytes = max(ws_bytes, rnc.binding.lib().dprc_linear_workspace_bytes(
            rnc.DPRC_F32 if dtype == "f32" else rnc.DPRC_BF16, M, K, N, 1))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=DEV)

    def call(j):
        dY, X, W, Z, (dX, dW, db, dZ) = problems[j]
        rnc.dprc_linear_grad(dY, X, W, Z=Z, act="silu", p=0.1, seed=3, step=j, dX=dX, dW=dW,
                             db=db, dZ=dZ if j % 2 else None, ws=ws)

    alone = []
    for j in range(len(sizes)):
        torch.cuda.synchronize()
        call(j)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in problems[j][4][:3]])
    order, results = torch.randint(len(sizes), (60,), generator=_gen(9)).tolist(), []
    for j in order:
        for t in problems[j][4]:
            t.fill_(float("nan"))
        call(j)
        results.append([t.clone() for t in problems[j][4][:3]])
    torch.cuda.synchronize()
    for j, got in zip(order, results):
        for a, b in zip(got, alone[j]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,K,N", [(5001, 200, 4112), (3001, 512, 2000)])
@pytest.mark.parametrize("name,bias,p", [("none", False, 0.0), ("none", True, 0.1),
                                         ("gelu", True, 0.0)])
def test_linear_of_many_tiles(M, K, N, name, bias, p):
    """Sizes of a hundred 256 x 256 tiles and more, with ragged edges: the
    residual added, read and written in place, and the gradient."""
    X, W = _randn((M, K), "bf16", 21), _randn((N, K), "bf16", 22, K ** -0.5)
    b = _randn((N,), "bf16", 23) if bias else None
    r, dY = _randn((M, N), "bf16", 24), _randn((M, N), "bf16", 25)
    Xd, Wd, rd, gd = (t.to(DEV) for t in (X, W, r, dY))
    bd = None if b is None else b.to(DEV)
    f = [None if t is None else to_f64(t) for t in (X, W, b, r)]
    y, z = ops.linear(f[0], f[1], f[2], name, p, 41, 3, f[3])
    ez, ea = _linear_bounds("bf16", f[0], f[1], f[2], z, name)
    kw = dict(bias=bd, act=name, p=p, seed=41, step=3)
    Z = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    out = rnc.dprc_linear(Xd, Wd, residual=rd, Z=Z, **kw)
    _close(Z, z, _round("bf16", z) + ez)
    _close(out, y, _round("bf16", y) + ea / (1 - p) + 3 * ULP * np.abs(y))
    assert torch.equal(out, rnc.dprc_linear(Xd, Wd, residual=rd, **kw))
    acc = rd.clone()
    rnc.dprc_linear(Xd, Wd, residual=acc, out=acc, **kw)
    assert torch.equal(out, acc)

    # the gradient at the kernel's own Z, which both sides then hold exactly
    dX, dW = torch.empty_like(Xd), torch.empty_like(Wd)
    db, dZ = torch.empty(N, dtype=torch.bfloat16, device=DEV), torch.empty_like(Z)
    rnc.dprc_linear_grad(gd, Xd, Wd, Z=Z, act=name, p=p, seed=41, step=3, dX=dX, dW=dW, db=db, dZ=dZ)
    gX, gW, gb, gZ = ops.linear_grad(to_f64(dY), f[0], f[1], to_f64(Z), name, p, 41, 3)
    ez = 2.0 ** -17 * np.abs(to_f64(dY)) * (1 + np.abs(to_f64(Z)))
    _close(dZ, gZ, _round("bf16", gZ) + ez)
    eZ = 2.0 ** -8 * np.abs(gZ) + ez  # dZ as it enters the products
    aX, aW = np.abs(f[0]), np.abs(f[1])
    _close(dX, gX, _round("bf16", gX) + eZ @ aW + (N / 16 + 80) * ULP * (np.abs(gZ) @ aW))
    _close(dW, gW, _round("bf16", gW) + eZ.T @ aX + (M / 16 + 80) * ULP * (np.abs(gZ).T @ aX))
    _close(db, gb, _round("bf16", gb) + ez.sum(0) + M * ULP * np.abs(gZ).sum(0))


@pytest.mark.parametrize("N,V", [(8193, 1 << 30), (200_003, (1 << 21) + 3), (65_537, 300)])
def test_plans_in_one_buffer(N, V):
    """Orders of several digits, one after the other in the same memory."""
    buf = torch.empty(rnc.binding.lib().dprc_embed_plan_bytes(N, V), dtype=torch.uint8, device=DEV)
    step = (4 * N + 255) // 256 * 256
    for seed in range(4):
        tok = torch.randint(-1, V, (1, N), generator=_gen(seed))
        tok[0, :N // 2] = torch.randint(0, 1 + seed, (N // 2,), generator=_gen(seed + 9))
        rnc.dprc_embed_plan(tok.to(DEV), V, buf=buf)
        key = np.where(tok[0].numpy() < 0, V, tok[0].numpy())
        order = np.argsort(key, kind="stable")
        raw = buf.cpu().numpy()
        assert (raw[:4 * N].view(np.uint32) == key[order]).all()
        assert (raw[step:step + 4 * N].view(np.int32) == order).all()


@pytest.mark.parametrize("M,K,N", [(3001, 475, 2466), (2300, 264, 2049), (5001, 2049, 136)])
@pytest.mark.parametrize("name,bias,p", [("none", True, 0.1), ("gelu", False, 0.4)])
def test_linear_of_many_odd_tiles(M, K, N, name, bias, p):
    test_linear_of_many_tiles(M, K, N, name, bias, p)


@pytest.mark.parametrize("M,K,N", [(2305, 130, 2049), (3001, 1027, 70)])
def test_linear_of_many_odd_tiles_f32(M, K, N):
    X, W = _randn((M, K), "f32", 31), _randn((N, K), "f32", 32, K ** -0.5)
    b, r = _randn((N,), "f32", 33), _randn((M, N), "f32", 34)
    f = [to_f64(t) for t in (X, W, b, r)]
    y, z = ops.linear(f[0], f[1], f[2], "silu", 0.2, 51, 4, f[3])
    ez, ea = _linear_bounds("f32", f[0], f[1], f[2], z, "silu")
    Z = torch.empty((M, N), device=DEV)
    out = rnc.dprc_linear(X.to(DEV), W.to(DEV), bias=b.to(DEV), act="silu", p=0.2, seed=51, step=4,
                          residual=r.to(DEV), Z=Z)
    _close(Z, z, _round("f32", z) + ez)
    _close(out, y, _round("f32", y) + ea / 0.8 + 3 * ULP * np.abs(y))
    dX, dW = torch.empty((M, K), device=DEV), torch.empty((N, K), device=DEV)
    rnc.dprc_linear_grad(r.to(DEV), X.to(DEV), W.to(DEV), dX=dX, dW=dW)
    aX, aW, ar = (np.abs(t) for t in (f[0], f[1], f[3]))
    ref = f[3] @ f[1]
    _close(dX, ref, _round("f32", ref) + (6 * N / 16 + 84) * ULP * (ar @ aW))
    ref = f[3].T @ f[0]
    _close(dW, ref, _round("f32", ref) + (6 * M / 16 + 84) * ULP * (ar.T @ aX))
