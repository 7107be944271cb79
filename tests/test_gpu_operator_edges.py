"""The operators around the norm path where calls follow one another closely or
their inputs are at an end of the range."""

import numpy as np
import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from oracle import operators as ops
from randomized_norm_clipping_gb300.workloads import to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


@pytest.fixture(autouse=True)
def _no_device_error():
    rnc.dprc_device_error(reset=True)
    yield
    torch.cuda.synchronize()
    assert rnc.dprc_device_error(reset=True) == 0


@pytest.mark.parametrize("B,T,V", [(3, 3000, (1 << 20) + 5), (2, 6000, 1500), (4, 700, 90)])
def test_plans_norms_and_gradients_in_turn_without_a_pause(B, T, V):
    """Each call's kernels start while the ones before them end, in the same
    buffers every time.  Whole numbers, so that every sum is exact: n below
    2^24, dW below 2^24."""
    rounds, d = 12, 8
    toks = [torch.randint(0, 40 + j, (B, T), generator=_gen(j)) * (V // 60) % V
            for j in range(rounds)]
    Gs = [torch.randint(-1, 2, (B, T, d), generator=_gen(100 + j)).float() for j in range(rounds)]
    for t in toks:
        t[:, T - 5:] = -1
    dt, dg = [t.to(DEV) for t in toks], [g.to(DEV) for g in Gs]
    buf = rnc.dprc_embed_plan(dt[0], V).buf
    ns = [torch.empty(B, device=DEV) for _ in range(rounds)]
    dW = torch.empty(V, d, device=DEV)
    rows = []
    used = torch.unique(torch.cat([t.reshape(-1) for t in toks]))
    used = used[used >= 0].to(DEV)
    torch.cuda.synchronize()
    for j in range(rounds):
        plan = rnc.dprc_embed_plan(dt[j], V, buf=buf)
        rnc.dprc_embed_norm(dg[j], plan, ns[j])
        rnc.dprc_embed_grad(dg[j], plan, dW)
        rows.append(dW[used])
    for j in range(rounds):
        tok = toks[j].numpy()
        assert np.array_equal(to_f64(ns[j]), ops.embed_norm(to_f64(Gs[j]), tok, V)), j
        small = np.searchsorted(used.cpu().numpy(), np.where(tok < 0, 0, tok))
        small[tok < 0] = -1
        ref = ops.embed_grad(to_f64(Gs[j]), small, len(used))
        assert np.array_equal(to_f64(rows[j]), ref), j


@pytest.mark.parametrize("B,T,d", [(1, 513, 16), (5, 2000, 24), (3, 40, 2048 * 16), (9, 600, 8)])
def test_norms_whose_sums_a_cluster_joins(B, T, d):
    """More than 512 squares a sample, so that eight CTAs add them; whole
    numbers, exact sums, many calls in turn."""
    V = 1 << 20
    tok = torch.randperm(V, generator=_gen(1))[:B * T].view(B, T)  # no token twice
    G = torch.zeros(B, T, d)
    G[..., ::max(1, d // 8)] = torch.randint(-2, 3, (B, T, len(range(0, d, max(1, d // 8)))),
                                             generator=_gen(2)).float()
    g = G.to(DEV)
    plan = rnc.dprc_embed_plan(tok.to(DEV), V)
    ns = [rnc.dprc_embed_norm(g, plan, torch.empty(B, device=DEV)) for _ in range(50)]
    ref = (to_f64(G) ** 2).sum((1, 2))
    for n in ns:
        assert np.array_equal(to_f64(n), ref)


ULP = 2.0 ** -23
# the largest third derivatives: GELU 0.7813, SiLU 0.3127
THIRD = {"none": 0.0, "gelu": 0.8, "silu": 0.32}


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("M", [16, 90])
def test_linear_gradient_against_differences_along_it(M, act):
    """fp32: the library's gradient against central differences of its own forward
    map along the gradient's direction, where the slope is large against the
    differences' error, so that a gradient that is zero, halved, of the other sign,
    or zero in a tenth of its entries would fail."""
    K, N, kw = 48, 56, dict(act=act, p=0.2, seed=3, step=3)
    gen = [torch.randn(s, generator=_gen(i)) for i, s in enumerate(((M, K), (N, K), (N,), (M, N)))]
    X, W, b, dY = gen[0], 0.2 * gen[1], gen[2], gen[3]
    d = [t.to(DEV) for t in (X, W, b, dY)]
    Z = torch.empty((M, N), device=DEV)
    rnc.dprc_linear(d[0], d[1], bias=d[2], Z=Z, **kw)
    out = dict(dX=torch.empty_like(d[0]), dW=torch.empty_like(d[1]), db=torch.empty_like(d[2]))
    rnc.dprc_linear_grad(d[3], d[0], d[1], Z=Z, **kw, **out)
    x, w, bias, dy = (to_f64(t) for t in (X, W, b, dY))
    z = ops.linear(x, w, bias, act, 0.2, 3, 3)[1]
    ref = ops.linear_grad(dy, x, w, z, act, 0.2, 3, 3)
    weight = np.abs(dy) * ops.dropout_factor(M * N, 0.2, 3, 3).reshape(M, N)
    # the forward's error: a sum's (as in test_gpu_operators.py), the activation's
    # and the output's rounding
    ez = (6 * K / 16 + 84) * ULP * (np.abs(x) @ np.abs(w).T + np.abs(bias))
    forward = (weight * (1.2 * ez + 2.0 ** -21 * (1 + np.abs(z)))).sum()
    for i, k in enumerate(("dX", "dW", "db")):
        g, at = ref[i], (x, w, bias)[i]
        D = g / (np.abs(g).max() if i == 2 else np.sqrt((g ** 2).sum(-1, keepdims=True)))
        D = D.astype(np.float32).astype(np.float64)
        u = D @ w.T if i == 0 else x @ D.T if i == 1 else np.broadcast_to(D, (M, N))
        # central differences err by h^2 / 6 of the third derivative and by the
        # forward's error (and the moved operand's rounding) over h
        third = THIRD[act] * (weight * np.abs(u) ** 3).sum() / 6
        error = forward + 2.0 ** -24 * (np.abs(g) * (np.abs(at) + np.abs(D))).sum()
        h = 2.0 ** np.round(np.log2((error / (2 * third)) ** (1 / 3))) if third else 1.0
        tol = error / h + third * h * h
        slope = (to_f64(out[k]) * D).sum()
        assert tol < 0.03 * abs((g * D).sum()), (k, tol, slope)
        f = []
        for sign in (1, -1):
            v = list(d)
            v[i] = (d[i].double() + sign * h * torch.from_numpy(D).to(DEV)).float()
            y = rnc.dprc_linear(v[0], v[1], bias=v[2], **kw)
            f.append((y.double() * d[3].double()).sum().item())
        diff = (f[0] - f[1]) / (2 * h)
        assert abs(diff - slope) < tol, (k, diff, slope, tol)
        part = to_f64(out[k])
        part.reshape(-1)[::10] = 0.0
        for wrong in (0.0 * slope, 0.5 * slope, -slope, (part * D).sum()):
            assert abs(diff - wrong) > tol, (k, wrong)
