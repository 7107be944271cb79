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
