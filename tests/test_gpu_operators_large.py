"""The operators around the norm path on tensors of more than 2^31 elements:
offsets that pass 32 bits, in the table, the gradients, the stream of dropout
and the outputs of the linear map.

Values are chosen so that sums are exact in fp32 where a test says so; the
other bounds are those of test_gpu_operators.py.
"""

import numpy as np
import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from oracle import operators as ops
from randomized_norm_clipping_gb300.workloads import to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ULP = 2.0 ** -23
V, D = 1_200_000, 2048  # 2.46e9 elements
IDS = [0, 1, 1_048_575, 1_048_576, 1_048_577, 1_199_998, 1_199_999, 77]


@pytest.fixture(autouse=True)
def _clean():
    rnc.dprc_device_error(reset=True)
    yield
    assert rnc.dprc_device_error(reset=True) == 0
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def test_lookup_in_a_large_table():
    W = torch.zeros((V, D), dtype=torch.bfloat16, device=DEV)
    ids = torch.tensor(IDS, device=DEV)
    W[ids] = torch.randn((len(IDS), D), generator=_gen(1), device=DEV).bfloat16()
    tokens = ids[torch.randint(len(IDS), (5, 9), generator=_gen(2), device=DEV)]
    assert torch.equal(rnc.dprc_embed_lookup(W, tokens), W[tokens])


def test_gradient_of_a_large_table():
    ids = torch.tensor(IDS, device=DEV)
    tokens = ids[torch.randint(len(IDS), (3, 40), generator=_gen(3), device=DEV)]
    G = torch.randint(-3, 4, (3, 40, D), generator=_gen(4), device=DEV).bfloat16()
    dW = torch.full((V, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    rnc.dprc_embed_grad(G, rnc.dprc_embed_plan(tokens, V), dW)
    ref = torch.zeros((V, D), dtype=torch.bfloat16, device=DEV)
    for t in IDS:  # sums of small integers: exact, then rounded once
        ref[t] = G[tokens == t].float().sum(0).bfloat16()
    assert torch.equal(dW, ref)


def test_norm_over_many_positions():
    B, T, tokens_of = 2, 600_000, 5
    tokens = torch.randint(tokens_of, (B, T), generator=_gen(5), device=DEV)
    G = torch.empty((B, T, D), dtype=torch.bfloat16, device=DEV)
    sums = torch.zeros((B, tokens_of, D), device=DEV)
    for i in range(B):
        G[i] = torch.randint(-1, 2, (T, D), generator=_gen(6 + i), device=DEV, dtype=torch.int8)
        for t0 in range(0, T, 100_000):
            part = slice(t0, t0 + 100_000)
            sums[i].index_add_(0, tokens[i, part], G[i, part].float())  # below 2^24: exact
    n = torch.empty(B, device=DEV)
    plan = rnc.dprc_embed_plan(tokens, tokens_of)
    rnc.dprc_embed_norm(G, plan, n)
    ref = (to_f64(sums) ** 2).sum((1, 2))
    assert (np.abs(to_f64(n) - ref) <= tokens_of * D * ULP * ref).all()
    dW = torch.empty((tokens_of, D), dtype=torch.bfloat16, device=DEV)
    rnc.dprc_embed_grad(G, plan, dW)
    assert torch.equal(dW, sums.sum(0).bfloat16())


def test_dropout_of_a_large_tensor():
    N, first = (1 << 31) + 4099, 3
    x = torch.ones(N, dtype=torch.bfloat16, device=DEV)
    y = rnc.dprc_dropout(x, 0.25, 11, 12, first_element=first)
    for at in (0, (1 << 31) - 2000, N - 4000):
        f = torch.from_numpy(ops.dropout_factor(4000, 0.25, 11, 12, first + at)).bfloat16()
        assert torch.equal(y[at:at + 4000].cpu(), f)


def test_linear_with_a_large_output():
    M, K, N, p = 70_001, 64, 32_768, 0.1
    X = torch.randn((M, K), generator=_gen(9), device=DEV).bfloat16()
    W = torch.randn((N, K), generator=_gen(10), device=DEV).bfloat16()
    rows = [0, 65_535, 65_536, M - 1]
    Y = rnc.dprc_linear(X, W, p=p, seed=5, step=6)
    X64, W64 = to_f64(X[rows]), to_f64(W)
    keep = np.stack([ops.dropout_factor(N, p, 5, 6, r * N) for r in rows])
    ref, size = X64 @ W64.T * keep, np.abs(X64) @ np.abs(W64).T * keep
    bound = 2.0 ** -8 * np.abs(ref) + (K / 16 + 8) * ULP * size
    assert (np.abs(to_f64(Y[rows]) - ref) <= bound).all()

    dX, dZ = torch.empty_like(X), torch.empty_like(Y)
    rnc.dprc_linear_grad(Y, X, W, p=p, seed=5, step=6, dX=dX, dZ=dZ)
    z = to_f64(Y[rows]) * keep
    assert (np.abs(to_f64(dZ[rows]) - z) <= 2.0 ** -8 * np.abs(z)).all()
    ref, size = z @ W64, np.abs(z) @ np.abs(W64)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + (N / 16 + 70) * ULP) * size
    assert (np.abs(to_f64(dX[rows]) - ref) <= bound).all()

    dW, db = torch.empty_like(W), torch.empty(N, dtype=torch.bfloat16, device=DEV)
    rnc.dprc_linear_grad(Y, X, W, dW=dW, db=db)
    cols = [0, 127, 20_000, N - 1]
    y, x = Y[:, cols].double(), X.double()
    ref, size = (y.T @ x).cpu().numpy(), (y.abs().T @ x.abs()).cpu().numpy()
    bound = 2.0 ** -8 * np.abs(ref) + (M / 16 + 70) * ULP * size
    assert (np.abs(to_f64(dW[cols]) - ref) <= bound).all()
    ref, size = y.sum(0).cpu().numpy(), y.abs().sum(0).cpu().numpy()
    assert (np.abs(to_f64(db[cols]) - ref) <= 2.0 ** -8 * np.abs(ref) + M * ULP * size).all()
