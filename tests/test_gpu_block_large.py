"""Normalisation, rotary positions and attention on tensors of more than 2^31 elements: their
last rows against the float64 oracle, with the tolerances of test_gpu_block_operators.py.
"""

import numpy as np
import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from oracle import block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    torch.cuda.synchronize()
    assert rnc.dprc_device_error(reset=True) == 0
    torch.cuda.empty_cache()


def _np(t):
    return t.detach().double().cpu().numpy()


def _off(got, ref):
    return np.linalg.norm((_np(got) - ref).ravel()) / np.linalg.norm(ref.ravel())


@pytest.mark.parametrize("d", [1024, 1027])
def test_layernorm_of_many_rows(d):
    B, T, last = 2, (1 << 20) + 3, 40
    x = torch.zeros(B, T, d, dtype=BF16, device=DEV)
    dy = torch.zeros_like(x)
    g = torch.Generator().manual_seed(d)
    X, dY = (torch.randn(last, d, generator=g).to(BF16) for _ in range(2))
    x[1, -last:], dy[1, -last:] = X.to(DEV), dY.to(DEV)
    stats = torch.empty(B, T, 2, device=DEV)
    y = rnc.dprc_layernorm(x, None, None, stats=stats)
    ref, _, _ = block.layernorm(_np(X))
    assert _off(y[1, -last:], ref) <= 2.0 ** -8
    assert not y[0].any() and not y[1, :-last].any()
    dX, W, b = block.layernorm_grad(_np(dY)[None], _np(X)[None])
    dw, db, n = torch.empty(d, dtype=BF16, device=DEV), torch.empty(d, dtype=BF16, device=DEV), torch.empty(B, device=DEV)
    rnc.dprc_layernorm_grad(dy, x, stats, dX=y, dW=dw, db=db, n=n, norm_of_bias=True)
    assert _off(y[1, -last:], dX[0]) <= 2.0 ** -8
    assert not y[0].any() and not y[1, :-last].any()
    assert _off(dw, W[0]) <= 2.0 ** -8 and _off(db, b[0]) <= 2.0 ** -8
    # (statistics in fp32 and 40 terms: the bound of the short ones)
    assert abs(float(n[1]) / ((W ** 2).sum() + (b ** 2).sum()) - 1) <= 64 * 2.0 ** -24
    assert float(n[0]) == 0.0


def test_rotary_of_many_rows():
    B, T, H, D, last = 2, (1 << 20) + 3, 8, 128, 20
    x = torch.zeros(B, T, H, D, dtype=BF16, device=DEV)
    g = torch.Generator().manual_seed(0)
    X = torch.randn(1, last, H, D, generator=g).to(BF16)
    x[1, -last:] = X[0].to(DEV)
    at = torch.arange(T).expand(B, T).contiguous()
    freqs = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)
    for inter in (False, True):
        out = rnc.dprc_rotary(x, at.to(DEV), freqs.to(DEV), interleaved=inter)
        ref = block.rotary(_np(X), at[:1, -last:].numpy(), freqs.numpy(), interleaved=inter)
        assert _off(out[1, -last:], ref[0]) <= 2.0 ** -8
        assert not out[0].any() and not out[1, :-last].any()


@pytest.mark.parametrize("dtype,tol,grad_tol", [(BF16, 2.0 ** -7, 2.0 ** -6),
                                                (torch.float32, 1e-5, 2e-5)])
@pytest.mark.parametrize("Tq", [2, 150])
def test_attention_over_a_long_cache(Tq, dtype, tol, grad_tol):
    """The queries' document is the last keys; what is before them is padding."""
    B, T, H, D, last = 3, 1 << 17, 64, 128, 300
    k = torch.zeros(B, T, H, D, dtype=dtype, device=DEV)
    g = torch.Generator().manual_seed(Tq)
    Q, K, dO = (torch.randn(1, n, H, D, generator=g).to(dtype) for n in (Tq, last, Tq))
    k[-1, -last:] = K[0].to(DEV)
    docs = torch.full((B, T), -1, dtype=torch.int32)
    docs[:, -last:] = 3
    q, do = (torch.cat([torch.zeros_like(t)] * (B - 1) + [t]).to(DEV) for t in (Q, dO))
    lse = torch.empty(B, H, Tq, device=DEV)
    out = rnc.dprc_attention(q, k, k, docs=docs.to(DEV), lse=lse)
    ref = block.attention(_np(Q), _np(K), _np(K), dO=_np(dO))
    assert _off(out[-1], ref[0][0]) <= tol
    assert not out[:-1].any()
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    rnc.dprc_attention_grad(do, q, k, k, out, lse, docs=docs.to(DEV), dQ=dq, dK=dk, dV=dv)
    assert _off(dq[-1], ref[2][0]) <= grad_tol and not dq[:-1].any()
    for got, want in ((dk, ref[3]), (dv, ref[4])):
        assert _off(got[-1, -last:], want[0]) <= grad_tol
        assert not got[:-1].any() and not got[-1, :-last].any()
