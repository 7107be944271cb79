"""The torch modules on a batch without samples, forward and backward."""

import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from randomized_norm_clipping_gb300 import layers as lay

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [0, 7])
def test_modules_without_samples(dtype, T):
    emb = lay.Embedding(11, 24, device=DEV, dtype=dtype)
    lin = lay.Linear(24, 40, bias=True, act="gelu", p=0.2, device=DEV, dtype=dtype)
    drop = lay.Dropout(0.3)
    tok = torch.zeros((0, T), dtype=torch.int64, device=DEV)
    x = emb(tok)
    y = drop(lin(x, residual=torch.zeros((0, T, 40), device=DEV, dtype=dtype)))
    assert y.shape == (0, T, 40)
    y.sum().backward()
    for p in (emb.weight, lin.weight, lin.bias):
        assert p.grad.shape == p.shape and (p.grad == 0).all()
    torch.cuda.synchronize()
    assert rnc.dprc_device_error(reset=True) == 0
