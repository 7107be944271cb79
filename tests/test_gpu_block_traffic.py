"""Attention and normalisation beside copies on another stream that take the memory's rate: tiles
arrive late and in other orders than alone, and every result stays bitwise what it was.
"""

import pytest
import torch

import randomized_norm_clipping_gb300 as rnc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    torch.cuda.synchronize()
    assert rnc.dprc_device_error(reset=True) == 0


def _documents(B, T):
    ends = torch.tensor([0.11, 0.29, 0.33, 0.62, 0.94]) * T
    d = (torch.arange(T)[None] >= ends[:, None]).sum(0).int()
    d[int(0.94 * T):] = -1
    return d.expand(B, T).contiguous().to(DEV)


def _attention(B, Tq, T, H, Hkv, D, **mask):
    g = torch.Generator(device=DEV).manual_seed(Tq + D)
    q, k, v, do = (torch.randn(B, t, h, D, generator=g, device=DEV).to(BF16)
                   for t, h in ((Tq, H), (T, Hkv), (T, Hkv), (Tq, H)))
    lse = torch.empty(B, H, Tq, device=DEV)

    def run():
        out = rnc.dprc_attention(q, k, v, lse=lse, **mask)
        grads = [torch.empty_like(t) for t in (q, k, v)]
        rnc.dprc_attention_grad(do, q, k, v, out, lse, dQ=grads[0], dK=grads[1], dV=grads[2], **mask)
        return [out, lse.clone(), *grads]
    return run


def _norm(rows, d):
    g = torch.Generator(device=DEV).manual_seed(d)
    x, dy = (torch.randn(4, rows // 4, d, generator=g, device=DEV).to(BF16) for _ in range(2))

    def run():
        stats = torch.empty(4, rows // 4, 2, device=DEV)
        y = rnc.dprc_layernorm(x, stats=stats)
        dx, dw, n = torch.empty_like(x), torch.empty(d, device=DEV, dtype=BF16), torch.empty(4, device=DEV)
        rnc.dprc_layernorm_grad(dy, x, stats, dX=dx, dW=dw, n=n)
        return [y, stats, dx, dw, n]
    return run


CASES = {
    "documents of 64": lambda: _attention(2, 4096, 4096, 32, 8, 64, docs=_documents(2, 4096)),
    "causal of 64": lambda: _attention(2, 2048, 2048, 32, 8, 64),
    "all of 64, capped": lambda: _attention(2, 2000, 2000, 8, 8, 64, causal=False, cap=20.0),
    "documents of 128": lambda: _attention(2, 4096, 4096, 16, 4, 128, docs=_documents(2, 4096)),
    "causal of 128": lambda: _attention(2, 2048, 2048, 16, 4, 128),
    "few tokens of 64": lambda: _attention(8, 1, 8192, 32, 8, 64),
    "few tokens of 128": lambda: _attention(8, 3, 8192, 16, 4, 128),
    "one tile of rows": lambda: _attention(4, 30, 8192, 16, 4, 64),
    "norm of 2048": lambda: _norm(8192, 2048),
    "norm of 2049": lambda: _norm(8192, 2049),
    "norm of 8200": lambda: _norm(2048, 8200),
}


@pytest.mark.parametrize("name", CASES)
def test_results_beside_memory_traffic(name):
    run = CASES[name]()
    alone = run()
    torch.cuda.synchronize()
    a = torch.empty(1 << 28, device=DEV)
    b = torch.empty_like(a)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(12):
        with torch.cuda.stream(other):
            for _ in range(3):
                b.copy_(a)
        beside = run()
        for x, y in zip(alone, beside):
            assert torch.equal(x, y)
    torch.cuda.current_stream().wait_stream(other)
