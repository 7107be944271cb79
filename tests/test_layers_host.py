"""The torch modules without a GPU: the library's calls come from the oracle."""

import pytest
import torch

import host_library
from randomized_norm_clipping_gb300 import layers as lay


@pytest.fixture(autouse=True)
def _host(monkeypatch):
    host_library.install(monkeypatch)
    torch.manual_seed(3)


# ---- second derivatives ----------------------------------------------------
@pytest.mark.parametrize("which", ["embedding", "dropout", "linear"])
def test_second_derivatives_are_an_error(which):
    """The backward passes run outside the graph; a gradient of a gradient would
    take them for constants."""
    x = torch.randn(4, 6, requires_grad=True)
    if which == "embedding":
        m = lay.Embedding(5, 6)
        y, wrt = m(torch.tensor([[0, 1, 4, 4]])).tanh(), m.weight
    elif which == "dropout":
        y, wrt = lay.Dropout(0.4, seed=2)(x).tanh(), x
    else:
        y, wrt = lay.Linear(6, 3, act="gelu")(x).tanh(), x
    (g,) = torch.autograd.grad(y.sum(), wrt, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (g ** 2).sum().backward()


def test_first_derivatives_may_be_taken_twice():
    m, x = lay.Linear(6, 3, bias=True, act="silu", p=0.3, seed=4), torch.randn(5, 6)
    y = m(x)
    g = [torch.autograd.grad(y.sum(), m.weight, retain_graph=True)[0] for _ in range(2)]
    assert torch.equal(g[0], g[1])


# ---- what a backward pass goes by ------------------------------------------
@pytest.mark.parametrize("change", ["seed", "act", "p", "step"])
def test_backward_goes_by_the_call_and_not_by_the_module(change):
    m = lay.Linear(6, 3, bias=True, act="silu", p=0.4, seed=4)
    x = torch.randn(50, 6, requires_grad=True)
    wrt = [x, m.weight, m.bias]
    want = torch.autograd.grad(m(x).sum(), wrt)
    m.step = 0
    y = m(x)
    last, dy = m._last, torch.ones(50, 3)
    dz = m.preactivation_grad(dy, last)
    setattr(m, change, {"seed": 9, "act": "relu", "p": 0.1, "step": 5}[change])
    got = torch.autograd.grad(y.sum(), wrt)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(m.preactivation_grad(dy, last), dz)
