"""The torch modules without a GPU: the library's calls come from the oracle."""

import copy
import gc
import os
import pickle
import weakref

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


# ---- activation checkpointing ----------------------------------------------
def checkpoint(*args, **kw):
    # (it imports triton, which tests/test_oracle.py runs in its interpreter)
    os.environ["TRITON_INTERPRET"] = "1"
    from torch.utils import checkpoint as c
    return c.checkpoint(*args, **kw)


class _Blocks(torch.nn.Module):
    """Maps with dropout, one dropout shared by all, checkpointed or not."""

    def __init__(self, n=3):
        super().__init__()
        self.maps = torch.nn.ModuleList(lay.Linear(6, 6, act="silu", p=0.3, seed=10 + i)
                                        for i in range(n))
        self.drop = lay.Dropout(0.4, seed=77)

    def block(self, i, x):
        return self.drop(self.maps[i](x, residual=x)) + torch.rand(())  # (draws of its own too)

    def forward(self, x, how):
        for i in range(len(self.maps)):
            if how == "plain":
                x = self.block(i, x)
            elif how == "nested":
                x = checkpoint(lambda v, i=i: checkpoint(self.block, i, v, use_reentrant=False),
                               x, use_reentrant=False)
            else:
                x = checkpoint(self.block, i, x, use_reentrant=how == "reentrant")
        return x


def _run(model, how, batches):
    """Outputs and gradients of several passes in flight at once."""
    torch.manual_seed(8)
    for m in [*model.maps, model.drop]:
        m.step = 0
    model.zero_grad()
    xs = [x.clone().requires_grad_() for x in batches]
    ys = [model(x, how) for x in xs]
    for y in reversed(ys):
        (y ** 2).sum().backward()
    return ([y.detach() for y in ys], [x.grad for x in xs]
            + [p.grad.clone() for p in model.parameters()], [m.step for m in model.maps],
            model.drop.step)


@pytest.mark.parametrize("how", ["reentrant", "non-reentrant", "nested"])
def test_a_repeated_forward_pass_draws_the_same_mask(how):
    model = _Blocks()
    batches = [torch.randn(20, 6) for _ in range(3)]
    y0, g0, s0, d0 = _run(model, "plain", batches)
    y1, g1, s1, d1 = _run(model, how, batches)
    assert all(torch.equal(a, b) for a, b in zip(y0, y1))
    for a, b in zip(g0, g1):
        assert torch.allclose(a, b, rtol=1e-6, atol=1e-6)
    assert s1 == s0 == [3, 3, 3] and d1 == d0 == 9  # repetitions do not count


def test_a_repetition_that_cannot_be_told_is_an_error():
    m, x = lay.Linear(6, 3, p=0.4, seed=1), torch.randn(50, 6, requires_grad=True)
    y = checkpoint(m, x, use_reentrant=False, preserve_rng_state=False)
    torch.rand(3)
    with pytest.raises(RuntimeError, match="preserve_rng_state"):
        y.tanh().sum().backward()


def test_step_repeats_a_run():
    m, x = lay.Dropout(0.4, seed=1), torch.ones(200)
    a = [m(x) for _ in range(3)]
    m.step = 0
    assert all(torch.equal(m(x), v) for v in a) and not torch.equal(a[0], a[1])


# ---- seeds -----------------------------------------------------------------
def test_modules_built_with_the_defaults_draw_masks_of_their_own():
    x = torch.ones(4000)
    ms = [lay.Dropout(0.5) for _ in range(4)]
    kept = torch.stack([m(x) != 0 for m in ms]).double()
    # independent masks agree in half of the elements (five standard errors)
    for i in range(4):
        for j in range(i):
            same = float((kept[i] == kept[j]).double().mean())
            assert abs(same - 0.5) < 5 * 0.5 / 4000 ** 0.5
    seeds = {lay.Linear(3, 3, p=0.1).seed for _ in range(50)} | {m.seed for m in ms}
    assert len(seeds) == 54 and all(0 <= s < 1 << 63 for s in seeds)


def test_a_given_seed_is_kept():
    assert [lay.Dropout(0.5, seed=s).seed for s in (0, 7)] == [0, 7]
    assert lay.Linear(3, 3, p=0.1, seed=5).seed == 5


def test_copies_of_a_module_draw_masks_of_their_own():
    block = torch.nn.Sequential(lay.Linear(3, 3, p=0.2), lay.Dropout(0.5))
    copies = [copy.deepcopy(block) for _ in range(3)]
    assert len({m.seed for b in [block, *copies] for m in b}) == 8
    assert torch.equal(copies[0][0].weight, block[0].weight)
    assert copies[0][0].weight is not block[0].weight
    given = lay.Dropout(0.5, seed=4)
    assert copy.deepcopy(given).seed == 4
    twice = copy.deepcopy(torch.nn.ModuleList([given, given]))  # one module stays one module
    assert twice[0] is twice[1]


# ---- state -----------------------------------------------------------------
def _net():
    return torch.nn.Sequential(lay.Linear(5, 5, p=0.3), lay.Dropout(0.4),
                               torch.nn.Sequential(lay.Linear(5, 5, p=0.2, seed=(1 << 64) - 3)))


def test_a_restored_run_goes_on_with_its_masks():
    x, a = torch.randn(30, 5), _net()
    for _ in range(3):
        a(x)
    b = _net()
    assert b[0].seed != a[0].seed
    b.load_state_dict(a.state_dict())
    assert [m.step for m in (b[0], b[1], b[2][0])] == [3, 3, 3]
    assert b[2][0].seed == (1 << 64) - 3
    assert torch.equal(a(x), b(x)) and torch.equal(a(x), b(x))


def test_states_without_masks_load_as_before():
    a = _net()
    for _ in range(2):
        a(torch.randn(3, 5))
    seed = a[0].seed
    plain = {k: v for k, v in a.state_dict().items() if k.endswith("weight")}
    a.load_state_dict(plain)  # as saved by modules that kept no masks
    assert a[0].seed == seed and a[0].step == 2
    # a map without dropout has the keys of torch.nn.Linear
    m = lay.Linear(5, 4, bias=True)
    torch.nn.Linear(5, 4).load_state_dict(m.state_dict())
    assert set(m.state_dict()) == {"weight", "bias"}
    with pytest.raises(RuntimeError, match="nexpected"):
        m.load_state_dict({**m.state_dict(), "mask": torch.zeros(2)})


# ---- memory ----------------------------------------------------------------
def test_nothing_of_a_pass_is_kept_after_its_backward_pass():
    m = lay.Linear(6, 3, act="silu")
    y = m(torch.randn(4, 6))
    kept = weakref.ref(m._last[0].untyped_storage())
    assert kept() is not None
    y.sum().backward()
    del y
    gc.collect()
    assert m._last is None and kept() is None
    # a later forward pass's is not the earlier one's to clear
    a, b = m(torch.randn(4, 6)), m(torch.randn(4, 6))
    a.sum().backward()
    assert m._last is not None
    b.sum().backward()
    assert m._last is None
    y = checkpoint(m, torch.randn(4, 6, requires_grad=True), use_reentrant=False)
    y.sum().backward()
    assert m._last is None


def test_modules_pickled_before_they_kept_passes_load():
    m = lay.Linear(5, 3, act="silu", p=0.2, seed=4)
    old = {k: v for k, v in m.__dict__.items() if k not in ("_passes", "_seed_given")}
    new = lay.Linear.__new__(lay.Linear)
    new.__setstate__(old)
    x = torch.randn(6, 5)
    assert torch.equal(new(x), m(x)) and copy.deepcopy(new).seed == 4
    again = pickle.loads(pickle.dumps(m))
    assert (again.seed, again.step) == (4, 1) and torch.equal(again(x), m(x))
