"""The clipping step without a GPU (the library's calls from the oracle): which
models it may take, so that every sample's contribution is bounded."""

import numpy as np
import pytest
import torch

import host_library
from randomized_norm_clipping_gb300 import layers as lay
from randomized_norm_clipping_gb300.step import RandomizedClippingStep

B, T, D = 4, 8, 6


@pytest.fixture(autouse=True)
def _host(monkeypatch):
    host_library.install(monkeypatch)
    torch.manual_seed(3)


def _embedding(kind, n=10, d=D):
    return lay.Embedding(n, d) if kind == "library" else torch.nn.Embedding(n, d)


class _Positions(torch.nn.Module):
    """Tokens plus positions, the positions' ids as `ids` makes them."""

    def __init__(self, kind, ids, t=T):
        super().__init__()
        self.tok, self.pos = _embedding(kind), _embedding(kind, t)
        self.head = torch.nn.Linear(D, D, bias=False)
        self.ids = ids

    def forward(self, tok):
        return self.head(self.tok(tok) + self.pos(self.ids(tok)))


def _losses(model, tok):
    return (model(tok) ** 2).mean(dim=(1, 2))


def _reference(losses_of, params, n, C):
    """Norms and the clipped sum by a loop over the samples."""
    norms, grads = [], []
    for i in range(n):
        g = torch.autograd.grad(losses_of(i), params)
        norms.append(sum(float((t.double() ** 2).sum()) for t in g))
        grads.append(g)
    c = np.minimum(1.0, C / np.sqrt(norms))
    return np.array(norms), [sum(c[i] * grads[i][j] for i in range(n)) for j in range(len(params))]


def _check(model, losses, losses_of, n=B, C=0.3):
    step = RandomizedClippingStep(model, C=C, sigma=0.0, k=D)
    params = step.parameters()
    norms, total = _reference(losses_of, params, n, C)
    eye = [torch.eye(m.out_features) for m in step.layers]
    out = step(losses(), step=0, projections=eye)
    assert np.allclose(out["n"].numpy(), norms, rtol=1e-4)
    for prm, ref in zip(params, total):
        assert torch.allclose(prm.grad, ref, rtol=1e-4, atol=1e-6)
    out = step(losses(), step=1, projections=eye)  # what was looked at once is taken at once
    assert np.allclose(out["n"].numpy(), norms, rtol=1e-4)
    step.close()


@pytest.mark.parametrize("kind", ["library", "torch"])
@pytest.mark.parametrize("t", [T, T + 1, B])
@pytest.mark.parametrize("shape", ["T", "1 T"])
def test_positions_shared_by_the_batch_are_refused(kind, t, shape):
    ids = {"T": lambda tok: torch.arange(t), "1 T": lambda tok: torch.arange(t)[None]}[shape]
    model = _Positions(kind, ids, t)
    tok = torch.randint(0, 10, (B, t))
    step = RandomizedClippingStep(model, C=1.0, sigma=0.0, k=D)
    with pytest.raises(ValueError, match="sample"):
        step(_losses(model, tok), step=0)
    step.close()


@pytest.mark.parametrize("kind", ["library", "torch"])
def test_positions_of_every_sample_are_taken(kind):
    model = _Positions(kind, lambda tok: torch.arange(T).expand(tok.shape[0], T))
    tok = torch.randint(0, 10, (B, T))
    _check(model, lambda: _losses(model, tok), lambda i: _losses(model, tok[i:i + 1]).sum())


@pytest.mark.parametrize("shape", ["T", "1 T"])
def test_one_sample_owns_every_position(shape):
    ids = {"T": lambda tok: torch.arange(T), "1 T": lambda tok: torch.arange(T)[None]}[shape]
    model = _Positions("library", ids)
    tok = torch.randint(0, 10, (1, T))
    _check(model, lambda: _losses(model, tok), lambda i: _losses(model, tok).sum(), n=1)


class _Rows(torch.nn.Module):
    """Works on rows (batch and positions in one axis)."""

    def __init__(self, major):
        super().__init__()
        self.embed, self.up = lay.Embedding(10, D), lay.Linear(D, D, bias=True, act="silu")
        self.head = torch.nn.Linear(D, D, bias=False)
        self.major = major

    def forward(self, tok):
        n, t = tok.shape
        if self.major == "sample":
            return self.head(self.up(self.embed(tok.reshape(-1)))).view(n, t, D)
        return self.head(self.up(self.embed(tok.t().reshape(-1)))).view(t, n, D).transpose(0, 1)


def test_rows_of_one_sample_after_another_are_taken():
    model, tok = _Rows("sample"), torch.randint(0, 10, (B, T))
    _check(model, lambda: _losses(model, tok), lambda i: _losses(model, tok[i:i + 1]).sum())


def test_rows_of_mixed_samples_are_refused():
    model, tok = _Rows("position"), torch.randint(0, 10, (B, T))
    step = RandomizedClippingStep(model, C=1.0, sigma=0.0, k=D)
    with pytest.raises(ValueError, match="sample"):
        step(_losses(model, tok), step=0)
    step.close()


@pytest.mark.parametrize("shape", [(T, D), (1, T, D), (2, T, D)])
def test_linear_maps_of_shared_inputs_are_refused(shape):
    class Shared(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.side = torch.nn.Linear(D, D, bias=False)
            self.main = torch.nn.Linear(D, D, bias=False)
            self.register_buffer("table", torch.randn(shape))

        def forward(self, x):
            return self.main(x) + self.side(self.table).reshape(-1, T, D)[:1]

    model, x = Shared(), torch.randn(B, T, D)
    step = RandomizedClippingStep(model, C=1.0, sigma=0.0, k=D)
    with pytest.raises(ValueError, match="sample"):
        step((model(x) ** 2).mean(dim=(1, 2)), step=0)
    step.close()


def test_one_token_a_sample_is_taken():
    class Classes(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.embed, self.head = _embedding("torch"), torch.nn.Linear(D, D, bias=False)

        def forward(self, y):
            return self.head(self.embed(y))[:, None]

    model, y = Classes(), torch.randint(0, 10, (B,))
    _check(model, lambda: _losses(model, y), lambda i: _losses(model, y[i:i + 1]).sum())


class _Twice(torch.nn.Module):
    def __init__(self, which):
        super().__init__()
        self.embed = lay.Embedding(10, D)
        self.a = torch.nn.Linear(D, D, bias=False) if which == "torch" else lay.Linear(D, D)
        self.which = which

    def forward(self, tok):
        x = self.embed(tok)
        if self.which == "embedding":
            x = x + self.embed(tok.flip(1))
        x = self.a(x)
        return x if self.which == "embedding" else self.a(torch.tanh(x))


@pytest.mark.parametrize("which", ["embedding", "library", "torch"])
def test_a_layer_used_twice_is_refused(which):
    model, tok = _Twice(which), torch.randint(0, 10, (B, T))
    step = RandomizedClippingStep(model, C=1.0, sigma=0.0, k=D)
    with pytest.raises(ValueError, match="more than once"):
        step(_losses(model, tok), step=0)
    step.close()


@pytest.mark.parametrize("kind", ["library", "torch"])
def test_an_earlier_forward_pass_does_not_count(kind):
    model = _Positions(kind, lambda tok: torch.arange(T).expand(tok.shape[0], T))
    tok = torch.randint(0, 10, (B, T))
    kept = []

    def losses():
        kept.append(_losses(model, tok))  # looked at, with its graph, and not stepped on
        return _losses(model, tok)

    _check(model, losses, lambda i: _losses(model, tok[i:i + 1]).sum())


def test_checkpointed_blocks_step_as_others():
    """A block that is repeated in each of the step's backward passes, with dropout."""
    import os
    os.environ["TRITON_INTERPRET"] = "1"  # (checkpoint imports triton: tests/test_oracle.py)
    from torch.utils.checkpoint import checkpoint

    class Model(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.embed = lay.Embedding(10, D)
            self.up = lay.Linear(D, D, bias=True, act="gelu", p=0.3, seed=5)
            self.drop = lay.Dropout(0.2, seed=6)
            self.head = torch.nn.Linear(D, D, bias=False)
            self.repeat = False

        def block(self, x):
            return self.drop(self.up(x), residual=x)

        def forward(self, tok):
            x = self.embed(tok)
            x = checkpoint(self.block, x, use_reentrant=False) if self.repeat else self.block(x)
            return self.head(x)

    model, tok = Model(), torch.randint(0, 10, (B, T))
    step = RandomizedClippingStep(model, C=0.05, sigma=0.0, k=D)
    eye = [torch.eye(m.out_features) for m in step.layers]
    got = []
    for repeat in (False, True):
        model.repeat, model.up.step, model.drop.step = repeat, 0, 0
        out = step(_losses(model, tok), step=0, projections=eye)
        got.append([out["n"], out["c"]] + [p.grad.clone() for p in step.parameters()])
        assert model.up.step == model.drop.step == 1
    step.close()
    for a, b in zip(*got):
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-7)


def test_bias_plans_are_made_once_a_size(monkeypatch):
    class TwoLengths(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.a, self.b = lay.Linear(D, D, bias=True), lay.Linear(D, D, bias=True)

        def forward(self, x):
            return self.b(self.a(x)[:, ::2])

    made = []
    plan = host_library.embed_plan
    monkeypatch.setattr(host_library.binding, "dprc_embed_plan",
                        lambda tok, V, **kw: (made.append(tuple(tok.shape)), plan(tok, V))[1])
    model = TwoLengths()
    step = RandomizedClippingStep(model, C=1.0, sigma=0.0, k=D)
    for b in (B, B, B + 1, B):
        step(_losses(model, torch.randn(b, T, D)), step=0)
    assert sorted(made) == [(B, T // 2), (B, T), (B + 1, T // 2), (B + 1, T)]
    for b in range(1, 60):
        step(_losses(model, torch.randn(b, T, D)), step=0)
    assert len(step._bias_plans) <= 16  # sizes come and go
    step.close()


def test_the_refusal_names_what_is_covered():
    model = torch.nn.Sequential(lay.Embedding(5, D), torch.nn.LayerNorm(D))
    with pytest.raises(ValueError, match="'1.weight'.*linear weights.*layers.Linear.*embeddings"):
        RandomizedClippingStep(model, C=1.0, sigma=0.0)


def test_packed_samples_are_taken():
    """All samples' positions behind a leading axis of one, sample after sample."""
    class Packed(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.embed, self.up = lay.Embedding(10, D), lay.Linear(D, D, bias=True, act="silu")
            self.head = torch.nn.Linear(D, D, bias=False)

        def forward(self, tok):
            n, t = tok.shape
            return self.head(self.up(self.embed(tok.reshape(1, n * t)))).view(n, t, D)

    model, tok = Packed(), torch.randint(0, 10, (B, T))
    _check(model, lambda: _losses(model, tok), lambda i: _losses(model, tok[i:i + 1]).sum())
