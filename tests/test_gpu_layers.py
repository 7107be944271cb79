"""The torch modules over the operators (randomized_norm_clipping_gb300.layers)
and the clipping step over models made of them.

The references are plain torch modules of the same arithmetic in float64, or a
loop over the samples; dropout masks come from the oracle.
"""

import numpy as np
import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from oracle import operators as ops
from randomized_norm_clipping_gb300 import layers as lay
from randomized_norm_clipping_gb300.example_lm import train
from randomized_norm_clipping_gb300.step import RandomizedClippingStep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _close(a, b, rtol):
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    assert (a - b).norm() <= rtol * b.norm(), ((a - b).norm() / b.norm()).item()


# fp32 through one layer: sums of some hundred products, rounded at 2^-23 each
F32 = 2e-6


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_linear_module_gradients(act, p):
    torch.manual_seed(1)
    m = lay.Linear(72, 56, bias=True, act=act, p=p, seed=11).to(DEV)
    with torch.no_grad():
        m.bias.normal_()
    x = torch.randn(3, 40, 72, device=DEV, requires_grad=True)
    r = torch.randn(3, 40, 56, device=DEV, requires_grad=True)
    dy = torch.randn(3, 40, 56, device=DEV)
    y = m(x, residual=r)
    y.backward(dy)
    assert m.step == (1 if p else 0)
    xd, wd, bd, rd = (t.detach().double().requires_grad_() for t in (x, m.weight, m.bias, r))
    z = xd @ wd.t() + bd
    f = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act]
    h = f(z)
    if p:
        keep = ops.dropout_factor(3 * 40 * 56, p, 11, 1).reshape(3, 40, 56)
        h = h * torch.from_numpy(keep).to(DEV)
    ref = h + rd
    ref.backward(dy.double())
    _close(y, ref, F32)
    for a, b in ((x.grad, xd.grad), (m.weight.grad, wd.grad), (m.bias.grad, bd.grad),
                 (r.grad, rd.grad)):
        _close(a, b, F32)
    m.eval()
    _close(m(x, residual=r), f(z) + rd, F32)  # no dropout outside training


def test_backward_twice_draws_the_same_mask():
    m = lay.Dropout(0.4, seed=5).to(DEV)
    x = torch.randn(1000, device=DEV, requires_grad=True)
    y = m(x)
    g1 = torch.autograd.grad(y.sum(), x, retain_graph=True)[0]
    g2 = torch.autograd.grad(y.sum(), x)[0]
    keep = torch.from_numpy(ops.dropout_factor(1000, 0.4, 5, 1)).to(DEV)
    assert torch.equal(g1, g2)
    _close(g1, keep, 1e-7)
    _close(y, x.detach().double() * keep, 1e-6)
    assert not torch.equal(m(x) == 0, y == 0)  # the next pass, another mask


def test_embedding_module_gradient():
    m = lay.Embedding(50, 24, scale=1.5).to(DEV)
    tok = torch.randint(-1, 50, (4, 37), device=DEV)
    out = m(tok)
    dy = torch.randn_like(out)
    out.backward(dy)
    w = m.weight.detach().cpu().numpy()
    assert np.allclose(out.detach().cpu().numpy(), ops.embed_lookup(w, tok.cpu().numpy(), 1.5),
                       rtol=1e-6)
    ref = ops.embed_grad(dy.cpu().double().numpy(), tok.cpu().numpy(), 50, None, 1.5)
    assert np.allclose(m.weight.grad.cpu().numpy(), ref, atol=1e-5)


def test_views_and_odd_offsets():
    m = lay.Linear(24, 16).to(DEV)
    base = torch.randn(9, 25, device=DEV)
    x = base[:, 1:]  # not contiguous
    _close(m(x), x.double() @ m.weight.double().t(), F32)
    y = torch.randn(24 * 5 + 1, device=DEV)[1:].view(5, 24)  # contiguous, 4 bytes off
    _close(m(y), y.double() @ m.weight.double().t(), F32)
    e = lay.Embedding(7, 8).to(DEV)
    tok = torch.randint(0, 7, (13,), device=DEV)[1:]
    assert torch.equal(e(tok), e.weight[tok])


class _Model(torch.nn.Module):
    """Embedding, a fused map with bias and activation, a residual map, a head."""

    def __init__(self, embedding):
        super().__init__()
        self.embed = embedding
        self.up = lay.Linear(32, 64, bias=True, act="silu")
        self.down = lay.Linear(64, 32, bias=True)
        self.head = torch.nn.Linear(32, 32, bias=False)
        with torch.no_grad():
            self.up.bias.normal_()

    def forward(self, tok):
        x = self.embed(tok)
        return self.head(self.down(self.up(x), residual=x))


def _losses(model, tok):
    return (model(tok).float() ** 2).mean(dim=(1, 2))


@pytest.mark.parametrize("kind", ["library", "torch", "torch padded"])
def test_step_reproduces_per_sample_clipping(kind):
    # with P = I for every linear weight, and exact norms of the rest, the step
    # is per-sample clipping of all parameters, here computed by a loop
    torch.manual_seed(7)
    emb = (lay.Embedding(40, 32, scale=2.0) if kind == "library"
           else torch.nn.Embedding(40, 32, padding_idx=3 if "padded" in kind else None))
    model = _Model(emb).to(DEV)
    tok = torch.randint(0, 40, (5, 30), device=DEV)
    tok[:, 20:] = tok[:, :10]  # repeated tokens: sums before squares
    tok[1, 5:15] = 3
    step = RandomizedClippingStep(model, C=1.0, sigma=0.0, k=64)
    params = step.parameters()
    assert len(params) == len(list(model.parameters()))
    norms, grads = [], []
    for i in range(5):
        g = torch.autograd.grad(_losses(model, tok[i:i + 1]).sum(), params)
        norms.append(sum(float((t.double() ** 2).sum()) for t in g))
        grads.append([t.double() for t in g])
    n_ref = np.array(norms)
    step.C = C = float(np.median(np.sqrt(n_ref)))
    c_ref = np.minimum(1.0, C / np.sqrt(n_ref))
    eye = [torch.eye(m.out_features, device=DEV) for m in step.layers]
    out = step(_losses(model, tok), step=0, projections=eye)
    # three layers of fp32 sums on either side
    assert np.allclose(out["n"].cpu().numpy(), n_ref, rtol=1e-4)
    assert np.allclose(out["c"].cpu().numpy(), c_ref, rtol=1e-4)
    for j, prm in enumerate(params):
        ref = sum(c_ref[i] * grads[i][j] for i in range(5))
        _close(prm.grad, ref, 1e-4)
    step.close()


def test_step_with_dropout_uses_one_mask_throughout():
    # the recorded norms must be those of the masked forward pass: compare with
    # automatic differentiation of the same pass, sample by sample
    torch.manual_seed(8)
    model = _Model(lay.Embedding(40, 32)).to(DEV)
    model.down.p, model.down.seed = 0.3, 77
    tok = torch.randint(0, 40, (4, 25), device=DEV)
    step = RandomizedClippingStep(model, C=1e9, sigma=0.0, k=64)  # nothing clips
    losses = _losses(model, tok)
    params = step.parameters()
    per = [torch.autograd.grad(losses[i], params, retain_graph=True) for i in range(4)]
    n_ref = [sum(float((t.double() ** 2).sum()) for t in g) for g in per]
    eye = [torch.eye(m.out_features, device=DEV) for m in step.layers]
    out = step(losses, step=0, projections=eye)
    assert np.allclose(out["n"].cpu().numpy(), n_ref, rtol=1e-4)
    for j, prm in enumerate(params):
        _close(prm.grad, sum(g[j].double() for g in per), 1e-4)
    step.close()


@pytest.mark.parametrize("method", ["hutch", "hutchpp"])
def test_noise_covers_every_parameter(method):
    model = _Model(lay.Embedding(40, 32)).to(DEV)
    tok = torch.randint(0, 40, (3, 16), device=DEV)
    k = 16
    grads = {}
    for sigma in (0.0, 2.0):
        step = RandomizedClippingStep(model, C=0.5, sigma=sigma, k=k, method=method, seed=3)
        step(_losses(model, tok), step=4)
        grads[sigma] = torch.cat([p.grad.reshape(-1) for p in step.parameters()])
        step.close()
    z = (grads[2.0] - grads[0.0]).double() / (2.0 * 0.5)
    n = z.numel()
    assert abs(float(z.mean())) < 5 / n ** 0.5 and abs(float(z.var()) - 1) < 5 * (2 / n) ** 0.5


def test_step_refuses_what_it_cannot_norm():
    emb = lay.Embedding(10, 8)
    head = torch.nn.Linear(8, 10, bias=False)
    head.weight = emb.weight
    with pytest.raises(ValueError, match="shared"):
        RandomizedClippingStep(torch.nn.Sequential(emb, head), C=1.0, sigma=0.0)
    with pytest.raises(ValueError, match="sparse"):
        RandomizedClippingStep(torch.nn.Sequential(torch.nn.Embedding(10, 8, sparse=True)),
                               C=1.0, sigma=0.0)
    with pytest.raises(ValueError):
        RandomizedClippingStep(torch.nn.Sequential(emb, torch.nn.LayerNorm(8)), C=1.0, sigma=0.0)
    with pytest.raises(ValueError):
        lay.Linear(8, 8, act="tanh")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_example_model_learns(dtype):
    loss = train(steps=40, dtype=dtype)
    assert all(np.isfinite(loss))
    # a uniform guess over 256 tokens has loss ln 256 = 5.55
    assert np.mean(loss[-5:]) < np.mean(loss[:3]) - 1.0, (loss[:3], loss[-5:])


def test_embedding_only_model():
    emb = lay.Embedding(20, 16).to(DEV)
    tok = torch.tensor([[1, 1, 2], [3, 4, 5]], device=DEV)
    step = RandomizedClippingStep(emb, C=1.0, sigma=0.0)
    losses = emb(tok).sum(dim=(1, 2))
    out = step(losses, step=0)
    assert np.allclose(out["n"].cpu().numpy(), [5 * 16, 3 * 16])
    c = out["c"].cpu().numpy()
    assert np.allclose(emb.weight.grad[1].cpu().numpy(), 2 * c[0], rtol=1e-6)
    assert rnc.dprc_device_error(reset=True) == 0
    step.close()
