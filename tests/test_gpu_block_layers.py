"""The torch modules of a transformer block and the clipping step over them on the GPU: a
run of the operators as a model makes it, against torch's automatic differentiation in 64
bits and loops over the samples."""

import numpy as np
import pytest
import torch

import randomized_norm_clipping_gb300 as rnc
from oracle import block
from randomized_norm_clipping_gb300 import example_lm
from randomized_norm_clipping_gb300 import layers as lay
from randomized_norm_clipping_gb300.step import RandomizedClippingStep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _no_device_error():
    torch.manual_seed(5)
    yield
    torch.cuda.synchronize()
    assert rnc.dprc_device_error(reset=True) == 0


def _close(a, b, rtol):
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    assert torch.isfinite(a).all()
    assert (a - b).norm() <= rtol * b.norm(), ((a - b).norm() / b.norm()).item()


def _norm64(x, w):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * w


def _turn64(x, freqs):
    P = freqs.numel()
    angle = torch.arange(x.shape[1], device=x.device)[:, None].double() * freqs.to(x.device)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., :P], x[..., P:2 * P]
    return torch.cat((a * c - b * s, a * s + b * c, x[..., 2 * P:]), -1)


def _attend64(q, k, v, docs, cap):
    G = q.shape[2] // k.shape[2]
    T = q.shape[1]
    k, v = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    z = torch.einsum("bihd,bjhd->bhij", q, k) * q.shape[-1] ** -0.5
    z = cap * torch.tanh(z / cap)
    i = torch.arange(T, device=q.device)
    see = (i[:, None] >= i) & (docs[:, :, None] == docs[:, None])
    z = z.masked_fill(~see[:, None], -float("inf"))
    return torch.einsum("bhij,bjhd->bihd", torch.softmax(z, -1), v)


# bf16: some ten roundings (2^-8 at most each, 2^-9.2 in the mean square) one after another
# in a chain of six operators, whose gradients double them: 20 2^-9.2 = 3.4e-2 at the most.
# fp32: the sums of a chain of six, near 1e-6 each.
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-5), (torch.bfloat16, 3.4e-2)])
def test_a_block_of_operators(dtype, tol):
    """Normalisation, product, rotary positions, attention over packed documents, product."""
    B, T, W, H, Hkv, D = 2, 150, 64, 8, 2, 24
    norm = lay.LayerNorm(W, center=False, bias=False).to(DEV, dtype)
    rows = lay.Linear(W, (H + 2 * Hkv) * D).to(DEV, dtype)
    att = lay.Attention(H, Hkv, D, cap=8.0, freqs=lay.rotary_freqs(D // 2)).to(DEV, dtype)
    back = lay.Linear(H * D, W).to(DEV, dtype)
    with torch.no_grad():
        norm.weight.add_(0.1 * torch.randn_like(norm.weight))
    docs = torch.sort(torch.randint(0, 3, (B, T)), 1).values.int().to(DEV)
    x = torch.randn(B, T, W).to(DEV, dtype).requires_grad_()
    u = torch.randn(B, T, W).to(DEV, dtype)
    params = [norm.weight, rows.weight, back.weight]
    y = back(att(rows(norm(x)), docs=docs), residual=x)
    got = torch.autograd.grad((y * u).sum(), [x, *params])
    xd, wn, wr, wb = (t.detach().double().requires_grad_() for t in (x, *params))
    r = (_norm64(xd, wn) @ wr.t()).view(B, T, H + 2 * Hkv, D)
    qk = _turn64(r[:, :, :H + Hkv], att.freqs)
    o = _attend64(qk[:, :, :H], qk[:, :, H:], r[:, :, H + Hkv:], docs, 8.0)
    ref = xd + o.reshape(B, T, H * D) @ wb.t()
    _close(y, ref, tol)
    for a, b in zip(got, torch.autograd.grad((ref * u.double()).sum(), [xd, wn, wr, wb])):
        _close(a, b, tol)


def test_step_clips_a_model_with_attention():
    """Per-sample norms and the clipped sum against a loop over the samples (fp32)."""
    m = example_lm.TinyLM(vocab=40, width=32, hidden=32, blocks=2, p=0.0, dtype=torch.float32,
                          heads=4).to(DEV)
    with torch.no_grad():
        for mixer in m.mixers:
            mixer.norm.weight.add_(0.1 * torch.randn_like(mixer.norm.weight))
    tok = torch.randint(0, 40, (5, 33), device=DEV)
    f = lambda t: (m(t) ** 2).mean(dim=(1, 2))  # noqa: E731
    step = RandomizedClippingStep(m, C=1.0, sigma=0.0, k=32)
    params = step.parameters()
    per = [torch.autograd.grad(f(tok[i:i + 1]).sum(), params) for i in range(5)]
    n = np.array([sum(float((t.double() ** 2).sum()) for t in g) for g in per])
    step.C = C = float(np.median(np.sqrt(n)))
    c = np.minimum(1.0, C / np.sqrt(n))
    assert any(p is m.mixers[0].norm.weight for p in params)
    # (P = I gives the exact norms; the maps here are 32 to 64 wide)
    step.k = 64
    eye = [torch.nn.functional.pad(torch.eye(l.out_features, device=DEV),
                                   (0, 64 - l.out_features)) for l in step.layers]
    out = step(f(tok), step=0, projections=eye)
    assert np.allclose(out["n"].cpu().numpy(), n, rtol=1e-4)
    for j, p in enumerate(params):
        _close(p.grad, sum(c[i] * per[i][j].double() for i in range(5)), 1e-4)
    step.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_generation_over_a_cache(dtype):
    """Logits of single tokens over the cache against those of the whole pass."""
    m = example_lm.TinyLM(vocab=64, width=64, hidden=64, blocks=2, p=0.0, dtype=dtype,
                          heads=8).to(DEV).eval()
    tok = torch.randint(0, 64, (3, 20), device=DEV)
    with torch.no_grad():
        whole = m(tok)
        caches = [x.cache(3, 20, DEV) for x in m.mixers]
        at = torch.zeros(3, dtype=torch.int32, device=DEV)
        for a, b in ((0, 7), (7, 8), (8, 9), (9, 20)):
            x = m.embed(tok[:, a:b])
            for mixer, blk, cache in zip(m.mixers, m.blocks, caches):
                x = blk(mixer.extend(x, cache, at))
            at = at + (b - a)
            # the same roundings but those of weights in another order of tiles
            _close(m.head(m.norm(x)), whole[:, a:b], 1e-5 if dtype is torch.float32 else 3e-2)
    assert m.generate(tok, 4).shape == (3, 4)


def test_example_with_heads_runs():
    loss = example_lm.train(steps=3, B=4, T=40, heads=4)
    assert all(np.isfinite(loss))


# ---- captured, replayed, side by side -------------------------------------------
def _calls(dtype, seed):
    """Calls that need workspaces of every kind, and their outputs."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)  # noqa: E731
    B, T, H, Hkv, D = 2, 300, 4, 2, 64
    q, k, v, do = r(B, T, H, D), r(B, T, Hkv, D), r(B, T, Hkv, D), r(B, T, H, D)
    q1, k1 = r(B, 1, H, D), r(B, 3000, Hkv, D)
    docs = torch.sort(torch.randint(0, 3, (B, T), device=DEV, generator=g), 1).values.int()
    x, w = r(B, T, 128), r(128)
    stats, n = torch.empty(B, T, 2, device=DEV), torch.empty(B, device=DEV)
    lse = torch.empty(B, H, T, device=DEV)
    outs = [torch.empty_like(t) for t in (q, q, k, v, q1, x, x, w)]
    pos = torch.arange(T, device=DEV).expand(B, T).contiguous()
    freqs = lay.rotary_freqs(32).to(DEV)
    turned = torch.empty_like(q)

    def run():
        rnc.dprc_rotary(q, pos, freqs, out=turned)
        rnc.dprc_attention(turned, k, v, docs=docs, out=outs[0], lse=lse)
        rnc.dprc_attention_grad(do, turned, k, v, outs[0], lse, docs=docs, dQ=outs[1], dK=outs[2],
                                dV=outs[3])
        rnc.dprc_attention(q1, k1, k1, out=outs[4])
        rnc.dprc_layernorm(x, w, stats=stats, out=outs[5])
        rnc.dprc_layernorm_grad(outs[5], x, stats, w, dX=outs[6], dW=outs[7], n=n)

    return run, outs + [lse, n, turned]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_calls_and_streams(dtype):
    calls = [_calls(dtype, s) for s in range(2)]
    want = []
    for run, outs in calls:
        run()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.zero_()
    # two graphs, replayed side by side on streams of their own
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for (run, _), s in zip(calls, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run()
        graphs.append(graph)
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, outs), ref in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):  # and as calls on two streams
        for (run, _), s in zip(calls, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for (_, outs), ref in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_training_pass_captured_beside_an_eager_graph():
    """A forward and backward pass captured while an eager pass's graph lives."""
    att = lay.Attention(4, 2, 64, freqs=lay.rotary_freqs(32)).to(DEV)
    norm = lay.LayerNorm(512).to(DEV)
    x = torch.randn(2, 100, 512, device=DEV, requires_grad=True)
    eager = att(norm(x))
    (want,) = torch.autograd.grad(eager.square().sum(), x, retain_graph=True)
    pos = att.positions(2, 100, DEV)
    x2 = x.detach().clone().requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.autograd.grad(att(norm(x2), positions=pos).square().sum(), x2)  # (warm)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (got,) = torch.autograd.grad(att(norm(x2), positions=pos).square().sum(), x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(torch.autograd.grad(eager.square().sum(), x)[0], want)


def test_given_stream_and_workspace():
    q = torch.randn(1, 1, 4, 64, device=DEV).bfloat16()
    k = torch.randn(1, 4000, 2, 64, device=DEV).bfloat16()
    want = rnc.dprc_attention(q, k, k)
    ref, _ = block.attention(*(t.double().cpu().numpy() for t in (q, k, k)))
    assert np.abs(want.double().cpu().numpy() - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    assert torch.equal(rnc.dprc_attention(q, k, k, stream=s).cpu(), want.cpu())
    ws = torch.full((8 << 20,), 255, dtype=torch.uint8, device=DEV)  # (needs no zeroing)
    assert torch.equal(rnc.dprc_attention(q, k, k, ws=ws), want)
    with pytest.raises(rnc.DprcError):
        rnc.dprc_attention(q, k, k, ws=ws[:16])
