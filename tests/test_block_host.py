"""Normalisation, rotary positions and attention without a GPU: the float64 oracle pinned to
loops, automatic differentiation and planted mistakes; the C entry points' and the
binding's refusals (no kernel runs); the torch modules and the clipping step over them
with the library's calls from the oracle."""

import copy
import ctypes
import math

import numpy as np
import pytest
import torch

import block_library
from oracle import block
from randomized_norm_clipping_gb300 import binding, example_lm
from randomized_norm_clipping_gb300 import layers as lay
from randomized_norm_clipping_gb300.step import RandomizedClippingStep


def _rng(seed):
    return np.random.default_rng(seed)


# ---- the oracle --------------------------------------------------------------
def _loops(Q, K, V, causal, cap, slopes, docs, prefix, lengths, first):
    """Attention pair by pair."""
    B, Tq, H, D = Q.shape
    Tk, Hkv = K.shape[1:3]
    out = np.zeros(Q.shape)
    for b in range(B):
        for h in range(H):
            for t in range(Tq):
                i = (Tk - Tq if first is None else first[b]) + t
                w, total = [], 0.0
                for j in range(Tk if lengths is None else lengths[b]):
                    if causal and not (j <= i or (prefix is not None and j < prefix[b])):
                        continue
                    if docs is not None and (not 0 <= i < Tk or docs[b][i] < 0
                                             or docs[b][i] != docs[b][j]):
                        continue
                    s = float(Q[b, t, h] @ K[b, j, h // (H // Hkv)]) / math.sqrt(D)
                    if cap:
                        s = cap * math.tanh(s / cap)
                    if slopes is not None:
                        s -= slopes[h] * abs(i - j)
                    w.append((math.exp(s), j))
                    total += w[-1][0]
                for e, j in w:
                    out[b, t, h] += e / total * V[b, j, h // (H // Hkv)]
    return out


MASKS = [dict(), dict(causal=False), dict(prefix=np.array([3, 0])), dict(lengths=np.array([4, 0])),
         dict(docs=np.array([[0, 0, 1, 1, 1, -1, 1], [5, 5, -1, 5, 2, 2, -1]])),
         dict(docs=np.array([[0, 0, 1, 1, 1, -1, 1], [5, 5, -1, 5, 2, 2, -1]]), causal=False),
         dict(first=np.array([-2, 9])), dict(lengths=np.array([5, 7]), first=np.array([1, 3]))]


@pytest.mark.parametrize("k", range(len(MASKS)))
@pytest.mark.parametrize("cap,bias", [(0.0, False), (2.0, True)])
@pytest.mark.parametrize("Tq", [7, 3])
def test_attention_oracle_matches_loops(k, cap, bias, Tq):
    r = _rng(k)
    Q, K, V = r.standard_normal((2, Tq, 4, 5)), r.standard_normal((2, 7, 2, 5)), r.standard_normal((2, 7, 2, 5))
    slopes = np.array([0.5, 0.25, 0.1, 0.0]) if bias else None
    m = dict(causal=True, docs=None, prefix=None, lengths=None, first=None)
    m.update(MASKS[k])
    out, lse = block.attention(Q, K, V, None, m["causal"], cap, slopes, m["docs"], m["prefix"],
                               m["lengths"], m["first"])
    assert np.allclose(out, _loops(Q, K, V, m["causal"], cap, slopes, m["docs"], m["prefix"],
                                   m["lengths"], m["first"]), atol=1e-12)
    assert ((out == 0).all(-1) == np.isinf(lse).transpose(0, 2, 1)).all()


@pytest.mark.parametrize("mistake", ["cap after the mask's scale", "no group", "border", "none"])
def test_planted_attention_mistakes_are_caught(mistake):
    r = _rng(9)
    Q, K, V = r.standard_normal((1, 6, 4, 8)), r.standard_normal((1, 6, 2, 8)), r.standard_normal((1, 6, 2, 8))
    good = _loops(Q, K, V, True, 1.0, None, None, None, None, None)
    if mistake == "no group":  # heads taken in turn instead of by groups
        bad = block.attention(Q[:, :, [0, 2, 1, 3]], K, V, cap=1.0)[0][:, :, [0, 2, 1, 3]]
    elif mistake == "border":
        bad = block.attention(Q, K, V, cap=1.0, first=np.array([1]))[0]
    elif mistake == "none":
        bad = block.attention(Q, K, V, cap=1.0)[0]
    else:
        bad = block.attention(Q, K, V, scale=1.0, cap=1.0)[0]
    assert np.allclose(bad, good, atol=1e-12) == (mistake == "none")


@pytest.mark.parametrize("k", range(len(MASKS)))
def test_attention_gradient_matches_autograd(k):
    """torch's automatic differentiation of elementary operations in 64 bits."""
    r = _rng(20 + k)
    m = MASKS[k]
    Q, K, V, dO = (torch.tensor(r.standard_normal((2, 7, h, 5)), requires_grad=h != 0) for h in (4, 2, 2, 4))
    see = np.stack([block.sees(b, 7, 7, **{"causal": True, **m})[0] for b in range(2)])
    pos = np.stack([block.sees(b, 7, 7, **{"causal": True, **m})[1] for b in range(2)])
    slopes = np.array([0.5, 0.25, 0.1, 0.0])
    z = torch.einsum("bihd,bjhd->bhij", Q, K.repeat_interleave(2, 2)) * 5 ** -0.5
    z = 2.0 * torch.tanh(z / 2.0)
    z = z - torch.tensor(slopes)[None, :, None, None] * torch.tensor(
        np.abs(pos[:, None, :, None] - np.arange(7)))
    e = torch.exp(z) * torch.tensor(see)[:, None]
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    out = torch.einsum("bhij,bjhd->bihd", p, V.repeat_interleave(2, 2))
    g = torch.autograd.grad((out * dO.detach()).sum(), (Q, K, V))
    got = block.attention(*(x.detach().numpy() for x in (Q, K, V)), cap=2.0, slopes=slopes,
                          dO=dO.detach().numpy(), **m)
    assert np.allclose(got[0], out.detach().numpy(), atol=1e-12)
    for a, b in zip(got[2:5], g):
        assert np.allclose(a, b.numpy(), atol=1e-11)


@pytest.mark.parametrize("center", [True, False])
def test_layernorm_gradient_matches_autograd(center):
    r = _rng(5)
    X, dY = r.standard_normal((3, 4, 6)) + 1.0, r.standard_normal((3, 4, 6))
    w, b = r.standard_normal(6), r.standard_normal(6)
    x, tw, tb = (torch.tensor(v, requires_grad=True) for v in (X, w, b))
    mu = x.mean(-1, keepdim=True) if center else 0.0
    y = (x - mu) / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + 1e-5) * tw + tb
    assert np.allclose(block.layernorm(X, w, b, 1e-5, center)[0], y.detach().numpy(), atol=1e-12)
    dX, W, bs = block.layernorm_grad(dY, X, w, 1e-5, center)
    g = torch.autograd.grad((y * torch.tensor(dY)).sum(), (x, tw, tb), retain_graph=True)
    for u, v in zip((dX, W.sum(0), bs.sum(0)), g):
        assert np.allclose(u, v.numpy(), atol=1e-11)
    for i in range(3):  # by sample
        gi = torch.autograd.grad((y[i] * torch.tensor(dY[i])).sum(), tw, retain_graph=True)[0]
        assert np.allclose(W[i], gi.numpy(), atol=1e-11)


def test_rotary_keeps_lengths_and_turns_back():
    r = _rng(6)
    X, pos = r.standard_normal((2, 3, 2, 10)), r.integers(-50, 50, (2, 3, 2))
    f = r.uniform(0.01, 1.0, 4)
    for inter in (False, True):
        y = block.rotary(X, pos, f, [1, 3], inter)
        assert np.allclose((y ** 2).sum(-1), (X ** 2).sum(-1)) and (y[..., 8:] == X[..., 8:]).all()
        assert np.allclose(block.rotary(y, pos, f, [1, 3], inter, inverse=True), X)
    # a product of two turned rows goes by the difference of their positions
    q, k = r.standard_normal((1, 1, 1, 8)), r.standard_normal((1, 1, 1, 8))
    at = lambda x, p: block.rotary(x, np.array([[p]]), f)  # noqa: E731
    assert np.allclose((at(q, 7) * at(k, 3)).sum(), (at(q, 107) * at(k, 103)).sum())


# ---- refusals ------------------------------------------------------------------
A16 = 0x10000  # an aligned address that nothing reads: the calls fail their checks first


@pytest.fixture(scope="module")
def lib():
    import os
    from randomized_norm_clipping_gb300 import build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding.lib()


def _strides(*v):
    return (ctypes.c_int64 * 3)(*v)


class Args(ctypes.Structure):
    """dprc_attention_args."""
    _fields_ = [(n, ctypes.c_void_p) for n in "QKV"] + [
        (n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "v_stride")] + [
        ("dtype", ctypes.c_int)] + [(n, ctypes.c_int64) for n in ("B", "Tq", "Tk", "H", "Hkv", "D")] + [
        ("scale", ctypes.c_float), ("cap", ctypes.c_float), ("causal", ctypes.c_int)] + [
        (n, ctypes.c_void_p) for n in ("slopes", "docs", "prefix", "lengths", "first")]


def test_packed_arguments_are_the_structure():
    a = _args()
    packed = binding._ATTENTION_ARGS.pack(A16, A16, A16, 1 << 20, 256, 64, 1 << 20, 128, 64, 1 << 20,
                                          128, 64, 1, 2, 100, 100, 4, 2, 64, 0.125, 0.0, 1, 0, 0, 0,
                                          0, 0)
    assert packed == bytes(a)


def _args(**kw):
    a = Args(A16, A16, A16, _strides(1 << 20, 256, 64), _strides(1 << 20, 128, 64),
                               _strides(1 << 20, 128, 64), 1, 2, 100, 100, 4, 2, 64, 0.125, 0.0, 1,
                               None, None, None, None, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


ATTENTION_REFUSALS = [
    (dict(Q=None), 1), (dict(K=None), 1), (dict(dtype=5), 3), (dict(B=0), 2), (dict(Tq=-1), 2),
    (dict(Tk=(1 << 20) + 1), 2), (dict(H=5), 2), (dict(Hkv=0), 2), (dict(D=0), 2), (dict(D=129), 2),
    (dict(B=65535), 2), (dict(scale=float("inf")), 2), (dict(cap=-1.0), 2),
    (dict(cap=float("nan")), 2), (dict(q_stride=_strides(1, -1, 1)), 2),
    (dict(K=A16 + 1), 4), (dict(docs=A16 + 2), 4), (dict(lengths=A16 + 1), 4)]


@pytest.mark.parametrize("change,status", ATTENTION_REFUSALS, ids=lambda v: str(v)[:30])
def test_attention_refusals(lib, change, status):
    a = _args(**change)
    s = _strides(1 << 20, 256, 64)
    assert lib.dprc_attention(ctypes.byref(a), A16, None, A16, 1 << 40, None) == status
    assert lib.dprc_attention_grad(ctypes.byref(a), A16, s, A16, s, A16, A16, s, A16, s, A16, s, A16,
                                   1 << 40, None) == status
    if status in (2, 3):
        assert lib.dprc_attention_workspace_bytes(ctypes.byref(a), 0) == 0


def test_attention_call_refusals(lib):
    a, s = _args(), _strides(1 << 20, 256, 64)
    need = lib.dprc_attention_workspace_bytes(ctypes.byref(a), 0)
    grad = lib.dprc_attention_workspace_bytes(ctypes.byref(a), 1)
    assert grad >= 2 * 4 * 100 * 4
    f, g = lib.dprc_attention, lib.dprc_attention_grad
    assert lib.dprc_attention(None, A16, None, A16, need, None) == 1
    assert f(ctypes.byref(a), None, None, A16, need, None) == 1
    assert f(ctypes.byref(a), A16 + 2, None, A16, need, None) == 4
    assert f(ctypes.byref(a), A16, A16 + 2, A16, need, None) == 4
    assert f(ctypes.byref(a), A16, None, None, need, None) == 5
    assert f(ctypes.byref(a), A16, None, A16, need - 1, None) == 5
    assert f(ctypes.byref(a), A16, None, A16 + 8, need, None) == 4
    assert g(ctypes.byref(a), A16, s, A16, s, A16, None, s, None, s, None, s, A16, grad, None) == 1
    assert g(ctypes.byref(a), A16, s, A16, s, A16, A16, None, None, s, None, s, A16, grad, None) == 1
    assert g(ctypes.byref(a), None, s, A16, s, A16, A16, s, None, s, None, s, A16, grad, None) == 1
    assert g(ctypes.byref(a), A16, s, A16, s, None, A16, s, None, s, None, s, A16, grad, None) == 1
    assert g(ctypes.byref(a), A16, s, A16, s, A16, A16 + 1, s, None, s, None, s, A16, grad, None) == 4
    assert g(ctypes.byref(a), A16, s, A16, s, A16, A16, _strides(-1, 1, 1), None, s, None, s, A16,
             grad, None) == 2
    assert g(ctypes.byref(a), A16, s, A16, s, A16, A16, s, None, s, None, s, A16, grad - 1, None) == 5


def test_results_whose_rows_overlap_are_refused(lib):
    a, s = _args(Hkv=4), _strides(1 << 20, 256, 64)  # (B 2, 100 tokens, 4 heads of 64)
    n = 1 << 40
    for bad in (_strides(0, 256, 64), _strides(1 << 20, 0, 64), _strides(1 << 20, 256, 0),
                _strides(1 << 20, 192, 64), _strides(1 << 20, 256, 63), _strides(25599, 256, 64)):
        for where in range(3):
            out = [x for k in range(3) for x in ((A16, bad) if k == where else (None, s))]
            assert lib.dprc_attention_grad(ctypes.byref(a), A16, s, A16, s, A16, *out, A16, n, None) == 2
        assert lib.dprc_rotary(A16, s, 1, 2, 100, 4, 64, A16, 8, 1, (ctypes.c_int64 * 1)(8), A16, 0, 0,
                               A16, bad, None) == 2
    # (an axis of one has any stride: this call gets as far as its workspace)
    one = _args(B=1, Tq=1, Tk=1, H=1, Hkv=1)
    z = _strides(0, 0, 0)
    assert lib.dprc_attention_grad(ctypes.byref(one), A16, z, A16, z, A16, A16, z, A16, z, A16, z, None,
                                   0, None) == 5


def test_layernorm_refusals(lib):
    f, g = lib.dprc_layernorm, lib.dprc_layernorm_grad
    ok = (A16, None, None, 1, 2, 3, 64, 1e-5, 1, A16, None, None)

    def with_(i, v):
        return f(*(v if k == i else x for k, x in enumerate(ok)))

    assert with_(0, None) == 1 and with_(9, None) == 1 and with_(3, 2) == 3
    assert with_(4, 0) == 2 and with_(4, 65536) == 2 and with_(5, -1) == 2
    assert with_(6, 0) == 2 and with_(6, 16385) == 2
    assert with_(7, float("nan")) == 2 and with_(7, -1.0) == 2
    assert with_(0, A16 + 4) == 4 and with_(1, A16 + 2) == 4 and with_(10, A16 + 8) == 4
    assert with_(5, 0) == 0  # no tokens: nothing to do
    size = lib.dprc_layernorm_workspace_bytes(2, 3, 64, 1)
    assert size > 0 and lib.dprc_layernorm_workspace_bytes(0, 3, 64, 1) == 0
    ok_g = (A16, A16, A16, None, 1, 2, 3, 64, 1, A16, A16, None, A16, 0, 0, None, A16, size, None)

    def grad(**kw):
        at = dict(dY=0, X=1, stats=2, d=7, dX=9, dW=10, n=12, c=15, ws=16, size=17)
        v = list(ok_g)
        for k, x in kw.items():
            v[at[k]] = x
        return g(*v)

    assert grad(dY=None) == 1 and grad(X=None) == 1 and grad(stats=None) == 1
    assert grad(dX=None, dW=None, n=None) == 1
    assert grad(d=0) == 2 and grad(dX=A16 + 2) == 4 and grad(n=A16 + 2) == 4 and grad(c=A16 + 1) == 4
    assert grad(ws=None) == 5 and grad(size=size - 1) == 5 and grad(ws=A16 + 4) == 4


def test_rotary_refusals(lib):
    s = _strides(4096, 64, 16)

    def call(X=A16, xs=s, dtype=1, B=2, T=3, H=4, D=16, pos=A16, size=8, axes=1, sections=(8,),
             freqs=A16, out=A16, os=s):
        sec = None if sections is None else (ctypes.c_int64 * len(sections))(*sections)
        return lib.dprc_rotary(X, xs, dtype, B, T, H, D, pos, size, axes, sec, freqs, 0, 0, out, os,
                               None)

    assert call(dtype=3) == 3 and call(size=2) == 3
    assert call(B=-1) == 2 and call(T=-1) == 2 and call(H=0) == 2 and call(D=4097) == 2
    assert call(B=1 << 20, T=1 << 20) == 2 and call(axes=0) == 2 and call(axes=9, sections=(1,) * 9) == 2
    assert call(sections=(9,)) == 2 and call(sections=(-1,)) == 2 and call(axes=2, sections=(4, 5)) == 2
    assert call(sections=None) == 1 and call(X=None) == 1 and call(out=None) == 1
    assert call(pos=None) == 1 and call(freqs=None) == 1 and call(xs=None) == 1
    assert call(xs=_strides(1, -1, 1)) == 2 and call(X=A16 + 1) == 4 and call(pos=A16 + 4) == 4
    assert call(freqs=A16 + 4) == 4 and call(T=0) == 0


def test_binding_refusals():
    x = torch.zeros(2, 3, 4, 8)
    for call in (lambda: binding.dprc_attention(x, x, x), lambda: binding.dprc_layernorm(x),
                 lambda: binding.dprc_rotary(x, torch.zeros(2, 3).long(), torch.ones(4).double()),
                 lambda: binding.dprc_layernorm_grad(x, x, x, dX=x),
                 lambda: binding.dprc_attention_grad(x, x, x, x, x, x, dQ=x)):
        with pytest.raises(ValueError, match="device tensors"):
            call()


class Fake:
    """What a call looks at of a device tensor."""
    is_cuda = True
    requires_grad = False

    def __init__(self, shape, dtype=torch.float32, device=0, stride=None):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device = torch.device("cuda", device)
        self._stride = stride

    def stride(self):
        if self._stride is not None:
            return self._stride
        return torch.empty(self.shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return self._stride is None

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return A16


I32, F64 = torch.int32, torch.float64
ATT = dict(Q=((2, 5, 4, 8),), K=((2, 7, 2, 8),), V=((2, 7, 2, 8),), slopes=((4,),), docs=((2, 7), I32),
           prefix=((2,), I32), lengths=((2,), I32), first=((2,), I32), ws=((1 << 20,), torch.uint8))
CALLS = {
    "attention": (binding.dprc_attention, dict(ATT, out=((2, 5, 4, 8),), lse=((2, 4, 5),))),
    "attention_grad": (binding.dprc_attention_grad, dict(
        ATT, dO=((2, 5, 4, 8),), O=((2, 5, 4, 8),), lse=((2, 4, 5),), dQ=((2, 5, 4, 8),),
        dK=((2, 7, 2, 8),), dV=((2, 7, 2, 8),))),
    "layernorm": (binding.dprc_layernorm, dict(X=((2, 3, 8),), weight=((8,),), bias=((8,),),
                                               out=((2, 3, 8),), stats=((2, 3, 2),))),
    "layernorm_grad": (binding.dprc_layernorm_grad, dict(
        dY=((2, 3, 8),), X=((2, 3, 8),), stats=((2, 3, 2),), weight=((8,),), dX=((2, 3, 8),),
        dW=((8,),), db=((8,),), n=((2,),), c=((2,),), ws=((1 << 20,), torch.uint8))),
    "rotary": (binding.dprc_rotary, dict(X=((2, 3, 4, 8),), positions=((2, 3), I32),
                                         freqs=((4,), F64), out=((2, 3, 4, 8),))),
}


@pytest.fixture
def fakes(monkeypatch):
    made = []

    class Lib:
        def __getattr__(self, name):
            return (lambda *a: 64) if name.endswith("_bytes") else (lambda *a: made.append(name) or 0)

    monkeypatch.setattr(binding, "lib", Lib)
    monkeypatch.setattr(binding, "_stream", lambda t, stream: 0)
    return made


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_other_devices_types_and_shapes_are_refused(name, fakes):
    f, spec = CALLS[name]
    f(**{k: Fake(*v) for k, v in spec.items()})
    assert fakes == ["dprc_" + name]
    for k, v in spec.items():
        others = {n: Fake(*w) for n, w in spec.items() if n != k}
        with pytest.raises((ValueError, TypeError)):
            f(**others, **{k: Fake(*v, **({} if len(v) > 1 else {"dtype": torch.float32}), device=1)})
        if k == "ws":
            continue
        with pytest.raises((ValueError, TypeError, binding.DprcError)):
            f(**others, **{k: Fake(v[0], torch.bfloat16)})
        wrong = (*v[0][:-1], v[0][-1] + 1)
        if not (name in ("layernorm", "rotary", "layernorm_grad") and k in ("X", "dY", "positions", "freqs")):
            with pytest.raises((ValueError, TypeError, binding.DprcError)):
                f(**others, **{k: Fake(wrong, *v[1:])})
    assert fakes == ["dprc_" + name]


def test_strided_heads_and_bad_sections_are_refused(fakes):
    spec = {k: Fake(*v) for k, v in CALLS["attention"][1].items()}
    with pytest.raises(ValueError, match="together"):
        binding.dprc_attention(**dict(spec, Q=Fake((2, 5, 4, 8), stride=(160, 32, 1, 4))))
    r = {k: Fake(*v) for k, v in CALLS["rotary"][1].items()}
    for sections in ([3], [2, 2], [5, -1]):
        with pytest.raises(ValueError, match="sections"):
            binding.dprc_rotary(**r, sections=sections)
    with pytest.raises(ValueError, match="positions"):
        binding.dprc_rotary(**dict(r, positions=Fake((2, 4), I32)))
    assert fakes == []


# ---- the torch modules ---------------------------------------------------------
@pytest.fixture
def host(monkeypatch):
    block_library.install(monkeypatch)
    torch.manual_seed(3)


def _directional(f, x, h=1e-3):
    """The slope of f along a direction of x against autograd's, in fp32."""
    v = torch.randn_like(x)
    (g,) = torch.autograd.grad(f(x), x)
    with torch.no_grad():
        diff = (f(x + h * v).double() - f(x - h * v).double()) / (2 * h)
    assert abs(float((g * v).sum()) - float(diff)) <= 2e-2 * max(1.0, abs(float(diff)))


@pytest.mark.parametrize("center", [True, False])
def test_layernorm_module(host, center):
    m = lay.LayerNorm(6, center=center)
    x, u = torch.randn(2, 3, 6, requires_grad=True), torch.randn(2, 3, 6)
    _directional(lambda t: (m(t) * u).sum(), x)
    ref = torch.nn.functional.layer_norm(x, (6,)) if center else torch.nn.functional.rms_norm(x, (6,), eps=1e-5)
    assert torch.allclose(m(x), ref, atol=1e-5)
    g = torch.autograd.grad((m(x) * u).sum(), (m.weight, m.bias))
    assert torch.allclose(g[0], (u * ref).sum((0, 1)), atol=1e-4)
    assert torch.allclose(g[1], u.sum((0, 1)), atol=1e-5)
    (gx,) = torch.autograd.grad((m(x).tanh() * u).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        gx.square().sum().backward()


def test_attend_and_rotary_functions(host):
    q, k, v = (torch.randn(2, 5, h, 4, requires_grad=True) for h in (4, 2, 2))
    u = torch.randn(2, 5, 4, 4)
    kw = dict(cap=3.0, docs=torch.tensor([[0, 0, 0, 1, 1], [2, 2, -1, -1, -1]]).int())
    for x, f in ((q, lambda t: lay.attend(t, k, v, **kw)), (k, lambda t: lay.attend(q, t, v, **kw)),
                 (v, lambda t: lay.attend(q, k, t, **kw))):
        _directional(lambda t: (f(t) * u).sum(), x)
    freqs, pos = lay.rotary_freqs(2), torch.arange(5).expand(2, 5)
    _directional(lambda t: (lay.rotary(t, pos, freqs) * u).sum(), q)
    with pytest.raises(ValueError, match="slopes"):
        lay.attend(q, k, v, slopes=torch.ones(4, requires_grad=True))


def test_attention_module_is_its_parts(host):
    m = lay.Attention(4, 2, 6, cap=5.0, slopes=torch.tensor([0.5, 0.2, 0.1, 0.0]),
                      freqs=lay.rotary_freqs(3))
    rows = torch.randn(2, 7, 48, requires_grad=True)
    docs = torch.tensor([[0, 0, 0, 1, 1, 1, -1]] * 2).int()
    y = m(rows, docs=docs)
    r = rows.view(2, 7, 8, 6)
    pos = torch.arange(7).expand(2, 7)
    q, k = (lay.rotary(t, pos, m.freqs) for t in (r[:, :, :4], r[:, :, 4:6]))
    z = lay.attend(q, k, r[:, :, 6:], cap=5.0, slopes=m.slopes, docs=docs).reshape(2, 7, 24)
    assert torch.allclose(y, z, atol=1e-6)
    u = torch.randn_like(y)
    a, b = (torch.autograd.grad((t * u).sum(), rows, retain_graph=True)[0] for t in (y, z))
    assert torch.allclose(a, b, atol=1e-5)
    with pytest.raises(ValueError, match="rows"):
        m(torch.randn(2, 7, 47))
    c = copy.deepcopy(m).to(torch.bfloat16)
    assert c.freqs.dtype == torch.float64 and c.slopes.dtype == torch.float32


def _reference(losses, params, C):
    per = [torch.autograd.grad(l, params, retain_graph=True, allow_unused=True) for l in losses]
    n = np.array([sum(float((t.double() ** 2).sum()) for t in g if t is not None) for g in per])
    c = np.minimum(1.0, C / np.sqrt(n))
    return n, [sum(c[i] * g[j] for i, g in enumerate(per)) for j in range(len(params))]


@pytest.mark.parametrize("trained", ["both", "weight", "bias", "rms"])
def test_step_takes_normalisations(host, trained):
    """With P = I the step is per-sample clipping of all parameters."""
    m = torch.nn.Sequential(lay.Embedding(9, 8), lay.LayerNorm(8, center=trained != "rms"),
                            lay.Linear(8, 8, bias=True, act="silu"), lay.LayerNorm(8),
                            torch.nn.Linear(8, 8, bias=False))
    if trained == "weight":
        m[1].bias.requires_grad_(False)
    if trained == "bias":
        m[1].weight.requires_grad_(False)
    with torch.no_grad():
        for p in m.parameters():
            p.add_(0.1 * torch.randn_like(p))
    tok = torch.randint(0, 9, (4, 6))
    f = lambda: (m(tok) ** 2).mean(dim=(1, 2))  # noqa: E731
    step = RandomizedClippingStep(m, C=0.3, sigma=0.0, k=8)
    params = step.parameters()
    assert {id(p) for p in params} == {id(p) for p in m.parameters() if p.requires_grad}
    n, total = _reference(f(), params, 0.3)
    out = step(f(), step=0, projections=[torch.eye(l.out_features) for l in step.layers])
    assert np.allclose(out["n"].numpy(), n, rtol=1e-4)
    for p, ref in zip(params, total):
        assert torch.allclose(p.grad, ref, rtol=1e-3, atol=1e-6)
    step.close()


def test_step_refuses_shared_normalisations(host):
    a, b = lay.LayerNorm(8), lay.LayerNorm(8)
    b.weight = a.weight
    with pytest.raises(ValueError, match="shared"):
        RandomizedClippingStep(torch.nn.Sequential(a, b), C=1.0, sigma=0.0)
    m = lay.LayerNorm(8)
    step = RandomizedClippingStep(m, C=1.0, sigma=0.0)
    x = torch.randn(3, 4, 8)
    with pytest.raises(ValueError, match="more than once"):
        step((m(m(x)) ** 2).sum(dim=(1, 2)), step=0)
    step.close()


def test_example_with_heads(host):
    """Its per-sample norms, and its generation against the whole pass."""
    torch.manual_seed(1)
    m = example_lm.TinyLM(vocab=16, width=16, hidden=16, blocks=2, p=0.0, dtype=torch.float32, heads=4)
    tok = torch.randint(0, 16, (3, 7))
    f = lambda: (m(tok) ** 2).mean(dim=(1, 2))  # noqa: E731
    step = RandomizedClippingStep(m, C=0.3, sigma=0.0, k=16)
    params = step.parameters()
    n, total = _reference(f(), params, 0.3)
    out = step(f(), step=0, projections=[torch.eye(l.out_features) for l in step.layers])
    assert np.allclose(out["n"].numpy(), n, rtol=1e-3)
    for p, ref in zip(params, total):
        assert torch.allclose(p.grad, ref, rtol=1e-2, atol=1e-5)
    step.close()
    got = m.eval().generate(tok, 5)
    seq = tok
    for _ in range(5):
        seq = torch.cat((seq, m(seq)[:, -1:].argmax(-1)), 1)
    assert torch.equal(got, seq[:, 7:])
