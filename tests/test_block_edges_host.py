"""The torch modules and the binding of a transformer block's operators at the borders of what they
take, without a GPU (the library's calls from the float64 oracle, or none).
"""

import pytest
import torch

import block_library
from randomized_norm_clipping_gb300 import binding
from randomized_norm_clipping_gb300 import layers as lay


@pytest.fixture
def host(monkeypatch):
    block_library.install(monkeypatch)
    torch.manual_seed(7)


MASKS = {
    "docs": torch.tensor([[0, 0, 1, 1, 1], [2, 2, 2, -1, -1]], dtype=torch.int32),
    "prefix": torch.tensor([3, 0], dtype=torch.int32),
    "lengths": torch.tensor([4, 2], dtype=torch.int32),
    "first": torch.tensor([1, 0], dtype=torch.int32),
    "slopes": torch.tensor([0.5, 0.25, 0.1, 0.0]),
}


# (the module's queries stand at 0, 1, 2, ..)
@pytest.mark.parametrize("name,module", [(n, m) for n in MASKS for m in (False, True)
                                         if (n, m) != ("first", True)])
def test_a_mask_that_changes_before_the_backward_pass_raises(host, name, module):
    mask = MASKS[name].clone()
    rows = torch.randn(2, 5, 48, requires_grad=True)
    if module:
        m = lay.Attention(4, 2, 6, slopes=mask if name == "slopes" else None)
        call = lambda: m(rows, **({} if name == "slopes" else {name: mask}))  # noqa: E731
        mask = m.slopes if name == "slopes" else mask
    else:
        q, k, v = rows.view(2, 5, 8, 6).split([4, 2, 2], 2)
        call = lambda: lay.attend(q, k, v, **{name: mask})  # noqa: E731
    u = torch.randn_like(call())
    (before,) = torch.autograd.grad((call() * u).sum(), rows, retain_graph=True)
    y = (call() * u).sum()
    mask.copy_(mask.flip(-1))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    (after,) = torch.autograd.grad((call() * u).sum(), rows)
    assert not torch.equal(before, after)  # (the change is one that the gradient shows)


class Fake:
    """What a call looks at of a device tensor."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def calls(monkeypatch):
    """The names and arguments of the library's calls, which do nothing."""
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or (64 if name.endswith("_bytes") else 0)

    monkeypatch.setattr(binding, "lib", Lib)
    return made


def _sizes(calls):
    """(B, T, d) of the normalisation's gradient and of its workspace, as they were called."""
    at = dict(dprc_layernorm_workspace_bytes=0, dprc_layernorm_grad=5)
    return [a[at[name]:at[name] + 3] for name, a in calls]


def test_rows_are_samples_only_where_samples_count(calls, monkeypatch):
    monkeypatch.setattr(binding, "_scratch", lambda *a: Fake(64, dtype=torch.uint8))
    f = lambda *shape, **kw: binding.dprc_layernorm_grad(  # noqa: E731
        Fake(*shape), Fake(*shape), Fake(*shape[:-1], 2), stream=0, **kw)
    f(70000, 8, dX=Fake(70000, 8), dW=Fake(8))
    f(70000, 3, 8, dW=Fake(8))
    assert _sizes(calls) == [(1, 70000, 8)] * 2 + [(1, 210000, 8)] * 2
    del calls[:]
    f(7, 3, 8, dW=Fake(8), c=Fake(7))
    f(7, 3, 8, n=Fake(7))
    f(8, dX=Fake(8))
    assert _sizes(calls) == [(7, 3, 8)] * 4 + [(1, 1, 8)] * 2


def test_batches_without_samples(calls, monkeypatch):
    """A gradient of no samples is zeros (a call of no tokens), norms of none are nothing."""
    monkeypatch.setattr(binding, "_scratch", lambda *a: Fake(64, dtype=torch.uint8))
    x, st = Fake(0, 5, 8), Fake(0, 5, 2)
    binding.dprc_layernorm_grad(x, x, st, dX=x, dW=Fake(8), n=Fake(0), c=Fake(0), stream=0)
    assert _sizes(calls) == [(1, 0, 8)] * 2 and calls[1][1][12] is None and calls[1][1][15] is None
    del calls[:]
    binding.dprc_layernorm_grad(x, x, st, n=Fake(0), stream=0)
    q, kv, lse = Fake(0, 5, 4, 8), Fake(0, 9, 2, 8), Fake(0, 4, 5)
    assert binding.dprc_attention(q, kv, kv, out=q, lse=lse, stream=0) is q
    binding.dprc_attention_grad(q, q, kv, kv, q, lse, dQ=q, dK=kv, dV=kv, stream=0)
    binding.dprc_layernorm_grad(Fake(2, 0, 8), Fake(2, 0, 8), Fake(2, 0, 2), dX=Fake(2, 0, 8), stream=0)
    binding.dprc_attention_grad(Fake(2, 0, 4, 8), Fake(2, 0, 4, 8), Fake(2, 9, 2, 8), Fake(2, 9, 2, 8),
                                Fake(2, 0, 4, 8), Fake(2, 4, 0), dQ=Fake(2, 0, 4, 8), stream=0)
    assert calls == []
    # a call that asks for nothing is the library's to refuse, as any such call
    binding.dprc_attention_grad(q, q, kv, kv, q, lse, stream=0)
    binding.dprc_layernorm_grad(x, x, st, stream=0)
    assert [name for name, _ in calls if not name.endswith("_bytes")] == [
        "dprc_attention_grad", "dprc_layernorm_grad"]
    with pytest.raises(ValueError):  # (arguments are looked at all the same)
        binding.dprc_attention(q, kv, Fake(0, 8, 2, 8), out=q, stream=0)
