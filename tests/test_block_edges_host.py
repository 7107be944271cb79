"""The torch modules and the binding of a transformer block's operators at the borders of what they
take, without a GPU (the library's calls from the float64 oracle, or none).
"""

import pytest
import torch

import block_library
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
