"""The operators' calls refuse tensors of different GPUs, without a GPU."""

import pytest
import torch

from randomized_norm_clipping_gb300 import binding


class Fake:
    """What a call looks at of a device tensor."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.float32, device=0):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device = torch.device("cuda", device)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 0x10000


class Calls:
    """A library whose sizes are some and whose calls succeed."""

    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 64
        return lambda *a: self.made.append(name) or 0


@pytest.fixture
def lib(monkeypatch):
    calls = Calls()
    monkeypatch.setattr(binding, "lib", lambda: calls)
    monkeypatch.setattr(binding, "_stream", lambda t, stream: 0)
    monkeypatch.setattr(binding, "_empty",
                        lambda like, shape, st, given, dtype=None: Fake(shape, dtype or like.dtype,
                                                                        like.get_device()))
    return calls


def _plan(device=0):
    return binding.EmbedPlan(2, 5, 10, Fake((64,), torch.uint8, device))


CALLS = {
    "lookup tokens": lambda o: binding.dprc_embed_lookup(
        Fake((10, 8)), Fake((2, 5), torch.int64, o)),
    "lookup out": lambda o: binding.dprc_embed_lookup(
        Fake((10, 8)), Fake((2, 5), torch.int64), out=Fake((2, 5, 8), device=o)),
    "plan buffer": lambda o: binding.dprc_embed_plan(
        Fake((2, 5), torch.int64), 10, buf=Fake((64,), torch.uint8, o)),
    "norm plan": lambda o: binding.dprc_embed_norm(
        Fake((2, 5, 8)), _plan(o), Fake((2,)), ws=Fake((64,), torch.uint8)),
    "norm workspace": lambda o: binding.dprc_embed_norm(
        Fake((2, 5, 8)), _plan(), Fake((2,)), ws=Fake((64,), torch.uint8, o)),
    "norm n": lambda o: binding.dprc_embed_norm(
        Fake((2, 5, 8)), _plan(), Fake((2,), device=o), ws=Fake((64,), torch.uint8)),
    "gradient plan": lambda o: binding.dprc_embed_grad(
        Fake((2, 5, 8)), _plan(o), Fake((10, 8)), ws=Fake((64,), torch.uint8)),
    "gradient workspace": lambda o: binding.dprc_embed_grad(
        Fake((2, 5, 8)), _plan(), Fake((10, 8)), ws=Fake((64,), torch.uint8, o)),
    "gradient factors": lambda o: binding.dprc_embed_grad(
        Fake((2, 5, 8)), _plan(), Fake((10, 8)), c=Fake((2,), device=o),
        ws=Fake((64,), torch.uint8)),
    "dropout residual": lambda o: binding.dprc_dropout(
        Fake((8,)), 0.1, 1, 1, residual=Fake((8,), device=o)),
    "linear W": lambda o: binding.dprc_linear(
        Fake((4, 8)), Fake((6, 8), device=o), ws=Fake((64,), torch.uint8)),
    "linear workspace": lambda o: binding.dprc_linear(
        Fake((4, 8)), Fake((6, 8)), ws=Fake((64,), torch.uint8, o)),
    "linear gradient workspace": lambda o: binding.dprc_linear_grad(
        Fake((4, 6)), Fake((4, 8)), Fake((6, 8)), dX=Fake((4, 8)),
        ws=Fake((64,), torch.uint8, o)),
}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS.keys())
def test_tensors_of_two_gpus_are_refused(lib, call):
    call(0)
    assert len(lib.made) == 1  # the same call on one GPU reaches the library
    with pytest.raises(ValueError, match="cuda:1"):
        call(1)
    assert len(lib.made) == 1


# ---- arguments that must be refused in the binding's own words ---------------
def test_widths_of_zero_are_refused_by_the_library(lib, monkeypatch):
    monkeypatch.setattr(Calls, "__getattr__",
                        lambda self, name: lambda *a: 0 if name.endswith("_bytes") else 2)
    with pytest.raises(binding.DprcError):
        binding.dprc_linear(Fake((4, 0)), Fake((6, 0)))
    with pytest.raises(binding.DprcError):
        binding.dprc_linear_grad(Fake((4, 0)), Fake((4, 8)), Fake((0, 8)), dX=Fake((4, 8)))


def test_unknown_activations_are_refused(lib):
    ws = Fake((64,), torch.uint8)
    with pytest.raises(ValueError, match="tanh"):
        binding.dprc_linear(Fake((4, 8)), Fake((6, 8)), act="tanh", ws=ws)
    with pytest.raises(ValueError, match="tanh"):
        binding.dprc_linear_grad(Fake((4, 6)), Fake((4, 8)), Fake((6, 8)), act="tanh",
                                 dX=Fake((4, 8)), ws=ws)
    assert not lib.made
