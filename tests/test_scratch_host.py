"""Workspaces that the binding keeps between calls, without a GPU."""

import pytest
import torch

from randomized_norm_clipping_gb300 import binding


class _Like:
    dtype, device = torch.float32, "cpu"

    def get_device(self):
        return 0


@pytest.fixture
def made(monkeypatch):
    """Every allocation, and an emptied store."""
    got = []

    def empty(like, shape, stream, given, dtype=None):
        got.append((shape[0], stream))
        return torch.empty(*shape, dtype=dtype)

    monkeypatch.setattr(binding, "_empty", empty)
    monkeypatch.setattr(binding, "_capturing", lambda: False)
    monkeypatch.setattr(binding, "_current_stream_id", lambda device: 3, raising=False)
    binding._scratch_kept.__dict__.clear()
    yield got
    binding._scratch_kept.__dict__.clear()


def test_a_workspace_is_kept_and_an_outgrown_one_let_go(made):
    like = _Like()
    a = binding._scratch(1000, like, 16, None)
    assert binding._scratch(2000, like, 16, None) is a and len(made) == 1
    import weakref
    gone = weakref.ref(a)
    b = binding._scratch(a.numel() + 1, like, 16, None)
    assert b.numel() > a.numel() and len(made) == 2
    del a
    assert gone() is None  # (the allocator hands its memory on in the stream's order)


def test_the_default_stream_keeps_its_workspace(made, monkeypatch):
    monkeypatch.setattr(binding, "_current_stream_id", lambda device: 0, raising=False)
    a = binding._scratch(1000, _Like(), 0, None)
    assert binding._scratch(1000, _Like(), 0, None) is a


def test_nothing_is_kept_for_handles_that_torch_does_not_own(made, monkeypatch):
    """Such a stream may be destroyed with work pending and its handle given out
    again."""
    like = _Like()
    a, b = (binding._scratch(1000, like, 0x7F00, 0x7F00) for _ in range(2))
    assert a is not b
    monkeypatch.setattr(binding, "_current_stream_id", lambda device: 0x7F00, raising=False)
    a, b = (binding._scratch(1000, like, 0x7F00, None) for _ in range(2))  # current, external
    assert a is not b and not binding._scratch_kept.__dict__


def test_a_capture_gets_workspaces_of_its_own(made, monkeypatch):
    kept = binding._scratch(1000, _Like(), 16, None)
    monkeypatch.setattr(binding, "_capturing", lambda: True)
    assert binding._scratch(1000, _Like(), 16, None) is not kept
