"""The binding's choice of a stream (no GPU needed)."""
import types

import pytest
import torch

import resident_expert_routed_gb300 as moe


@pytest.mark.parametrize("missing", ["_device", "_raw_stream"])
def test_the_current_stream_by_the_public_way(monkeypatch, missing):
    """A torch build without the calls that give the handle at once: the Stream object's is taken."""
    monkeypatch.setattr(moe, missing, None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=0x77))
    assert moe._stream(None) == 0x77


def test_a_given_stream_is_taken(monkeypatch):
    monkeypatch.setattr(moe, "_raw_stream", lambda d: 0x55 + d)
    monkeypatch.setattr(moe, "_device", lambda: 1)
    assert moe._stream(types.SimpleNamespace(cuda_stream=0x99)) == 0x99
    assert moe._stream(None) == 0x56
