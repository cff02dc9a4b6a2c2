"""The current stream's handle, with torch's private calls and without them (no GPU)."""
import types

import pytest
import torch

from mixture_experts_layer_41_b200 import api


@pytest.mark.parametrize("missing", ["_raw_stream", "_raw_device"])
def test_current_stream_without_the_private_calls(missing, monkeypatch):
    monkeypatch.setattr(api, "_raw_stream", lambda device: 5)
    monkeypatch.setattr(api, "_raw_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=7))
    assert api._s(None) == 5
    monkeypatch.setattr(api, missing, None)
    assert api._s(None) == 7
    assert api._s(9) == 9 and api._s(types.SimpleNamespace(cuda_stream=3)) == 3


@pytest.mark.gpu
def test_current_stream_handles_agree():
    torch.zeros(1, device="cuda")
    assert api._s(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(torch.cuda.Stream()):
        assert api._s(None) == torch.cuda.current_stream().cuda_stream != 0
