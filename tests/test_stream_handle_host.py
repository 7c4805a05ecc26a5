"""Which stream a call without one runs on (no GPU needed): torch's current stream, with and without
torch's inner function for its handle."""
import types

import pytest
import torch

from transformer_gqa_attention_gb300 import abi


@pytest.fixture
def cuda(monkeypatch):
    """A torch that thinks it has initialised CUDA, device 3 current."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0x51))
    return monkeypatch


def test_the_current_streams_handle(cuda):
    cuda.setattr(torch._C, "_cuda_getCurrentRawStream", {3: 0x52}.__getitem__, raising=False)
    assert abi._stream(None) == 0x52


def test_without_the_inner_function(cuda):
    cuda.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert abi._stream(None) == 0x51


def test_a_handle_or_a_stream_that_is_given():
    assert abi._stream(0) == 0 and abi._stream(77) == 77
    assert abi._stream(types.SimpleNamespace(cuda_stream=0x53)) == 0x53
