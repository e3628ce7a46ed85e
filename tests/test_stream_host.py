"""The binding's current stream: torch's internal calls where they exist, else the
public ones, on the current device either way."""
import types

import pytest
import torch

from head_latent_attention_get_b200 import _capi as C


@pytest.fixture
def fake_cuda(monkeypatch):
    monkeypatch.setattr(C, "_device_calls", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=1000 + (device or 0)))


def test_without_the_internal_calls(fake_cuda, monkeypatch):
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    assert C._stream(None) == 1001


def test_with_the_internal_calls(fake_cuda, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 2, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 500 + device, raising=False)
    assert C._stream(None) == 502


def test_given_streams():
    assert C._stream(7) == 7
    assert C._stream(types.SimpleNamespace(cuda_stream=9)) == 9
