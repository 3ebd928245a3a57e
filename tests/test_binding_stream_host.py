"""The binding's default stream, without a GPU."""

import types

import torch

from aware_block_transforms_amd import _lib


def test_default_stream_is_the_current_one(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    assert _lib._stream(None) == 1003
    assert _lib._stream(0) == 0 and _lib._stream(77) == 77


def test_default_stream_where_torch_has_no_raw_handle(monkeypatch):
    # the raw handle's function is not part of torch's documented interface
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=2003))
    assert _lib._stream(None) == 2003
