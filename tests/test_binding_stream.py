"""Which stream a call without one takes (no device needed)."""

import types

import torch

from attn_fwd_05_b200 import binding


def test_current_stream_without_the_private_accessor(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0x1234))
    assert binding._stream(None) == 0x1234


def test_current_stream_with_it(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x5000 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert binding._stream(None) == 0x5003


def test_a_stream_given_as_a_number():
    assert binding._stream(0) == 0 and binding._stream(77) == 77
