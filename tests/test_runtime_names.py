"""The binding finds the current device and stream with or without torch's short forms."""
import types

import pytest
import torch

import exact_attention_online_gb300 as fa


@pytest.mark.parametrize("short", [True, False], ids=["short", "public"])
def test_current_device_and_stream(monkeypatch, short):
    monkeypatch.setattr(fa, "_cuda", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=1000 + device))
    for name, form in (("_cuda_getDevice", lambda: 3),
                       ("_cuda_getCurrentRawStream", lambda device: 1000 + device)):
        if short:
            monkeypatch.setattr(torch._C, name, form, raising=False)
        else:
            monkeypatch.delattr(torch._C, name, raising=False)
    assert fa._current_index() == 3
    assert fa._stream(None) == 1003
