"""The training-step operators' binding without a GPU."""
import contextlib
import types

import pytest
import torch

from memory_aware_device_gb300 import train


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    there, here = (types.SimpleNamespace(device=torch.device("cuda", i)) for i in (1, 0))
    with pytest.raises(ValueError, match="cuda:1"):
        train._enter(torch.device("cuda", 0), there)
    train._enter(torch.device("cuda", 0), here).leave()
