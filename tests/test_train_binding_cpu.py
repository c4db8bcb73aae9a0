"""The training-step operators' binding without a GPU."""
import contextlib
import copy
import pickle
import types

import pytest
import torch

from memory_aware_device_gb300 import build as nbuild
from memory_aware_device_gb300 import train


@pytest.fixture(scope="module", autouse=True)
def built():
    nbuild.build()


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    there, here = (types.SimpleNamespace(device=torch.device("cuda", i)) for i in (1, 0))
    with pytest.raises(ValueError, match="cuda:1"):
        train._enter(torch.device("cuda", 0), there)
    train._enter(torch.device("cuda", 0), here).leave()


def test_copied_buffers_do_not_use_the_original_workspace():
    out = train.Routing.empty(3000, 200, 4, device="cpu")
    deep, back = copy.deepcopy(out), pickle.loads(pickle.dumps(out))
    assert deep.call.key == out.call.key and deep.call.tail != out.call.tail
    for other in (out, deep, back):
        assert len(other) == 6 and other.ids.shape == (3000, 4)
        if other.call is not None:      # else a call makes its own
            assert other.call.tail == (other.call.workspace.data_ptr(), other.call.workspace.numel())
            assert not other.call.workspace[:256].any()
    assert deep.ids.data_ptr() != out.ids.data_ptr()
    assert copy.copy(out).call is out.call
