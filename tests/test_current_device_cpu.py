"""Tensors of a device that is not the current one are refused: a launch goes to the current device, whose kernels would be
given the other one's addresses.  Runs without a GPU: the two questions to CUDA are stood in for."""
import types

import pytest
import torch

from linear_recurrence_sequence_gb300 import api


@pytest.fixture()
def devices(monkeypatch):
    """Two devices, of which .current is the current one; their streams' handles are 100 and 101."""
    now = types.SimpleNamespace(current=0)

    def stream(device):
        d = torch.device("cuda") if device is None else torch.device(device)
        index = now.current if d.index is None else d.index
        return types.SimpleNamespace(cuda_stream=100 + index, device=torch.device("cuda", index))

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", stream)
    return now


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("of", [torch.device, str])
def test_only_the_current_devices_stream(devices, current, of):
    devices.current = current
    assert api._stream(of(f"cuda:{current}")) == 100 + current
    with pytest.raises(ValueError, match=f"cuda:{1 - current}.*current device"):
        api._stream(of(f"cuda:{1 - current}"))
    assert api._stream(of("cuda")) == 100 + current
    assert api._stream(None) == 100 + current
