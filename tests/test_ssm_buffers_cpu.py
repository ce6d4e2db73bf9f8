"""What the selective scan's, the convolution's and the embedding's bindings hand to the library: every output has the room
that the kernels write.  Runs without a GPU: the entries are stood in for."""
import os

import pytest
import torch

from linear_recurrence_sequence_gb300 import api

BF, F, U8 = torch.bfloat16, torch.float32, torch.uint8
B, L, D, N = 2, 8, 64, 16


class _Library:
    """The library, with entries that only take down their arguments."""

    def __init__(self, lib, stands_for):
        self._lib, self._stands_for, self.calls = lib, stands_for, []

    def __getattr__(self, name):
        if name not in self._stands_for:
            return getattr(self._lib, name)

        def entry(*args):
            self.calls.append((name, args))
            return 0
        return entry


@pytest.fixture()
def library(monkeypatch):
    if not os.path.exists(api.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    fake = _Library(api._load(), {"selective_scan_backward"})
    monkeypatch.setattr(api, "_load", lambda: fake)
    monkeypatch.setattr(api, "_stream", lambda device: None)
    return fake


def _z(*shape, dtype=F):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("h0", [_z(1), _z(1, D, N), _z(B, D, N, dtype=torch.float64), _z(B, D, N).transpose(1, 2), _z(B, D, N)],
                         ids=["one value", "one row", "64 bits", "transposed", "the forward's"])
@pytest.mark.parametrize("dhT", [False, True])
def test_dh0_has_its_own_shape(library, h0, dhT):
    """The backward looks only at whether there is an h0: whatever the tensor is, dh0 is [B, D, N] FP32 (a server's slot may
    have gone on to other sequences)."""
    x, s = _z(B, L, D, dtype=BF), _z(B, L, N, dtype=BF)
    saved = torch.empty(api.selective_scan_workspace_bytes(B, L, D, N)[0], dtype=U8)
    g = api.selective_scan_backward(x, _z(B, D, N) if dhT else None, x, x, _z(D, N), s, s, None, None, None, h0, None, saved)
    assert len(library.calls) == 1
    dh0 = g["dh0"]
    assert dh0.shape == (B, D, N) and dh0.dtype == F and dh0.is_contiguous() and dh0.device == x.device
    assert library.calls[0][1][-4] == dh0.data_ptr()
