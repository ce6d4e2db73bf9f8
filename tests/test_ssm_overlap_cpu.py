"""Outputs that begin where an input or another output does are refused on the host: by the forwards, the steps and the
backwards of the convolution and the scan, and by the embedding.  Other kernels' CTAs may still read what one writes."""
import ctypes
import os

import pytest
import torch

from linear_recurrence_sequence_gb300 import api

# (the places are no memory: an entry that took them would launch)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a GPU")

ARG = 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return api._load()


_alive = []


def at(i):
    return (1 << 20) + (i << 16)


def V(i):
    return ctypes.c_void_p(at(i))


def R(i, batch=64 * 8, token=64):
    _alive.append(api._Rows(at(i), batch, token))
    return ctypes.addressof(_alive[-1])


# Arguments in their order: ("in"), ("out") a vector, ("rows in"), ("rows out"), "any" (may lie anywhere), or a value.
CONV = ["rows in", "in", "in", "in", "in"]
SCAN = ["rows in", "rows in", "in", "rows in", "rows in", "in", "in", "rows in"]
ENTRIES = {
    "causal_conv_forward": CONV + [2, 8, 64, 4, 1, "out", "out", None],
    "causal_conv_step": ["rows in", "in", "in", "state", "in", 2, 64, 4, 1, "out", None],
    "causal_conv_backward": ["in"] + CONV + [2, 8, 64, 4, 1, "rows out", "any", "any", "out", 0, "any", None],
    "selective_scan_forward": SCAN + ["in", "in", 2, 8, 64, 16, "out", "any", "any", "any", None],
    "selective_scan_step": SCAN + ["state", "in", 2, 64, 16, "out", None],
    "selective_scan_backward": ["in", "any"] + SCAN + ["in", 2, 8, 64, 16, "any", "rows out", "rows out", "any", "out", "out", "any",
                                                       "any", "rows out", "any", 0, "any", None],
    "embedding_forward": ["in", "in", 0, 4, 9, 64, 1.0, "out", None],
    "embedding_backward": ["in", "in", 4, 9, 64, 1.0, "out", 0, 0, "any", None],
}


def _arguments(kinds, places):
    return [R(places[i]) if k in ("rows in", "rows out") else V(places[i]) if isinstance(k, str) else k for i, k in enumerate(kinds)]


def _cases():
    for name, kinds in ENTRIES.items():
        outs = [i for i, k in enumerate(kinds) if k in ("out", "rows out")]
        ins = [i for i, k in enumerate(kinds) if k in ("in", "rows in", "state")]
        for o in outs:
            for i in ins + [p for p in outs if p < o]:
                yield name, o, i


@pytest.mark.parametrize("name,out,other", list(_cases()))
def test_refused(lib, name, out, other):
    kinds = ENTRIES[name]
    places = list(range(1, len(kinds) + 1))   # every argument at a place of its own ...
    places[out] = places[other]               # ... but for these two
    assert getattr(lib, name)(*_arguments(kinds, places)) == ARG
