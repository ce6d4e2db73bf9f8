"""The selective scan's limits on the host."""
import ctypes
import os

import pytest

from linear_recurrence_sequence_gb300 import api

OK, UNSUPPORTED = 0, 2


@pytest.mark.parametrize("B,L,D,N,expect", [
    (1, 8, 1 << 26, 1, OK), (1, 8, (1 << 26) + 8, 1, UNSUPPORTED), (1, 2, 1 << 29, 1, UNSUPPORTED), (1, 1, 1 << 29, 1, OK)])
def test_tokens_rows_are_within_32_bits_of_a_tiles_first(B, L, D, N, expect):
    """The kernels address a tile's eight rows of dy, which are D apart, from the first one's with 32 bits: 7 D of more
    than 2^31 would be another place in memory.  (One token has no second row.)"""
    if not os.path.exists(api.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    n = [ctypes.c_size_t(0) for _ in range(3)]
    assert api._load().selective_scan_workspace_bytes(B, L, D, N, *[ctypes.byref(v) for v in n]) == expect
