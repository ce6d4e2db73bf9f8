"""CPU-only checks of the training-step operators' C entries: sizes, shapes and
bad arguments are answered on the host before any CUDA call."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_sequence_gb300 import api
    if not os.path.exists(api.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return api._load()


OK, ARG, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 4)


def _ce(lib, T, V, D, grad=0):
    f, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = lib.linear_ce_workspace_bytes(T, V, D, grad, ctypes.byref(f), ctypes.byref(b))
    return st, f.value, b.value


@pytest.mark.parametrize("T,V,D,expect", [
    (1, 1, 8, OK), (8192, 65536, 2048, OK), (333, 5003, 328, OK), (1 << 23, 2, 8, OK), (0, 5, 8, ARG), (5, 0, 8, ARG),
    (5, 5, 0, ARG), (5, 5, 12, UNSUPPORTED), ((1 << 23) + 1, 5, 8, UNSUPPORTED), (5, (1 << 23) + 1, 8, UNSUPPORTED),
    (5, 5, (1 << 16) + 8, UNSUPPORTED),
])
def test_linear_ce_shapes(lib, T, V, D, expect):
    st, fwd, bwd = _ce(lib, T, V, D)
    assert st == expect
    if st == OK:
        assert fwd % 256 == 0 and bwd % 256 == 0 and fwd >= 256 + 8 * T
        assert bwd >= 2 * T * D + 2 * T * min(V, 256)


def test_linear_ce_keeps_one_piece_of_the_vocabulary(lib):
    """The backward's scratch does not grow with the vocabulary once a piece is full."""
    T, D = 65536, 1024
    sizes = [_ce(lib, T, V, D)[2] for V in (1 << 14, 1 << 17, 1 << 20)]
    logits = [2 * T * V for V in (1 << 14, 1 << 17, 1 << 20)]
    assert sizes[2] < logits[2] / 100
    assert max(sizes) < (512 << 20) + 6 * T * D + (8 << 20) + 2 * T * 256


def test_linear_ce_bad_arguments(lib):
    assert _ce(lib, 5, 5, 8, grad=3)[0] == ARG
    fwd = [P, P, P, 5, 5, 8, 0.0, P, P, P, P, None]
    for i, bad in ((0, None), (1, ODD), (2, None), (6, -1.0), (6, float("nan")), (6, float("inf")), (7, None), (8, ODD),
                   (9, None), (10, None), (10, ODD)):
        a = list(fwd)
        a[i] = bad
        assert lib.linear_ce_forward(*a) == ARG, i
    bwd = [P, P, P, P, None, P, 5, 5, 8, 0.0, P, P, 0, P, None]
    for i, bad in ((0, None), (3, None), (4, ODD), (5, None), (10, None), (11, ODD), (12, 2), (13, None)):
        a = list(bwd)
        a[i] = bad
        assert lib.linear_ce_backward(*a) == ARG, i   # (5: neither dloss nor total)


@pytest.mark.parametrize("T,D,expect", [(1, 8, OK), (16384, 1024, OK), (3, 8192, OK), (0, 64, ARG), (3, 0, ARG),
                                        (3, 12, UNSUPPORTED), (3, 8200, UNSUPPORTED)])
def test_gated_norm_shapes(lib, T, D, expect):
    s, c = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert lib.gated_norm_workspace_bytes(T, D, ctypes.byref(s), ctypes.byref(c)) == expect
    if expect == OK:
        assert s.value >= 8 * T and c.value >= 8 * D


def test_gated_norm_bad_arguments(lib):
    # x, y, gate, gamma_post, scale, gamma_pre, T, D, eps, r, h, saved, stream
    fwd = [P, P, P, P, P, P, 4, 64, 1e-6, P, P, P, None]
    for i, bad in ((0, None), (1, ODD), (2, ODD), (5, ODD), (8, 0.0), (8, float("nan")), (8, 1.5), (9, None), (10, None),
                   (11, ODD)):
        a = list(fwd)
        a[i] = bad
        assert lib.gated_norm_forward(*a) == ARG, i
    # without a branch there is nothing for a gate, a scale, a second norm or r
    none = [P, None, None, None, None, P, 4, 64, 1e-6, None, P, P, None]
    for i in (2, 3, 4, 9):
        a = list(none)
        a[i] = P
        assert lib.gated_norm_forward(*a) == ARG, i
    # dr, dh, x, y, gate, gamma_post, scale, gamma_pre, T, D, eps, saved, dx, dy, dgate, dgamma_post, dscale,
    # dgamma_pre, scratch, stream
    bwd = [P] * 8 + [4, 64, 1e-6] + [P] * 8 + [None]
    for i, bad in ((0, ODD), (1, None), (11, None), (12, None), (13, None), (14, None), (15, None), (16, None),
                   (17, None), (18, None)):
        a = list(bwd)
        a[i] = bad
        assert lib.gated_norm_backward(*a) == ARG, i
    a = list(bwd)
    a[4] = None          # no gate, yet its gradient is asked for
    assert lib.gated_norm_backward(*a) == ARG


def test_adamw_bad_arguments(lib):
    from linear_recurrence_sequence_gb300 import api

    def tensors(**change):
        t = (api._AdamwTensor * 2)()
        for e in t:
            for k in ("param", "master", "grad", "m", "v"):
                setattr(e, k, 1 << 20)
            e.n, e.weight_decay, e.grad_dtype = 300, 0.1, 1
        for k, v in change.items():
            setattr(t[1], k, v)
        return t

    def step(t, count=2, step=P, lr=P, b1=0.9, b2=0.95, eps=1e-8, max_norm=1.0, norm=P, scratch=P):
        return lib.lrs_adamw_step(ctypes.addressof(t) if t is not None else None, count, step, lr, b1, b2, eps, max_norm,
                                  norm, scratch, None)

    assert step(None) == ARG and step(tensors(), count=0) == ARG
    for change in ({"param": None}, {"grad": None}, {"m": None}, {"v": (1 << 20) + 4}, {"master": (1 << 20) + 2},
                   {"n": 0}, {"grad_dtype": 7}, {"m_scale": 1 << 20}, {"v_scale": 1 << 20}, {"weight_decay": -1.0},
                   {"weight_decay": float("nan")}):
        assert step(tensors(**change)) == ARG, change
    assert step(tensors(n=1 << 41)) == UNSUPPORTED
    for kw in ({"step": None}, {"lr": None}, {"b1": 1.0}, {"b2": -0.5}, {"b1": float("nan")}, {"eps": 0.0},
               {"eps": float("inf")}, {"max_norm": -1.0}, {"max_norm": float("nan")}, {"norm": None}, {"scratch": None},
               {"scratch": ODD}):
        assert step(tensors(), **kw) == ARG, kw
    n = ctypes.c_size_t(0)
    assert lib.lrs_adamw_scratch_bytes(0, ctypes.byref(n)) == ARG
    assert lib.lrs_adamw_scratch_bytes(14, None) == ARG
    assert lib.lrs_adamw_scratch_bytes(900, ctypes.byref(n)) == OK and n.value > 256
