"""CPU-only checks of the causal convolution's, the selective scan's and the embedding's entries: sizes, shapes, strides
and bad arguments are answered on the host before any CUDA call."""
import ctypes
import os

import pytest
import torch

from linear_recurrence_sequence_gb300 import api

OK, ARG, UNSUPPORTED = 0, 1, 2
AT = 1 << 20
P = ctypes.c_void_p(AT)
ODD = ctypes.c_void_p(AT + 4)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return api._load()


_alive = []


def R(data=AT, batch=64 * 8, token=64):
    _alive.append(api._Rows(data, batch, token))
    return ctypes.addressof(_alive[-1])


def _refused(fn, good, bad):
    for i, v in bad:
        a = list(good)
        a[i] = v
        assert fn(*a) == ARG, (i, v)


# ---------------------------------------------------------------------------- the convolution
@pytest.mark.parametrize("B,L,D,W,expect", [
    (1, 1, 8, 2, OK), (4, 4096, 1024, 4, OK), (3, 1009, 328, 3, OK), (0, 5, 8, 4, ARG), (1, 0, 8, 4, ARG), (1, 5, 0, 4, ARG),
    (1, 5, 8, 0, ARG), (1, 5, 12, 4, UNSUPPORTED), (1, 5, 8, 1, UNSUPPORTED), (1, 5, 8, 5, UNSUPPORTED),
    (1 << 15, 1 << 20, 64, 4, UNSUPPORTED), ((1 << 31) - 1, 128, 8, 4, UNSUPPORTED)])
def test_causal_conv_shapes(lib, B, L, D, W, expect):
    n = ctypes.c_size_t(0)
    assert lib.causal_conv_workspace_bytes(B, L, D, W, ctypes.byref(n)) == expect
    if expect == OK:
        assert n.value % 256 == 0 and n.value >= 4 * (W + 1) * D


def test_causal_conv_bad_arguments(lib):
    # x, weight, bias, state, reset, B, L, D, W, silu, y, state_out, stream
    Q = ctypes.c_void_p(AT + 4096)
    fwd = [R(), P, P, P, P, 2, 8, 64, 4, 1, Q, Q, None]
    _refused(lib.causal_conv_forward, fwd, [
        (0, None), (0, R(data=None)), (0, R(data=AT + 2)), (0, R(batch=-8)), (0, R(token=-8)), (0, R(batch=4)),
        (0, R(token=68)), (1, None), (1, ODD), (2, ODD), (3, ODD), (6, 0), (10, None), (10, ODD), (10, P), (11, ODD), (11, P)])
    # x, weight, bias, state, reset, B, D, W, silu, y, stream
    step = [R(), P, P, P, P, 2, 64, 4, 1, P, None]
    _refused(lib.causal_conv_step, step, [(0, None), (0, R(batch=12)), (1, None), (2, ODD), (3, None), (3, ODD), (9, None)])
    # dy, x, weight, bias, state, reset, B, L, D, W, silu, dx, dweight, dbias, dstate, grad_dtype, scratch, stream
    bwd = [P, R(data=AT + 64), P, P, P, P, 2, 8, 64, 4, 1, R(data=AT + 4096), P, P, P, 0, P, None]
    out = dict(data=AT + 4096)
    _refused(lib.causal_conv_backward, bwd, [
        (0, None), (1, None), (2, None), (4, None), (11, None), (11, R(token=56, **out)), (11, R(batch=8 * 64 - 8, **out)),
        (11, R(batch=0, **out)), (11, R()), (11, R(data=AT + 64)),   # (at dy, at x)
        (12, None), (13, ODD), (14, ODD), (15, 2), (16, None)])   # (4: a gradient of a state that is not there)


# ---------------------------------------------------------------------------- the scan
@pytest.mark.parametrize("B,L,D,N,expect", [
    (1, 1, 8, 1, OK), (4, 4096, 1024, 16, OK), (1, 32768, 2048, 16, OK), (3, 1009, 328, 12, OK), (256, 1, 2048, 64, OK),
    (0, 5, 8, 4, ARG), (1, 0, 8, 4, ARG), (1, 5, 0, 4, ARG), (1, 5, 8, 0, ARG), (1, 5, 12, 4, UNSUPPORTED),
    (1, 5, 8, 65, UNSUPPORTED), (1 << 16, 1 << 16, 8, 4, UNSUPPORTED), (1 << 10, 1 << 20, 4096, 4, UNSUPPORTED)])
def test_selective_scan_shapes(lib, B, L, D, N, expect):
    n = [ctypes.c_size_t(0) for _ in range(3)]
    assert lib.selective_scan_workspace_bytes(B, L, D, N, *[ctypes.byref(v) for v in n]) == expect
    if expect == OK:
        saved, fwd, bwd = (v.value for v in n)
        assert all(v % 256 == 0 for v in (saved, fwd, bwd))
        assert saved >= 4 * B * -(-L // 8) * D * N and fwd >= 256 and bwd >= 4 * D * N + 8 * B * L * N


def test_selective_scan_bad_arguments(lib):
    S = R(batch=8 * 48, token=48)
    # x, delta, a_log, b, c, d_skip, delta_bias, gate, h0, reset, B, L, D, N, y, hT, saved, scratch, stream
    ins = [R(), R(), P, S, S, P, P, R()]
    rows = [(0, None), (0, R(data=AT + 2)), (1, None), (1, R(token=4)), (2, None), (3, None), (3, R(data=AT + 1)),
            (3, R(token=-1)), (4, None), (4, R(batch=-1)), (5, ODD), (6, ODD), (7, R(batch=2))]
    rows += [(i, R(token=(1 << 26) + 8)) for i in (0, 1, 3, 4, 7)]
    outs = [AT + 4096 * i for i in range(1, 7)]
    o = [ctypes.c_void_p(v) for v in outs]
    fwd = ins + [P, P, 2, 8, 64, 16, o[0], P, P, P, None]
    _refused(lib.selective_scan_forward, fwd, rows + [(8, ODD), (13, 0), (14, None), (14, P), (15, None), (15, ODD), (16, ODD),
                                                      (17, None)])
    # .., state, reset, B, D, N, y, stream
    step = ins + [P, P, 2, 64, 16, P, None]
    _refused(lib.selective_scan_step, step, rows + [(8, None), (8, ODD), (13, None)])
    # dy, dhT, .., reset, B, L, D, N, saved, dx, ddelta, da_log, db, dc, dd_skip, ddelta_bias, dgate, dh0, grad_dtype, scratch
    dx, dd, dg = (R(data=v) for v in outs[:3])
    bwd = [P, P] + ins + [P, 2, 8, 64, 16, P, dx, dd, P, o[3], o[4], P, P, dg, P, 1, P, None]
    _refused(lib.selective_scan_backward, bwd, [(i + 2, v) for i, v in rows if not (i in (5, 6) and v is None)] + [
        (0, None), (0, ODD), (1, ODD), (15, None), (16, None), (16, R(data=outs[0], token=32)), (17, None),
        (17, R(data=outs[1], batch=0)), (18, None), (19, None), (20, ODD), (21, ODD), (22, ODD), (23, None),
        (23, R(data=outs[2], token=0)), (24, ODD), (25, 7), (26, None)])
    # two outputs at one place, an output at an input
    _refused(lib.selective_scan_backward, bwd, [(16, dd), (17, dg), (23, dx), (19, o[0]), (20, o[3]), (16, R()), (17, R()),
                                                (23, R()), (19, P), (20, P)])
    for gone in (7, 8, 9):   # an output whose input is not there
        a = list(bwd)
        a[gone] = None
        assert lib.selective_scan_backward(*a) == ARG, gone


# ---------------------------------------------------------------------------- the embedding
@pytest.mark.parametrize("T,V,D,expect", [
    (1, 1, 8, OK), (16384, 32768, 1024, OK), (5001, 50021, 2560, OK), (7, 1 << 23, 8, OK), (0, 5, 8, ARG), (5, 0, 8, ARG),
    (5, 5, 0, ARG), (5, 5, 12, UNSUPPORTED), (5, (1 << 23) + 1, 8, UNSUPPORTED), (5, 5, (1 << 16) + 8, UNSUPPORTED),
    ((1 << 28) + 1, 5, 8, UNSUPPORTED), (1 << 28, 5, (1 << 12) + 8, UNSUPPORTED)])
def test_embedding_shapes(lib, T, V, D, expect):
    n = ctypes.c_size_t(0)
    assert lib.embedding_workspace_bytes(T, V, D, ctypes.byref(n)) == expect
    if expect == OK:
        assert n.value % 256 == 0 and n.value >= 16 * T + 4 * V


def test_embedding_bad_arguments(lib):
    # tokens, w, w_dtype, T, V, D, scale, y, stream
    fwd = [P, P, 0, 4, 9, 64, 1.0, P, None]
    _refused(lib.embedding_forward, fwd, [(0, None), (0, ODD), (1, None), (1, ODD), (2, 2), (6, float("nan")), (6, float("inf")),
                                          (7, None), (7, ODD)])
    # dy, tokens, T, V, D, scale, dw, grad_dtype, accumulate, scratch, stream
    bwd = [P, P, 4, 9, 64, 1.0, P, 0, 0, P, None]
    _refused(lib.embedding_backward, bwd, [(0, None), (0, ODD), (1, None), (1, ODD), (5, float("-inf")), (6, None), (7, 5),
                                           (9, None), (9, ODD)])


# ---------------------------------------------------------------------------- the binding, on CPU tensors
BF, F, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture()
def stopped(monkeypatch, lib):
    """Calls with good arguments end at the stream."""
    def no_stream(device):
        raise RuntimeError("nothing is launched here")
    monkeypatch.setattr(api, "_stream", no_stream)


def _z(*shape, dtype=F):
    return torch.zeros(*shape, dtype=dtype)


def _conv():
    return {"x": _z(2, 8, 128, dtype=BF)[..., 64:], "weight": _z(4, 64), "bias": _z(64), "state": _z(2, 3, 64, dtype=BF),
            "reset": _z(2, 8, dtype=U8)}


def _scan():
    small = _z(2, 8, 7 + 32, dtype=BF)
    return {"x": _z(2, 8, 128, dtype=BF)[..., 64:], "delta": _z(2, 8, 64, dtype=BF), "a_log": _z(64, 16),
            "b": small[..., 7:23], "c": small[..., 23:], "d_skip": _z(64), "delta_bias": _z(64),
            "gate": _z(2, 8, 128, dtype=BF)[..., :64], "h0": _z(2, 64, 16), "reset": _z(2, 8, dtype=U8)}


CONV_BAD = {
    "x": [_z(2, 8, 64), _z(2, 64, dtype=BF), _z(2, 8, 132, dtype=BF)[..., 4:68], _z(2, 8, 68, dtype=BF)[..., :64],
          _z(2, 64, 8, dtype=BF).transpose(1, 2)],
    "weight": [_z(64, 4), _z(4, 64, dtype=BF), _z(64)], "bias": [_z(63), _z(64, dtype=BF)],
    "state": [_z(2, 4, 64, dtype=BF), _z(2, 3, 64)], "reset": [_z(2, 9, dtype=U8), _z(2, 8, dtype=torch.bool)]}
SCAN_BAD = {
    "x": CONV_BAD["x"], "delta": [_z(2, 8, 72, dtype=BF), _z(2, 8, 64)], "a_log": [_z(16, 64), _z(64, 16, dtype=BF), _z(64)],
    "b": [_z(2, 8, 15, dtype=BF), _z(2, 8, 16), _z(2, 8, 32, dtype=BF)[..., ::2]], "c": [_z(2, 8, 1, 16, dtype=BF), None],
    "d_skip": [_z(65)], "delta_bias": [_z(64, 1)], "gate": [_z(2, 8, 64), _z(2, 7, 64, dtype=BF)],
    "h0": [_z(2, 16, 64), _z(2, 64, 16, dtype=BF)], "reset": [_z(2, 8)]}


def _bad_calls(call, good, bad):
    with pytest.raises(RuntimeError, match="nothing is launched"):
        call(good())
    for k, values in bad.items():
        for v in values:
            with pytest.raises((ValueError, TypeError), match=k):
                call(good() | {k: v})


def test_conv_binding_refuses_by_name(stopped):
    _bad_calls(lambda a: api.causal_conv_forward(**a), _conv, CONV_BAD)
    dy = _z(2, 8, 64, dtype=BF)
    _bad_calls(lambda a: api.causal_conv_backward(dy, **a), _conv, CONV_BAD)
    with pytest.raises(ValueError, match="dy"):
        api.causal_conv_backward(dy[:, :7], **_conv())
    for dx in (_z(2, 8, 64), _z(1, 8, 64, dtype=BF).expand(2, 8, 64), _z(2, 8, 32, dtype=BF)):
        with pytest.raises((ValueError, TypeError), match="dx"):
            api.causal_conv_backward(dy, **_conv(), out={"dx": dx})
    n = api.causal_conv_workspace_bytes(2, 8, 64, 4)
    with pytest.raises(ValueError, match="scratch"):
        api.causal_conv_backward(dy, **_conv(), scratch=torch.empty(n - 1, dtype=U8))

    def step(**k):
        a = {"x": _z(2, 128, dtype=BF)[:, :64], "weight": _z(4, 64), "bias": None, "state": _z(2, 3, 64, dtype=BF)} | k
        return api.causal_conv_step(**a)
    with pytest.raises(RuntimeError, match="nothing is launched"):
        step()
    for k in ({"x": _z(2, 8, 64, dtype=BF)}, {"state": None}, {"state": _z(2, 2, 64, dtype=BF)}, {"reset": _z(2)}):
        with pytest.raises((ValueError, TypeError), match=next(iter(k))):
            step(**k)
    for W in (1, 5):
        with pytest.raises(api.LrsError):
            api.causal_conv_workspace_bytes(2, 8, 64, W)


def test_scan_binding_refuses_by_name(stopped):
    _bad_calls(lambda a: api.selective_scan_forward(**a), _scan, SCAN_BAD)
    dy, dhT = _z(2, 8, 64, dtype=BF), _z(2, 64, 16)
    n = api.selective_scan_workspace_bytes(2, 8, 64, 16)
    saved = torch.empty(n[0], dtype=U8)
    bwd = {k: v for k, v in SCAN_BAD.items() if k != "h0"}
    _bad_calls(lambda a: api.selective_scan_backward(dy, dhT, **a, saved=saved), _scan, bwd)
    for bad in (None, saved[:-1]):
        with pytest.raises(ValueError, match="saved"):
            api.selective_scan_backward(dy, dhT, **_scan(), saved=bad)
    with pytest.raises(ValueError, match="dhT"):
        api.selective_scan_backward(dy, dhT[:, :8], **_scan(), saved=saved)
    for key in ("dx", "ddelta", "dgate"):
        with pytest.raises(ValueError, match="rows overlap"):
            api.selective_scan_backward(dy, dhT, **_scan(), saved=saved, out={key: _z(2, 1, 64, dtype=BF).expand(2, 8, 64)})
    for i, fn in ((1, lambda s: api.selective_scan_forward(**_scan(), scratch=s)),
                  (2, lambda s: api.selective_scan_backward(dy, dhT, **_scan(), saved=saved, scratch=s))):
        with pytest.raises(ValueError, match="scratch"):
            fn(torch.empty(n[i] - 1, dtype=U8))
    s = {k: (v if k in ("a_log", "d_skip", "delta_bias", "h0") else v[:, 0].contiguous() if k == "reset" else v[:, 0]) for k, v in _scan().items()}
    s["state"] = s.pop("h0")
    with pytest.raises(RuntimeError, match="nothing is launched"):
        api.selective_scan_step(**s)
    for k in ({"state": None}, {"state": _z(2, 64, 15)}, {"b": s["b"][:, :9]}, {"reset": _z(3, dtype=U8)}):
        with pytest.raises((ValueError, TypeError), match=next(iter(k))):
            api.selective_scan_step(**s | k)
    with pytest.raises(api.LrsError):
        api.selective_scan_workspace_bytes(2, 8, 64, 65)


def test_embedding_binding_refuses_by_name(stopped):
    t, w, dy = _z(5, dtype=torch.int64), _z(9, 64, dtype=BF), _z(5, 64, dtype=BF)
    with pytest.raises(RuntimeError, match="nothing is launched"):
        api.embedding_forward(t, w)
    with pytest.raises(RuntimeError, match="nothing is launched"):
        api.embedding_backward(dy, t, 9)
    for a in ((t.int(), w), (t, w.half()), (t, w[0]), (t, w.t()), (_z(5, 2, dtype=torch.int64)[:, 0], w)):
        with pytest.raises((ValueError, TypeError)):
            api.embedding_forward(*a)
    for a, k in (((dy.float(), t, 9), {}), ((dy, t[:4], 9), {}), ((dy, t, 9), {"accumulate": True}),
                 ((dy, t, 9), {"accumulate": True, "out": {"dw": _z(9, 64)}}), ((dy, t, 9), {"out": {"dw": _z(8, 64, dtype=BF)}}),
                 ((dy, t, 9), {"scratch": torch.empty(16, dtype=U8)})):
        with pytest.raises((ValueError, TypeError)):
            api.embedding_backward(*a, **k)
    for T, V, D in ((0, 9, 64), (5, 0, 64), (5, 9, 63)):
        with pytest.raises(api.LrsError):
            api.embedding_workspace_bytes(T, V, D)
