"""Thin Python binding over the C ABI in ``include/samu.h``.

Argument marshalling only: tensors are checked for dtype, device and
contiguity, their ``data_ptr()`` and the current CUDA stream are handed to the
shared library, and every step of the computation runs in its CUDA kernels.
There is no fallback: if ``liblrs_gb300.so`` is missing or fails to load, every
call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "liblrs_gb300.so"
_lock = threading.Lock()
_lib = None

LRS_GRAD_BF16 = 0
LRS_GRAD_FP32 = 1
LRS_TRANSITION_CHAINED = 0
LRS_TRANSITION_CLOSED_FORM = 1

# names and argument kinds of every exported symbol (checked by the tests)
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_D = ctypes.c_double
_SZP = ctypes.POINTER(ctypes.c_size_t)
_SIGNATURES = {
    "lrs_status_string": ([_I], ctypes.c_char_p),
    "samu_status_string": ([_I], ctypes.c_char_p),
    "lrs_version": ([], _I),
    "lrs_device_status": ([_P, ctypes.POINTER(_I), _P], _I),
    "lrs_selftest_wait_timeout": ([_P, _P], _I),
    "lrs_profile_begin": ([_I], _I),
    "lrs_profile_end": ([_P, _P, _I, ctypes.POINTER(_I)], _I),
    "samu_set_chunk_transition": ([_I], _I),
    "samu_get_chunk_transition": ([], _I),
    "samu_workspace_bytes": ([_I, _I, _I, _SZP, _SZP], _I),
    "samu_forward": ([_P] * 10 + [_I, _I, _I] + [_P] * 6, _I),
    "samu_backward": ([_P] * 12 + [_I, _I, _I] + [_P, _P, _P, _I] + [_P] * 9, _I),
    "samu_forward_noalloc": ([_P] * 10 + [_I, _I, _I] + [_P] * 4, _I),
    "samu_forward_noalloc_status": ([ctypes.POINTER(_I), _P], _I),
    "samu_decode_params_floats": ([_I, _SZP], _I),
    "samu_decode_prepare": ([_P] * 6 + [_I, _P, _P], _I),
    "samu_decode_step": ([_P] * 6 + [_I, _I, _P, _P, _P], _I),
    "rglru_workspace_bytes": ([_I, _I, _I, _SZP, _SZP], _I),
    "rglru_forward": ([_P] * 6 + [_I, _I, _I] + [_P] * 6, _I),
    "rglru_backward": ([_P] * 8 + [_I, _I, _I] + [_P] * 4 + [_I] + [_P] * 4, _I),
    "rglru_proj_workspace_bytes": ([_I, _I, _I, _SZP, _SZP], _I),
    "rglru_proj_forward": ([_P] * 8 + [_I, _I, _I] + [_P] * 6, _I),
    "rglru_proj_backward": ([_P] * 10 + [_I, _I, _I] + [_P] * 2 + [_I] + [_P] * 8, _I),
    "samu_block_workspace_bytes": ([_I] * 4 + [_SZP, _SZP], _I),
    "samu_block_forward": ([_P] * 4 + [_I] * 4 + [_P] * 5, _I),
    "samu_block_backward": ([_P] * 6 + [_I] * 4 + [_P] * 6, _I),
    "lrs_dense_gemm": ([_I, _P, _P, _P, _I, _I, _I, _P, _P], _I),
    "rglru_block_workspace_bytes": ([_I] * 4 + [_SZP, _SZP], _I),
    "rglru_block_forward": ([_P] * 4 + [_I] * 4 + [_P] * 5, _I),
    "rglru_block_backward": ([_P] * 6 + [_I] * 4 + [_P] * 6, _I),
    "linear_ce_workspace_bytes": ([_I] * 4 + [_SZP, _SZP], _I),
    "linear_ce_forward": ([_P] * 3 + [_I] * 3 + [_F] + [_P] * 5, _I),
    "linear_ce_backward": ([_P] * 6 + [_I] * 3 + [_F] + [_P] * 2 + [_I] + [_P] * 2, _I),
    "gated_norm_workspace_bytes": ([_I, _I, _SZP, _SZP], _I),
    "gated_norm_forward": ([_P] * 6 + [_I, _I, _F] + [_P] * 4, _I),
    "gated_norm_backward": ([_P] * 8 + [_I, _I, _F] + [_P] * 9, _I),
    "lrs_adamw_scratch_bytes": ([_I, _SZP], _I),
    "lrs_adamw_step": ([_P, _I, _P, _P, _D, _D, _F, _F] + [_P] * 3, _I),
}

# samu_block_params / samu_block_grads (include/samu.h): one pointer per field, in order
BLOCK_PARAMS = ("gamma1", "w_in", "conv_k", "conv_b", "nu", "theta", "w_phi", "w_r", "a_phi", "a_r",
                "w_o", "gamma2", "w_mlp_in", "w_mlp_out")


class _BlockParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in BLOCK_PARAMS]


class _BlockGrads(ctypes.Structure):
    _fields_ = [("d" + n, ctypes.c_void_p) for n in BLOCK_PARAMS]


# rglru_block_params / rglru_block_grads: the block around the RG-LRU mixer
RGLRU_BLOCK_PARAMS = ("gamma1", "w_in", "conv_k", "conv_b", "w_x", "b_x", "w_a", "b_a", "alpha",
                      "w_o", "gamma2", "w_mlp_in", "w_mlp_out")


class _RgBlockParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in RGLRU_BLOCK_PARAMS]


class _RgBlockGrads(ctypes.Structure):
    _fields_ = [("d" + n, ctypes.c_void_p) for n in RGLRU_BLOCK_PARAMS]


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def _load():
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{_LIB_NAME} is not built ({path}); run __graft_entry__.build() first")
            lib = ctypes.CDLL(path)
            for name, (argtypes, restype) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = argtypes
                fn.restype = restype
            _lib = lib
    return _lib


class LrsError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = _load().lrs_status_string(status).decode()
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


def _check(fn: str, status: int):
    if status != 0:
        raise LrsError(fn, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    index = getattr(device, "index", None)
    if index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return torch._C._cuda_getCurrentRawStream(index)   # the same handle, without building a Stream object


def _need(t, name, dtype, device, shape=None):
    if t is not None and t.dtype is dtype and t.device == device and t.is_contiguous() and (
            shape is None or t.shape == shape):
        return t
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _opt(t, name, dtype, device, shape=None):
    return None if t is None else _need(t, name, dtype, device, shape)


def _buffer(t, name, nbytes, device):
    """t as a caller's buffer of at least nbytes on the device; allocated where t is None."""
    if t is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if t.device != device:
        raise ValueError(f"{name}: expected a buffer on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous buffer")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} buffer is too small: {t.numel() * t.element_size()} bytes of {nbytes}")
    return t


def _saved(t, nbytes, device):
    """The forward's saved buffer, handed to a backward."""
    if t is None:
        raise ValueError("saved must be the forward's saved buffer")
    return _buffer(t, "saved", nbytes, device)


def _like(t, out, key):
    """An output of t's shape and type (cheaper to allocate than by its shape)."""
    if out is None or out.get(key) is None:
        return torch.empty_like(t)
    return _need(out[key], key, t.dtype, t.device, t.shape)


def _empty(shape, dtype, device, out, key):
    if out is None or out.get(key) is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _need(out[key], key, dtype, device, shape)


# ---------------------------------------------------------------------------
# SAMU
# ---------------------------------------------------------------------------
def samu_workspace_bytes(B: int, L: int, D: int):
    lib = _load()
    s = ctypes.c_size_t(0)
    c = ctypes.c_size_t(0)
    _check("samu_workspace_bytes", lib.samu_workspace_bytes(B, L, D, ctypes.byref(s), ctypes.byref(c)))
    return int(s.value), int(c.value)


def samu_forward(x_sel, w, h0, reset, nu, theta, w_phi, w_r, a_phi, a_r, *, want_y32=False,
                 out=None, saved=None, scratch=None):
    """SAMU mixer forward through ``samu_forward``.  Returns dict(y, y32, hT, saved, scratch)."""
    dev = x_sel.device
    B, L, D = x_sel.shape
    M = D // 2
    _need(x_sel, "x_sel", torch.bfloat16, dev)
    _need(w, "w", torch.bfloat16, dev, (B, L, D))
    _opt(h0, "h0", torch.float32, dev, (B, M, 2))
    _opt(reset, "reset", torch.uint8, dev, (B, L))
    _need(nu, "nu", torch.float32, dev, (M,))
    _need(theta, "theta", torch.float32, dev, (M,))
    _need(w_phi, "w_phi", torch.float32, dev, (D + 1,))
    _need(w_r, "w_r", torch.float32, dev, (D + 1,))
    _need(a_phi, "a_phi", torch.float32, dev, (1,))
    _need(a_r, "a_r", torch.float32, dev, (1,))
    nsaved, nscratch = samu_workspace_bytes(B, L, D)
    y = _empty((B, L, D), torch.bfloat16, dev, out, "y")
    y32 = _empty((B, L, D), torch.float32, dev, out, "y32") if want_y32 else None
    hT = _empty((B, M, 2), torch.float32, dev, out, "hT")
    saved = _buffer(saved, "saved", nsaved, dev)
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    st = _load().samu_forward(_ptr(x_sel), _ptr(w), _ptr(h0), _ptr(reset), _ptr(nu), _ptr(theta),
                              _ptr(w_phi), _ptr(w_r), _ptr(a_phi), _ptr(a_r), B, L, D,
                              _ptr(y), _ptr(y32), _ptr(hT), _ptr(saved), _ptr(scratch), _stream(dev))
    _check("samu_forward", st)
    return {"y": y, "y32": y32, "hT": hT, "saved": saved, "scratch": scratch}


def samu_backward(dy, dhT, x_sel, w, h0, reset, nu, theta, w_phi, w_r, a_phi, a_r, saved, *,
                  grad_fp32=False, out=None, scratch=None):
    """SAMU mixer backward through ``samu_backward``.

    Returns dict(dx_sel, dw, dh0, dnu, dtheta, dw_phi, dw_r, da_phi, da_r, scratch).
    """
    dev = x_sel.device
    B, L, D = x_sel.shape
    M = D // 2
    _need(dy, "dy", torch.bfloat16, dev, (B, L, D))
    _opt(dhT, "dhT", torch.float32, dev, (B, M, 2))
    _need(x_sel, "x_sel", torch.bfloat16, dev)
    _need(w, "w", torch.bfloat16, dev, (B, L, D))
    _opt(reset, "reset", torch.uint8, dev, (B, L))
    nsaved, nscratch = samu_workspace_bytes(B, L, D)
    _saved(saved, nsaved, dev)
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    gdt = torch.float32 if grad_fp32 else torch.bfloat16
    o = {
        "dx_sel": _empty((B, L, D), gdt, dev, out, "dx_sel"),
        "dw": _empty((B, L, D), gdt, dev, out, "dw"),
        "dh0": _empty((B, M, 2), torch.float32, dev, out, "dh0"),
        "dnu": _empty((M,), torch.float32, dev, out, "dnu"),
        "dtheta": _empty((M,), torch.float32, dev, out, "dtheta"),
        "dw_phi": _empty((D + 1,), torch.float32, dev, out, "dw_phi"),
        "dw_r": _empty((D + 1,), torch.float32, dev, out, "dw_r"),
        "da_phi": _empty((1,), torch.float32, dev, out, "da_phi"),
        "da_r": _empty((1,), torch.float32, dev, out, "da_r"),
    }
    st = _load().samu_backward(_ptr(dy), _ptr(dhT), _ptr(x_sel), _ptr(w), _ptr(h0), _ptr(reset), _ptr(nu),
                               _ptr(theta), _ptr(w_phi), _ptr(w_r), _ptr(a_phi), _ptr(a_r), B, L, D,
                               _ptr(saved), _ptr(o["dx_sel"]), _ptr(o["dw"]),
                               LRS_GRAD_FP32 if grad_fp32 else LRS_GRAD_BF16,
                               _ptr(o["dh0"]), _ptr(o["dnu"]), _ptr(o["dtheta"]), _ptr(o["dw_phi"]),
                               _ptr(o["dw_r"]), _ptr(o["da_phi"]), _ptr(o["da_r"]), _ptr(scratch), _stream(dev))
    _check("samu_backward", st)
    o["scratch"] = scratch
    return o


def samu_forward_noalloc(x_sel, w, h0, reset, nu, theta, w_phi, w_r, a_phi, a_r, *, want_y32=False,
                         out=None):
    """SAMU forward through ``samu_forward_noalloc``: for callers that cannot
    allocate device memory for the workspace, the library keeps its
    intermediates in one fixed device array (LRS_NOALLOC_BYTES, shared by all
    calls on a device; calls that overlap on the GPU race).  Outputs are still
    caller-provided (``out``) or allocated here by torch.  Returns dict(y, y32, hT)."""
    dev = x_sel.device
    B, L, D = x_sel.shape
    M = D // 2
    _need(x_sel, "x_sel", torch.bfloat16, dev)
    _need(w, "w", torch.bfloat16, dev, (B, L, D))
    _opt(h0, "h0", torch.float32, dev, (B, M, 2))
    _opt(reset, "reset", torch.uint8, dev, (B, L))
    _need(nu, "nu", torch.float32, dev, (M,))
    _need(theta, "theta", torch.float32, dev, (M,))
    _need(w_phi, "w_phi", torch.float32, dev, (D + 1,))
    _need(w_r, "w_r", torch.float32, dev, (D + 1,))
    _need(a_phi, "a_phi", torch.float32, dev, (1,))
    _need(a_r, "a_r", torch.float32, dev, (1,))
    y = _empty((B, L, D), torch.bfloat16, dev, out, "y")
    y32 = _empty((B, L, D), torch.float32, dev, out, "y32") if want_y32 else None
    hT = _empty((B, M, 2), torch.float32, dev, out, "hT")
    st = _load().samu_forward_noalloc(_ptr(x_sel), _ptr(w), _ptr(h0), _ptr(reset), _ptr(nu), _ptr(theta),
                                      _ptr(w_phi), _ptr(w_r), _ptr(a_phi), _ptr(a_r), B, L, D,
                                      _ptr(y), _ptr(y32), _ptr(hT), _stream(dev))
    _check("samu_forward_noalloc", st)
    return {"y": y, "y32": y32, "hT": hT}


def samu_set_chunk_transition(kind: int) -> None:
    """Process-wide form of the SAMU maps kernels' item transitions
    (LRS_TRANSITION_CHAINED or LRS_TRANSITION_CLOSED_FORM) for later calls."""
    _check("samu_set_chunk_transition", _load().samu_set_chunk_transition(int(kind)))


def samu_get_chunk_transition() -> int:
    return int(_load().samu_get_chunk_transition())


# ---------------------------------------------------------------------------
# SAMU decode step
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def samu_decode_params_floats(D: int) -> int:
    n = ctypes.c_size_t(0)
    _check("samu_decode_params_floats", _load().samu_decode_params_floats(D, ctypes.byref(n)))
    return int(n.value)


def samu_decode_prepare(nu, theta, w_phi, w_r, a_phi, a_r, *, params=None):
    """Per-parameter part of the decode step through ``samu_decode_prepare``.  Returns the parameter block."""
    dev = nu.device
    M = nu.shape[0]
    D = 2 * M
    _need(nu, "nu", torch.float32, dev, (M,))
    _need(theta, "theta", torch.float32, dev, (M,))
    _need(w_phi, "w_phi", torch.float32, dev, (D + 1,))
    _need(w_r, "w_r", torch.float32, dev, (D + 1,))
    _need(a_phi, "a_phi", torch.float32, dev, (1,))
    _need(a_r, "a_r", torch.float32, dev, (1,))
    n = samu_decode_params_floats(D)
    params = torch.empty(n, dtype=torch.float32, device=dev) if params is None else _buffer(params, "params", 4 * n, dev)
    _check("samu_decode_prepare", _load().samu_decode_prepare(_ptr(nu), _ptr(theta), _ptr(w_phi), _ptr(w_r),
                                                             _ptr(a_phi), _ptr(a_r), D, _ptr(params), _stream(dev)))
    return params


def samu_decode_step(x_sel, w, state, params, reset=None, *, state_out=None, want_y32=False, out=None):
    """One token of each of B sequences through ``samu_decode_step``.  x_sel, w: [B,D] BF16; state: [B,M,2] FP32.

    state_out defaults to ``state`` (updated in place).  Returns dict(y, y32, state)."""
    dev = x_sel.device
    B, D = x_sel.shape
    M = D // 2
    _need(x_sel, "x_sel", torch.bfloat16, dev)
    _need(w, "w", torch.bfloat16, dev, (B, D))
    _need(state, "state", torch.float32, dev, (B, M, 2))
    _opt(reset, "reset", torch.uint8, dev, (B,))
    if params is not None:
        _buffer(params, "params", 4 * samu_decode_params_floats(D), dev)
    so = state if state_out is None else state_out
    _need(so, "state_out", torch.float32, dev, (B, M, 2))
    y = _empty((B, D), torch.bfloat16, dev, out, "y")
    y32 = _empty((B, D), torch.float32, dev, out, "y32") if want_y32 else None
    _check("samu_decode_step", _load().samu_decode_step(_ptr(x_sel), _ptr(w), _ptr(state), _ptr(so), _ptr(reset),
                                                       _ptr(params), B, D, _ptr(y), _ptr(y32), _stream(dev)))
    return {"y": y, "y32": y32, "state": so}


# ---------------------------------------------------------------------------
# RG-LRU
# ---------------------------------------------------------------------------
def rglru_workspace_bytes(B: int, L: int, D: int):
    lib = _load()
    s = ctypes.c_size_t(0)
    c = ctypes.c_size_t(0)
    _check("rglru_workspace_bytes", lib.rglru_workspace_bytes(B, L, D, ctypes.byref(s), ctypes.byref(c)))
    return int(s.value), int(c.value)


def rglru_forward(x, lx, la, alpha, h0, reset, *, want_y32=False, out=None, saved=None, scratch=None):
    """RG-LRU forward through ``rglru_forward``.  Returns dict(y, y32, hT, saved, scratch)."""
    dev = x.device
    B, L, D = x.shape
    _need(x, "x", torch.bfloat16, dev)
    _need(lx, "lx", torch.bfloat16, dev, (B, L, D))
    _need(la, "la", torch.bfloat16, dev, (B, L, D))
    _need(alpha, "alpha", torch.float32, dev, (D,))
    _opt(h0, "h0", torch.float32, dev, (B, D))
    _opt(reset, "reset", torch.uint8, dev, (B, L))
    nsaved, nscratch = rglru_workspace_bytes(B, L, D)
    y = _empty((B, L, D), torch.bfloat16, dev, out, "y")
    y32 = _empty((B, L, D), torch.float32, dev, out, "y32") if want_y32 else None
    hT = _empty((B, D), torch.float32, dev, out, "hT")
    saved = _buffer(saved, "saved", nsaved, dev)
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    st = _load().rglru_forward(_ptr(x), _ptr(lx), _ptr(la), _ptr(alpha), _ptr(h0), _ptr(reset), B, L, D,
                               _ptr(y), _ptr(y32), _ptr(hT), _ptr(saved), _ptr(scratch), _stream(dev))
    _check("rglru_forward", st)
    return {"y": y, "y32": y32, "hT": hT, "saved": saved, "scratch": scratch}


def rglru_backward(dy, dhT, x, lx, la, alpha, h0, reset, saved, *, grad_fp32=False, out=None, scratch=None):
    """RG-LRU backward through ``rglru_backward``.  Returns dict(dx, dlx, dla, dalpha, dh0, scratch)."""
    dev = x.device
    B, L, D = x.shape
    _need(dy, "dy", torch.bfloat16, dev, (B, L, D))
    _opt(dhT, "dhT", torch.float32, dev, (B, D))
    nsaved, nscratch = rglru_workspace_bytes(B, L, D)
    _saved(saved, nsaved, dev)
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    gdt = torch.float32 if grad_fp32 else torch.bfloat16
    o = {
        "dx": _empty((B, L, D), gdt, dev, out, "dx"),
        "dlx": _empty((B, L, D), gdt, dev, out, "dlx"),
        "dla": _empty((B, L, D), gdt, dev, out, "dla"),
        "dalpha": _empty((D,), torch.float32, dev, out, "dalpha"),
        "dh0": _empty((B, D), torch.float32, dev, out, "dh0"),
    }
    st = _load().rglru_backward(_ptr(dy), _ptr(dhT), _ptr(x), _ptr(lx), _ptr(la), _ptr(alpha), _ptr(h0),
                                _ptr(reset), B, L, D, _ptr(saved), _ptr(o["dx"]), _ptr(o["dlx"]), _ptr(o["dla"]),
                                LRS_GRAD_FP32 if grad_fp32 else LRS_GRAD_BF16,
                                _ptr(o["dalpha"]), _ptr(o["dh0"]), _ptr(scratch), _stream(dev))
    _check("rglru_backward", st)
    o["scratch"] = scratch
    return o


# ---------------------------------------------------------------------------
# RG-LRU with its block-diagonal gate projections
# ---------------------------------------------------------------------------
PROJ_BLOCKS = 16


def rglru_proj_workspace_bytes(B: int, L: int, D: int):
    lib = _load()
    s = ctypes.c_size_t(0)
    c = ctypes.c_size_t(0)
    _check("rglru_proj_workspace_bytes", lib.rglru_proj_workspace_bytes(B, L, D, ctypes.byref(s), ctypes.byref(c)))
    return int(s.value), int(c.value)


def _proj_params(x, w_x, b_x, w_a, b_a, alpha):
    dev = x.device
    B, L, D = x.shape
    dk = D // PROJ_BLOCKS
    _need(x, "x", torch.bfloat16, dev)
    for t, n in ((w_x, "w_x"), (w_a, "w_a")):
        _need(t, n, torch.bfloat16, dev, (PROJ_BLOCKS, dk, dk))
    for t, n in ((b_x, "b_x"), (b_a, "b_a"), (alpha, "alpha")):
        _need(t, n, torch.float32, dev, (D,))
    return dev, B, L, D, dk


def rglru_proj_forward(x, w_x, b_x, w_a, b_a, alpha, h0, reset, *, want_y32=False, out=None, saved=None,
                       scratch=None):
    """RG-LRU forward with the block-diagonal gate projections (``rglru_proj_forward``).
    Returns dict(y, y32, hT, saved, scratch)."""
    dev, B, L, D, dk = _proj_params(x, w_x, b_x, w_a, b_a, alpha)
    _opt(h0, "h0", torch.float32, dev, (B, D))
    _opt(reset, "reset", torch.uint8, dev, (B, L))
    nsaved, nscratch = rglru_proj_workspace_bytes(B, L, D)
    y = _empty((B, L, D), torch.bfloat16, dev, out, "y")
    y32 = _empty((B, L, D), torch.float32, dev, out, "y32") if want_y32 else None
    hT = _empty((B, D), torch.float32, dev, out, "hT")
    saved = _buffer(saved, "saved", nsaved, dev)
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    st = _load().rglru_proj_forward(_ptr(x), _ptr(w_x), _ptr(b_x), _ptr(w_a), _ptr(b_a), _ptr(alpha), _ptr(h0),
                                    _ptr(reset), B, L, D, _ptr(y), _ptr(y32), _ptr(hT), _ptr(saved), _ptr(scratch),
                                    _stream(dev))
    _check("rglru_proj_forward", st)
    return {"y": y, "y32": y32, "hT": hT, "saved": saved, "scratch": scratch}


def rglru_proj_backward(dy, dhT, x, w_x, b_x, w_a, b_a, alpha, h0, reset, saved, *, grad_fp32=False, out=None,
                        scratch=None):
    """Backward of rglru_proj_forward (``rglru_proj_backward``).
    Returns dict(dx, dw_x, db_x, dw_a, db_a, dalpha, dh0, scratch)."""
    dev, B, L, D, dk = _proj_params(x, w_x, b_x, w_a, b_a, alpha)
    _need(dy, "dy", torch.bfloat16, dev, (B, L, D))
    _opt(dhT, "dhT", torch.float32, dev, (B, D))
    nsaved, nscratch = rglru_proj_workspace_bytes(B, L, D)
    _saved(saved, nsaved, dev)
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    o = {
        "dx": _empty((B, L, D), torch.float32 if grad_fp32 else torch.bfloat16, dev, out, "dx"),
        "dw_x": _empty((PROJ_BLOCKS, dk, dk), torch.float32, dev, out, "dw_x"),
        "db_x": _empty((D,), torch.float32, dev, out, "db_x"),
        "dw_a": _empty((PROJ_BLOCKS, dk, dk), torch.float32, dev, out, "dw_a"),
        "db_a": _empty((D,), torch.float32, dev, out, "db_a"),
        "dalpha": _empty((D,), torch.float32, dev, out, "dalpha"),
        "dh0": _empty((B, D), torch.float32, dev, out, "dh0"),
    }
    st = _load().rglru_proj_backward(_ptr(dy), _ptr(dhT), _ptr(x), _ptr(w_x), _ptr(b_x), _ptr(w_a), _ptr(b_a),
                                     _ptr(alpha), _ptr(h0), _ptr(reset), B, L, D, _ptr(saved), _ptr(o["dx"]),
                                     LRS_GRAD_FP32 if grad_fp32 else LRS_GRAD_BF16, _ptr(o["dw_x"]), _ptr(o["db_x"]),
                                     _ptr(o["dw_a"]), _ptr(o["db_a"]), _ptr(o["dalpha"]), _ptr(o["dh0"]),
                                     _ptr(scratch), _stream(dev))
    _check("rglru_proj_backward", st)
    o["scratch"] = scratch
    return o


# ---------------------------------------------------------------------------
# One RecurrentBlock around the SAMU mixer
# ---------------------------------------------------------------------------
def samu_block_workspace_bytes(B: int, L: int, Dm: int, D: int, mixer: str = "samu"):
    lib = _load()
    s = ctypes.c_size_t(0)
    c = ctypes.c_size_t(0)
    fn = "samu_block_workspace_bytes" if mixer == "samu" else "rglru_block_workspace_bytes"
    _check(fn, getattr(lib, fn)(B, L, Dm, D, ctypes.byref(s), ctypes.byref(c)))
    return int(s.value), int(c.value)


def _block_shapes(Dm: int, D: int) -> dict:
    M, F, dk = D // 2, 3 * Dm, D // PROJ_BLOCKS
    return {"gamma1": (Dm,), "w_in": (2 * D, Dm), "conv_k": (4, D), "conv_b": (D,), "nu": (M,), "theta": (M,),
            "w_phi": (D + 1,), "w_r": (D + 1,), "a_phi": (1,), "a_r": (1,), "w_o": (Dm, D), "gamma2": (Dm,),
            "w_mlp_in": (2 * F, Dm), "w_mlp_out": (Dm, F), "w_x": (PROJ_BLOCKS, dk, dk), "b_x": (D,),
            "w_a": (PROJ_BLOCKS, dk, dk), "b_a": (D,), "alpha": (D,)}


_BLOCK_BF16 = ("w_in", "w_o", "w_mlp_in", "w_mlp_out", "w_x", "w_a")


def _block_kind(params: dict):
    """(mixer, names, params struct, grads struct, D) of a parameter dict."""
    if "nu" in params:
        return "samu", BLOCK_PARAMS, _BlockParams, _BlockGrads, 2 * params["nu"].numel()
    return "rglru", RGLRU_BLOCK_PARAMS, _RgBlockParams, _RgBlockGrads, params["alpha"].numel()


def _block_params(params: dict, Dm: int, dev):
    mixer, names, Struct, _, D = _block_kind(params)
    shapes = _block_shapes(Dm, D)
    st = Struct()
    for n in names:
        dt = torch.bfloat16 if n in _BLOCK_BF16 else torch.float32
        setattr(st, n, _need(params.get(n), n, dt, dev, shapes[n]).data_ptr())
    return st


def _state_shape(mixer, B, D):
    return (B, D // 2, 2) if mixer == "samu" else (B, D)


def samu_block_forward(x, params: dict, h0=None, reset=None, *, out=None, saved=None, scratch=None):
    """One RecurrentBlock forward through ``samu_block_forward`` (params with
    the SAMU mixer's nu, theta, ...) or ``rglru_block_forward`` (params with
    the RG-LRU mixer's w_x, b_x, w_a, b_a, alpha).  x: [B,L,Dm] BF16.
    Returns dict(out, hT, saved, scratch)."""
    dev = x.device
    B, L, Dm = x.shape
    _need(x, "x", torch.bfloat16, dev)
    mixer, _, _, _, D = _block_kind(params)
    sshape = _state_shape(mixer, B, D)
    _opt(h0, "h0", torch.float32, dev, sshape)
    _opt(reset, "reset", torch.uint8, dev, (B, L))
    ps = _block_params(params, Dm, dev)
    nsaved, nscratch = samu_block_workspace_bytes(B, L, Dm, D, mixer)
    y = _empty((B, L, Dm), torch.bfloat16, dev, out, "out")
    hT = _empty(sshape, torch.float32, dev, out, "hT")
    saved = _buffer(saved, "saved", nsaved, dev)
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    fn = "samu_block_forward" if mixer == "samu" else "rglru_block_forward"
    st = getattr(_load(), fn)(ctypes.cast(ctypes.pointer(ps), _P), _ptr(x), _ptr(h0), _ptr(reset), B, L, Dm, D,
                              _ptr(y), _ptr(hT), _ptr(saved), _ptr(scratch), _stream(dev))
    _check(fn, st)
    return {"out": y, "hT": hT, "saved": saved, "scratch": scratch}


def samu_block_backward(dout, dhT, x, params: dict, h0, reset, saved, *, out=None, scratch=None):
    """Backward of samu_block_forward (either mixer).  Returns dict(dx, dh0,
    d<param> for every parameter (FP32, the parameter's shape), scratch)."""
    dev = x.device
    B, L, Dm = x.shape
    mixer, names, _, Grads, D = _block_kind(params)
    sshape = _state_shape(mixer, B, D)
    _need(dout, "dout", torch.bfloat16, dev, (B, L, Dm))
    _opt(dhT, "dhT", torch.float32, dev, sshape)
    _opt(reset, "reset", torch.uint8, dev, (B, L))
    ps = _block_params(params, Dm, dev)
    nsaved, nscratch = samu_block_workspace_bytes(B, L, Dm, D, mixer)
    _saved(saved, nsaved, dev)
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    shapes = _block_shapes(Dm, D)
    o = {"dx": _empty((B, L, Dm), torch.bfloat16, dev, out, "dx"),
         "dh0": _empty(sshape, torch.float32, dev, out, "dh0")}
    gs = Grads()
    for n in names:
        o["d" + n] = _empty(shapes[n], torch.float32, dev, out, "d" + n)
        setattr(gs, "d" + n, o["d" + n].data_ptr())
    fn = "samu_block_backward" if mixer == "samu" else "rglru_block_backward"
    st = getattr(_load(), fn)(ctypes.cast(ctypes.pointer(ps), _P), _ptr(x), _ptr(h0), _ptr(reset), _ptr(dout),
                              _ptr(dhT), B, L, Dm, D, _ptr(saved), _ptr(o["dx"]), _ptr(o["dh0"]),
                              ctypes.cast(ctypes.pointer(gs), _P), _ptr(scratch), _stream(dev))
    _check(fn, st)
    o["scratch"] = scratch
    return o


LRS_GEMM_NT, LRS_GEMM_NN, LRS_GEMM_TN = 0, 1, 2


def dense_gemm(layout: int, A, B, M: int, N: int, K: int, *, out=None, scratch=None):
    """The block's tensor-core contraction on its own (``lrs_dense_gemm``):
    NT: C[M,N] = A[M,K] B[N,K]^T (BF16); NN: C = A[M,K] B[K,N] (BF16);
    TN: C[M,N] = A[K,M]^T B[K,N] (FP32)."""
    dev = A.device
    _need(A, "A", torch.bfloat16, dev, (K, M) if layout == LRS_GEMM_TN else (M, K))
    _need(B, "B", torch.bfloat16, dev, (N, K) if layout == LRS_GEMM_NT else (K, N))
    dt = torch.float32 if layout == LRS_GEMM_TN else torch.bfloat16
    C = out if out is not None else torch.empty((M, N), dtype=dt, device=dev)
    _need(C, "C", dt, dev, (M, N))
    scratch = _buffer(scratch, "scratch", 256, dev)
    _check("lrs_dense_gemm", _load().lrs_dense_gemm(layout, _ptr(A), _ptr(B), _ptr(C), M, N, K, _ptr(scratch),
                                                    _stream(dev)))
    return C


# ---------------------------------------------------------------------------
# Softmax cross entropy over a vocabulary
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def linear_ce_workspace_bytes(T: int, V: int, D: int, grad_fp32: bool = False):
    """(forward, backward) scratch bytes of the vocabulary loss."""
    f = ctypes.c_size_t(0)
    b = ctypes.c_size_t(0)
    _check("linear_ce_workspace_bytes",
           _load().linear_ce_workspace_bytes(T, V, D, LRS_GRAD_FP32 if grad_fp32 else LRS_GRAD_BF16, ctypes.byref(f),
                                             ctypes.byref(b)))
    return int(f.value), int(b.value)


def _ce_inputs(h, w, target):
    dev, shape = h.device, h.shape
    V, D = w.shape
    if not shape or shape[-1] != D:
        raise ValueError(f"h: expected shape (..., {D}), got {tuple(shape)}")
    _need(h, "h", torch.bfloat16, dev)
    _need(w, "w", torch.bfloat16, dev)
    _need(target, "target", torch.int64, dev, shape[:-1])
    return dev, target.numel(), V, D


def linear_ce_forward(h, w, target, *, softcap=0.0, out=None, scratch=None):
    """Softmax cross entropy of the logits h w^T through ``linear_ce_forward``.

    h: [..., D] BF16, w: [V, D] BF16, target: [...] int64 (negative: not counted); softcap c > 0 caps the logits
    to c tanh(z / c).  Returns dict(loss, lse (h's leading shape, FP32), total ([sum of losses, tokens counted]),
    scratch)."""
    dev, T, V, D = _ce_inputs(h, w, target)
    nscratch = linear_ce_workspace_bytes(T, V, D)[0]
    shape = target.shape
    loss = _empty(shape, torch.float32, dev, out, "loss")
    lse = _like(loss, out, "lse")
    total = _empty((2,), torch.float32, dev, out, "total")
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    st = _load().linear_ce_forward(h.data_ptr(), w.data_ptr(), target.data_ptr(), T, V, D, softcap, loss.data_ptr(),
                                   lse.data_ptr(), total.data_ptr(), scratch.data_ptr(), _stream(dev))
    if st:
        _check("linear_ce_forward", st)
    return {"loss": loss, "lse": lse, "total": total, "scratch": scratch}


def linear_ce_backward(h, w, target, lse, dloss=None, *, total=None, softcap=0.0, grad_fp32=False, out=None,
                       scratch=None):
    """Backward of linear_ce_forward (``linear_ce_backward``).

    dloss: [...] FP32 cotangents of the losses, or None for their mean over the tokens counted (then ``total`` is
    the forward's).  Returns dict(dh, dw, scratch), BF16 or (grad_fp32) FP32."""
    dev, T, V, D = _ce_inputs(h, w, target)
    _need(lse, "lse", torch.float32, dev, target.shape)
    _opt(dloss, "dloss", torch.float32, dev, target.shape)
    _opt(total, "total", torch.float32, dev, (2,))
    if dloss is None and total is None:
        raise ValueError("total is required where dloss is None")
    if dloss is not None and dloss.data_ptr() % 16:
        dloss = dloss.clone()   # a view such as weights[1:]; the entry takes 16-byte alignment
    nscratch = linear_ce_workspace_bytes(T, V, D, grad_fp32)[1]
    if grad_fp32:
        dh = _empty(h.shape, torch.float32, dev, out, "dh")
        dw = _empty(w.shape, torch.float32, dev, out, "dw")
    else:
        dh, dw = _like(h, out, "dh"), _like(w, out, "dw")
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    st = _load().linear_ce_backward(h.data_ptr(), w.data_ptr(), target.data_ptr(), lse.data_ptr(), _ptr(dloss),
                                    _ptr(total), T, V, D, softcap, dh.data_ptr(), dw.data_ptr(),
                                    LRS_GRAD_FP32 if grad_fp32 else LRS_GRAD_BF16, scratch.data_ptr(), _stream(dev))
    if st:
        _check("linear_ce_backward", st)
    return {"dh": dh, "dw": dw, "scratch": scratch}


# ---------------------------------------------------------------------------
# Norms before and after a residual branch, with its gate and scale
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def gated_norm_workspace_bytes(T: int, D: int):
    s = ctypes.c_size_t(0)
    c = ctypes.c_size_t(0)
    _check("gated_norm_workspace_bytes",
           _load().gated_norm_workspace_bytes(T, D, ctypes.byref(s), ctypes.byref(c)))
    return int(s.value), int(c.value)


def _gated_norm_inputs(x, y, gate, gamma_post, scale, gamma_pre):
    dev, shape = x.device, x.shape
    if not shape:
        raise ValueError("x: expected shape (..., D)")
    D = shape[-1]
    _need(x, "x", torch.bfloat16, dev)
    if y is not None:
        _need(y, "y", torch.bfloat16, dev, shape)
    if gate is not None:
        _need(gate, "gate", torch.bfloat16, dev, shape)
    vector = (D,)
    if gamma_post is not None:
        _need(gamma_post, "gamma_post", torch.float32, dev, vector)
    if scale is not None:
        _need(scale, "scale", torch.float32, dev, vector)
    if gamma_pre is not None:
        _need(gamma_pre, "gamma_pre", torch.float32, dev, vector)
    return dev, x.numel() // D if D else 0, D


def gated_norm_forward(x, y=None, gate=None, gamma_post=None, scale=None, gamma_pre=None, *, eps=1e-6, out=None,
                       saved=None):
    """r = x + scale GeLU(gate) RMSNorm(y; gamma_post), h = RMSNorm(r; gamma_pre) through ``gated_norm_forward``.

    x, y, gate: [..., D] BF16; the vectors [D] FP32; anything but x may be None (no gate, ones; without y no branch:
    h = RMSNorm(x; gamma_pre) and r is x itself).  Returns dict(r, h, saved)."""
    dev, T, D = _gated_norm_inputs(x, y, gate, gamma_post, scale, gamma_pre)
    nsaved, _ = gated_norm_workspace_bytes(T, D)
    r = _like(x, out, "r") if y is not None else None
    h = _like(x, out, "h")
    saved = _buffer(saved, "saved", nsaved, dev)
    st = _load().gated_norm_forward(x.data_ptr(), _ptr(y), _ptr(gate), _ptr(gamma_post), _ptr(scale), _ptr(gamma_pre),
                                    T, D, eps, _ptr(r), h.data_ptr(), saved.data_ptr(), _stream(dev))
    if st:
        _check("gated_norm_forward", st)
    return {"r": x if y is None else r, "h": h, "saved": saved}


def gated_norm_backward(dr, dh, x, y, gate, gamma_post, scale, gamma_pre, saved, *, eps=1e-6, out=None, scratch=None):
    """Backward of gated_norm_forward (``gated_norm_backward``).  dr may be None (zero).

    Returns dict(dx, dy, dgate, dgamma_post, dscale, dgamma_pre, scratch); dy, dgamma_post, dscale are None without a
    branch, dgate without a gate."""
    dev, T, D = _gated_norm_inputs(x, y, gate, gamma_post, scale, gamma_pre)
    _opt(dr, "dr", torch.bfloat16, dev, x.shape)
    _need(dh, "dh", torch.bfloat16, dev, x.shape)
    nsaved, nscratch = gated_norm_workspace_bytes(T, D)
    _saved(saved, nsaved, dev)
    scratch = _buffer(scratch, "scratch", nscratch, dev)
    o = {"dx": _like(x, out, "dx"), "dy": None, "dgate": None, "dgamma_post": None,
         "dscale": None, "dgamma_pre": _empty((D,), torch.float32, dev, out, "dgamma_pre")}
    if y is not None:
        o["dy"] = _like(x, out, "dy")
        o["dgamma_post"] = _empty((D,), torch.float32, dev, out, "dgamma_post")
        o["dscale"] = _empty((D,), torch.float32, dev, out, "dscale")
    if gate is not None:
        o["dgate"] = _like(x, out, "dgate")
    _check("gated_norm_backward",
           _load().gated_norm_backward(_ptr(dr), _ptr(dh), _ptr(x), _ptr(y), _ptr(gate), _ptr(gamma_post), _ptr(scale),
                                       _ptr(gamma_pre), T, D, eps, _ptr(saved), _ptr(o["dx"]), _ptr(o["dy"]),
                                       _ptr(o["dgate"]), _ptr(o["dgamma_post"]), _ptr(o["dscale"]),
                                       _ptr(o["dgamma_pre"]), _ptr(scratch), _stream(dev)))
    o["scratch"] = scratch
    return o


# ---------------------------------------------------------------------------
# AdamW over many tensors
# ---------------------------------------------------------------------------
class _AdamwTensor(ctypes.Structure):
    """lrs_adamw_tensor (include/samu.h)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + \
        [("n", ctypes.c_int64), ("weight_decay", ctypes.c_float), ("grad_dtype", ctypes.c_int)]


ADAMW_BLOCK = 256   # values that share one scale of an 8-bit state


def adamw_state(param, bits: int = 32) -> dict:
    """Zeroed state of one tensor: {"m", "v"} in FP32, or (bits = 8) E4M3 codes with {"m_scale", "v_scale"}."""
    if bits not in (8, 32):
        raise ValueError(f"bits: expected 8 or 32, got {bits}")
    dt = torch.float32 if bits == 32 else torch.float8_e4m3fn
    st = {k: torch.zeros(param.shape, dtype=torch.uint8 if bits == 8 else dt, device=param.device).view(dt)
          for k in ("m", "v")}
    if bits == 8:
        blocks = -(-param.numel() // ADAMW_BLOCK)
        for k in ("m_scale", "v_scale"):
            st[k] = torch.zeros(blocks, dtype=torch.float32, device=param.device)
    return st


class AdamwPlan:
    """The checked list of tensors of ``adamw_step`` (see ``adamw_plan``)."""

    def __init__(self, tensors):
        tensors = [dict(t) for t in tensors]
        if not tensors:
            raise ValueError("adamw_plan needs at least one tensor")
        self.device = tensors[0]["param"].device
        self.tensors = tensors
        self._list = (_AdamwTensor * len(tensors))()
        self._at = ctypes.addressof(self._list)
        for i, t in enumerate(tensors):
            self._set(i, t)
        n = ctypes.c_size_t(0)
        _check("lrs_adamw_scratch_bytes", _load().lrs_adamw_scratch_bytes(len(tensors), ctypes.byref(n)))
        self.scratch = torch.empty(n.value, dtype=torch.uint8, device=self.device)

    def _set(self, i, t):
        dev, p, name = self.device, t["param"], f"tensors[{i}]."
        master = t.get("master")
        _need(p, name + "param", torch.float32 if master is None else torch.bfloat16, dev)
        _opt(master, name + "master", torch.float32, dev, p.shape)
        q8 = t.get("m_scale") is not None
        for k in ("m", "v"):
            _need(t[k], name + k, torch.float8_e4m3fn if q8 else torch.float32, dev, p.shape)
        if q8 or t.get("v_scale") is not None:
            blocks = -(-p.numel() // ADAMW_BLOCK)
            for k in ("m_scale", "v_scale"):
                _need(t.get(k), name + k, torch.float32, dev, (blocks,))
        e = self._list[i]
        for k in ("param", "master", "m", "v", "m_scale", "v_scale"):
            x = t.get(k)
            setattr(e, k, None if x is None else x.data_ptr())
        e.n, e.weight_decay = p.numel(), float(t.get("weight_decay", 0.0))
        self._set_grad(i, t["grad"])

    def _set_grad(self, i, g):
        p = self.tensors[i]["param"]
        if g is None or g.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"tensors[{i}].grad: expected torch.float32 or torch.bfloat16, got {getattr(g, 'dtype', None)}")
        _need(g, f"tensors[{i}].grad", g.dtype, self.device, p.shape)
        self.tensors[i]["grad"] = g
        self._list[i].grad = g.data_ptr()
        self._list[i].grad_dtype = LRS_GRAD_FP32 if g.dtype == torch.float32 else LRS_GRAD_BF16

    def set_grads(self, grads):
        """New gradient tensors (same shapes), in the list's order."""
        grads = list(grads)
        if len(grads) != len(self.tensors):
            raise ValueError(f"expected {len(self.tensors)} gradients, got {len(grads)}")
        for i, g in enumerate(grads):
            self._set_grad(i, g)


def adamw_plan(tensors) -> AdamwPlan:
    """Checks a list of {"param", "grad", "m", "v"[, "master"][, "m_scale", "v_scale"][, "weight_decay"]} once, for
    ``adamw_step``.  param: FP32, or BF16 with an FP32 "master"; grad: FP32 or BF16; the state as ``adamw_state`` makes
    it.  The plan keeps the tensors; ``plan.set_grads`` replaces the gradients."""
    return AdamwPlan(tensors)


def adamw_step(plan: AdamwPlan, step, lr, *, beta1=0.9, beta2=0.95, eps=1e-8, max_norm=0.0, out=None):
    """One AdamW step over the plan's tensors, in place, through ``lrs_adamw_step``.

    step: int32 [1], the number of steps taken (advanced); lr: FP32 [1]; max_norm > 0 clips the gradients' norm over
    all tensors, and a step whose norm is not finite changes nothing.  Returns dict(norm (FP32 scalar, None without
    clipping), step)."""
    dev = plan.device
    _need(step, "step", torch.int32, dev, (1,))
    _need(lr, "lr", torch.float32, dev, (1,))
    norm = _empty((), torch.float32, dev, out, "norm") if max_norm > 0 else None
    _check("lrs_adamw_step",
           _load().lrs_adamw_step(plan._at, len(plan.tensors), step.data_ptr(), lr.data_ptr(), beta1, beta2, eps,
                                  max_norm, _ptr(norm), plan.scratch.data_ptr(), _stream(dev)))
    return {"norm": norm, "step": step}


def block_tensors_from_numpy(inp: dict, device) -> dict:
    """Device tensors of synth.block_inputs: {"x", "dout", "h0", "dhT", "reset", "params": {...}}."""
    params = {}
    for n in (BLOCK_PARAMS if inp.get("mixer", "samu") == "samu" else RGLRU_BLOCK_PARAMS):
        params[n] = _bf16(inp[n], device) if n in _BLOCK_BF16 else _f32(inp[n], device)
    out = {"x": _bf16(inp["x"], device), "dout": _bf16(inp["dout"], device), "h0": _f32(inp["h0"], device),
           "dhT": _f32(inp["dhT"], device), "params": params}
    out["reset"] = None if inp["reset"] is None else torch.from_numpy(inp["reset"]).to(device)
    return out


def selftest_wait_timeout(scratch, device=None) -> None:
    """Launches the library's failure-path self-test on ``scratch`` (see
    lrs_selftest_wait_timeout); with ``scratch=None``, on the status word of the
    no-allocation forward's fixed array (on ``device``)."""
    dev = scratch.device if scratch is not None else device
    _check("lrs_selftest_wait_timeout", _load().lrs_selftest_wait_timeout(_ptr(scratch), _stream(dev)))


def samu_forward_noalloc_status(device) -> int:
    """Status word of the most recent ``samu_forward_noalloc`` on ``device``
    (LRS_OK, or LRS_ERR_TIMEOUT; synchronises the current stream)."""
    v = ctypes.c_int(0)
    _check("samu_forward_noalloc_status",
           _load().samu_forward_noalloc_status(ctypes.byref(v), _stream(device)))
    return int(v.value)


def device_status(scratch, device=None) -> int:
    """Status word of the most recent call that used ``scratch`` (synchronises the stream)."""
    dev = scratch.device if device is None else device
    v = ctypes.c_int(0)
    _check("lrs_device_status", _load().lrs_device_status(_ptr(scratch), ctypes.byref(v), _stream(dev)))
    return int(v.value)


KERNEL_NAMES = {
    2: "samu_ctrl_fwd_kernel", 3: "samu_fwd_replay_kernel",
    4: "samu_bwd_main_kernel", 5: "samu_ctrl_bwd_kernel", 6: "samu_params_kernel",
    7: "rglru_scan_fwd_kernel", 8: "rglru_scan_bwd_kernel", 9: "rglru_alpha_kernels",
    10: "samu_fwd_maps_kernel", 11: "samu_bwd_maps_kernel", 12: "samu_decode_prepare_kernel",
    13: "samu_decode_step_kernel", 14: "proj_gemm_kernel<logits>", 15: "proj_gemm_kernel<dx, dW>",
    16: "proj_pack_kernel", 17: "block_gemm_kernel", 18: "rmsnorm_kernels", 19: "conv_kernels",
    20: "join_fwd_kernel", 21: "sum_parts_kernel", 22: "ce_gemm_kernel", 23: "ce_rows_kernels",
    24: "gated_norm_kernels", 25: "gated_norm_sum_kernel", 26: "adamw_norm_kernel", 27: "adamw_update_kernel",
}


def profile_begin(capacity: int) -> None:
    """Record CUDA events around every library kernel launched until profile_end()."""
    _check("lrs_profile_begin", _load().lrs_profile_begin(int(capacity)))


def profile_end(capacity: int):
    """Returns (list of (kernel name, ms) for the recorded launches, total launches seen)."""
    ids = (ctypes.c_int * capacity)()
    ms = (ctypes.c_float * capacity)()
    n = ctypes.c_int(0)
    _check("lrs_profile_end", _load().lrs_profile_end(ids, ms, capacity, ctypes.byref(n)))
    k = min(n.value, capacity)
    return [(KERNEL_NAMES.get(ids[i], str(ids[i])), float(ms[i])) for i in range(k)], int(n.value)


# ---------------------------------------------------------------------------
# numpy (seeded generator output) -> device tensors
# ---------------------------------------------------------------------------
def _bf16(bits: np.ndarray, device):
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)
    return t.to(device)


def _f32(a, device):
    if a is None:
        return None
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32).reshape(np.shape(a) or (1,))).to(device)


def samu_tensors_from_numpy(inp: dict, device) -> dict:
    out = {k: _bf16(inp[k], device) for k in ("x_sel", "w", "dy")}
    for k in ("nu", "theta", "w_phi", "w_r", "a_phi", "a_r", "h0", "dhT"):
        out[k] = _f32(inp[k], device)
    out["reset"] = None if inp["reset"] is None else torch.from_numpy(inp["reset"]).to(device)
    return out


def rglru_proj_tensors_from_numpy(inp: dict, device) -> dict:
    out = {k: _bf16(inp[k], device) for k in ("x", "w_x", "w_a", "dy")}
    for k in ("b_x", "b_a", "alpha", "h0", "dhT"):
        out[k] = _f32(inp[k], device)
    out["reset"] = None if inp["reset"] is None else torch.from_numpy(inp["reset"]).to(device)
    return out


def rglru_tensors_from_numpy(inp: dict, device) -> dict:
    out = {k: _bf16(inp[k], device) for k in ("x", "lx", "la", "dy")}
    for k in ("alpha", "h0", "dhT"):
        out[k] = _f32(inp[k], device)
    out["reset"] = None if inp["reset"] is None else torch.from_numpy(inp["reset"]).to(device)
    return out
