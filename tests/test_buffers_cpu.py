"""Buffers that a caller hands over (saved, scratch, decode parameters): a buffer on another device, strided or too
short is refused by name before anything is launched.  Runs without a GPU: the calls stop at the stream."""
import pytest
import torch

from linear_recurrence_sequence_gb300 import api

B, L, D = 1, 4, 64
M = D // 2
BF, F = torch.bfloat16, torch.float32


def _z(*shape, dtype=F):
    return torch.zeros(*shape, dtype=dtype)


def _samu_params():
    return [_z(M), _z(M), _z(D + 1), _z(D + 1), _z(1), _z(1)]


def _calls():
    """name -> (bytes, call): the call takes the buffer in question; every other argument is good."""
    x = _z(B, L, D, dtype=BF)
    state = _z(B, M, 2)
    h, w, t = _z(5, D, dtype=BF), _z(7, D, dtype=BF), _z(5, dtype=torch.int64)
    samu, rg = api.samu_workspace_bytes(B, L, D), api.rglru_workspace_bytes(B, L, D)
    ce, norm = api.linear_ce_workspace_bytes(5, 7, D), api.gated_norm_workspace_bytes(5, D)
    samu_saved, rg_saved = _z(samu[0], dtype=torch.uint8), _z(rg[0], dtype=torch.uint8)
    gn_saved = _z(norm[0], dtype=torch.uint8)
    return {
        "samu_forward saved": (samu[0], lambda b: api.samu_forward(x, x, None, None, *_samu_params(), saved=b)),
        "samu_forward scratch": (samu[1], lambda b: api.samu_forward(x, x, None, None, *_samu_params(), scratch=b)),
        "samu_backward saved": (samu[0], lambda b: api.samu_backward(x, None, x, x, None, None, *_samu_params(), b)),
        "samu_backward scratch": (samu[1], lambda b: api.samu_backward(x, None, x, x, None, None, *_samu_params(),
                                                                       samu_saved, scratch=b)),
        "rglru_forward saved": (rg[0], lambda b: api.rglru_forward(x, x, x, _z(D), None, None, saved=b)),
        "rglru_forward scratch": (rg[1], lambda b: api.rglru_forward(x, x, x, _z(D), None, None, scratch=b)),
        "rglru_backward saved": (rg[0], lambda b: api.rglru_backward(x, None, x, x, x, _z(D), None, None, b)),
        "rglru_backward scratch": (rg[1], lambda b: api.rglru_backward(x, None, x, x, x, _z(D), None, None, rg_saved,
                                                                       scratch=b)),
        "samu_decode_prepare params": (4 * api.samu_decode_params_floats(D),
                                       lambda b: api.samu_decode_prepare(*_samu_params(), params=b)),
        "samu_decode_step params": (4 * api.samu_decode_params_floats(D),
                                    lambda b: api.samu_decode_step(_z(B, D, dtype=BF), _z(B, D, dtype=BF), state, b)),
        "linear_ce_forward scratch": (ce[0], lambda b: api.linear_ce_forward(h, w, t, scratch=b)),
        "linear_ce_backward scratch": (ce[1], lambda b: api.linear_ce_backward(h, w, t, _z(5), _z(5), scratch=b)),
        "gated_norm_forward saved": (norm[0], lambda b: api.gated_norm_forward(h, h, saved=b)),
        "gated_norm_backward saved": (norm[0], lambda b: api.gated_norm_backward(None, h, h, h, None, None, None, None, b)),
        "gated_norm_backward scratch": (norm[1], lambda b: api.gated_norm_backward(None, h, h, h, None, None, None, None,
                                                                                   gn_saved, scratch=b)),
    }


def _proj_calls():
    d = 16 * 16   # a width that the gate projections take
    x = _z(1, 4, d, dtype=BF)
    wx = _z(api.PROJ_BLOCKS, d // api.PROJ_BLOCKS, d // api.PROJ_BLOCKS, dtype=BF)
    p = [wx, _z(d), wx, _z(d), _z(d)]
    n = api.rglru_proj_workspace_bytes(1, 4, d)
    saved = _z(n[0], dtype=torch.uint8)
    return {
        "rglru_proj_forward saved": (n[0], lambda b: api.rglru_proj_forward(x, *p, None, None, saved=b)),
        "rglru_proj_forward scratch": (n[1], lambda b: api.rglru_proj_forward(x, *p, None, None, scratch=b)),
        "rglru_proj_backward saved": (n[0], lambda b: api.rglru_proj_backward(x, None, x, *p, None, None, b)),
        "rglru_proj_backward scratch": (n[1], lambda b: api.rglru_proj_backward(x, None, x, *p, None, None, saved, scratch=b)),
    }


def _block_calls():
    dm, d = 256, 256
    shapes = api._block_shapes(dm, d)
    params = {k: _z(*shapes[k], dtype=BF if k in api._BLOCK_BF16 else F) for k in api.BLOCK_PARAMS}
    x = _z(1, 4, dm, dtype=BF)
    n = api.samu_block_workspace_bytes(1, 4, dm, d)
    saved = _z(n[0], dtype=torch.uint8)
    return {
        "samu_block_forward saved": (n[0], lambda b: api.samu_block_forward(x, params, saved=b)),
        "samu_block_forward scratch": (n[1], lambda b: api.samu_block_forward(x, params, scratch=b)),
        "samu_block_backward saved": (n[0], lambda b: api.samu_block_backward(x, None, x, params, None, None, b)),
        "samu_block_backward scratch": (n[1], lambda b: api.samu_block_backward(x, None, x, params, None, None, saved,
                                                                               scratch=b)),
        "dense_gemm scratch": (256, lambda b: api.dense_gemm(api.LRS_GEMM_NT, _z(8, 64, dtype=BF), _z(8, 64, dtype=BF), 8, 8,
                                                            64, scratch=b)),
    }


@pytest.fixture(scope="module")
def calls():
    import os
    if not os.path.exists(api.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return {**_calls(), **_proj_calls(), **_block_calls()}


NAMES = ["samu_forward saved", "samu_forward scratch", "samu_backward saved", "samu_backward scratch",
         "rglru_forward saved", "rglru_forward scratch", "rglru_backward saved", "rglru_backward scratch",
         "samu_decode_prepare params", "samu_decode_step params", "linear_ce_forward scratch", "linear_ce_backward scratch",
         "gated_norm_forward saved", "gated_norm_backward saved", "gated_norm_backward scratch",
         "rglru_proj_forward saved", "rglru_proj_forward scratch", "rglru_proj_backward saved",
         "rglru_proj_backward scratch", "samu_block_forward saved", "samu_block_forward scratch",
         "samu_block_backward saved", "samu_block_backward scratch", "dense_gemm scratch"]


@pytest.mark.parametrize("name", NAMES)
def test_refuses_a_buffer_by_name(calls, name, monkeypatch):
    def no_stream(device):
        raise RuntimeError("nothing is launched here")

    monkeypatch.setattr(api, "_stream", no_stream)
    n, call = calls[name]
    assert n > 0
    good = torch.empty(n, dtype=torch.uint8)
    for bad in (torch.empty(n, dtype=torch.uint8, device="meta"), torch.empty(2 * n, dtype=torch.uint8)[::2], good[:-1]):
        with pytest.raises(ValueError, match=name.split()[1]):
            call(bad)
    with pytest.raises(RuntimeError, match="nothing is launched"):   # a good one passes
        call(good)


def test_every_call_is_covered(calls):
    assert sorted(calls) == sorted(NAMES)
