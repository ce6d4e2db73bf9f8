"""The selective scan at rates e^a_log past FP32's range: a state keeps nothing of the token before, as if every token were a
sequence's first, and a step of dt = 0 keeps all of it."""
import math

import pytest
import torch

import ssm_reference as ref
from linear_recurrence_sequence_gb300 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32
GRADS = ("dx", "ddelta", "da_log", "db", "dc", "dd_skip", "ddelta_bias", "dgate", "dh0")


def _inputs(B, L, D, N, a_log, seed):
    gen = torch.Generator().manual_seed(seed)

    def r(*shape, s=1.0, d=BF):
        return (torch.randn(*shape, generator=gen) * s).to(d).to(DEV)

    i = {"x": r(B, L, D), "delta": r(B, L, D, s=0.7), "a_log": torch.full((D, N), a_log, device=DEV), "b": r(B, L, N), "c": r(B, L, N),
         "d_skip": r(D, d=F), "delta_bias": r(D, d=F) - 2.0, "gate": r(B, L, D), "h0": r(B, D, N, d=F)}
    return i, r(B, L, D, s=0.3), r(B, D, N, s=0.3, d=F)


# one chunk that ends inside a tile, whole tiles, several chunks
@pytest.mark.parametrize("B,L,D,N", [(2, 61, 64, 16), (3, 64, 8, 5), (1, 1, 24, 40), (1, 1999, 72, 12)])
@pytest.mark.parametrize("a_log", [60.0, 88.5, 89.0, 1e4, math.inf])
def test_nothing_is_kept(B, L, D, N, a_log):
    i, dy, dhT = _inputs(B, L, D, N, a_log, seed=L + N)
    f = api.selective_scan_forward(**i)
    g = api.selective_scan_backward(dy, dhT, *i.values(), None, f["saved"], grad_fp32=True)
    starts = torch.ones(B, L, dtype=torch.uint8, device=DEV)
    want = ref.scan(**{**i, "a_log": torch.zeros_like(i["a_log"])}, reset=starts, dy=dy, dhT=dhT)
    ref.check({"y": f["y"], "hT": f["hT"], **{k: g[k] for k in GRADS}}, want)
    state = i["h0"].clone()
    s = api.selective_scan_step(*(i[k][:, 0] if i[k].dim() == 3 else i[k] for k in ("x", "delta")), i["a_log"], i["b"][:, 0],
                                i["c"][:, 0], i["d_skip"], i["delta_bias"], i["gate"][:, 0], state)
    one = {k: v[:, :1] if k in ("x", "delta", "b", "c", "gate") else v for k, v in i.items()}
    ref.check({"y": s["y"][:, None], "hT": state}, ref.scan(**{**one, "a_log": torch.zeros_like(i["a_log"])}, reset=starts[:, :1]))


def test_a_step_of_zero_keeps_all():
    i, _, _ = _inputs(2, 100, 64, 16, 100.0, seed=3)
    i["delta"][:, 40:] = -math.inf
    whole = api.selective_scan_forward(**i, keep=False)
    part = {k: v[:, :40].contiguous() if k in ("x", "delta", "b", "c", "gate") else v for k, v in i.items()}
    ahead = api.selective_scan_forward(**part, keep=False)
    assert torch.equal(whole["hT"], ahead["hT"]) and torch.equal(whole["y"][:, :40], ahead["y"])
    assert bool(torch.isfinite(whole["y"]).all())
