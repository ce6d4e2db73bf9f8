"""The selective scan's decays at their ends.  Rates e^a_log past FP32's range: a state keeps nothing of the token before, as if
every token were a sequence's first, and a step of dt = 0 keeps all of it.  Decays near 1, whose errors a state adds up over all
that it keeps."""
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


@pytest.mark.parametrize("L", [50, 5000])
def test_a_step_of_zero_keeps_every_bit(L):
    """Whatever the rate, for any number of tokens, in one chunk and over several; in steps too."""
    B, D, N = 2, 64, 16
    i, _, _ = _inputs(B, L, D, N, 0.0, seed=L)
    i["a_log"] = (torch.rand(D, N, device=DEV) - 0.5) * 160
    i["delta"][:] = -math.inf
    f = api.selective_scan_forward(**i, keep=False)
    assert torch.equal(f["hT"], i["h0"])
    state = i["h0"].clone()
    api.selective_scan_step(i["x"][:, 0], i["delta"][:, 0], i["a_log"], i["b"][:, 0], i["c"][:, 0], i["d_skip"], i["delta_bias"],
                            i["gate"][:, 0], state)
    assert torch.equal(state, i["h0"])


@pytest.mark.parametrize("step", [False, True])
def test_decays_near_one_are_right_on_average(step):
    """With the same inputs at every token a state goes to dt x b / (1 - a).  That a is off by d moves it by d / (1 - a) of
    itself, whatever the number of tokens.  Over 1024 states that keep 25 to 500 tokens, d is within 2^-26 on average, a quarter
    of the spacing of FP32 numbers below 1 (each decay's own rounding and the rates' are as often up as down).

    The states' own rounding is not, token after token: h <- fl(a h + k) rises until a h + k is within half a spacing u of h,
    and stops there, short of k / (1 - a) by u / (2 (1 - a)).  That is u / (2 h) in units of d, known for each state.  (The
    forward's chunks start from zero and are joined by their sums of dt: none of them gets so far.)"""
    B, L, D, N = 1, 4000, 64, 16
    gen = torch.Generator().manual_seed(7)
    keep = 2.0 ** (-0.003 * 20.0 ** torch.rand(D, N, generator=gen, dtype=torch.float64))   # exponents from 0.003 to 0.06
    delta = torch.randn(1, 1, D, generator=gen).to(BF)
    dt = torch.nn.functional.softplus(delta.double()).view(D, 1)
    a_log = torch.log(-torch.log(keep) / dt).float().to(DEV)
    one = torch.ones(B, L, N, dtype=BF, device=DEV)
    x = torch.ones(B, L, D, dtype=BF, device=DEV)
    delta = delta.to(DEV).expand(B, L, D).contiguous()
    if step:
        h = torch.zeros(B, D, N, device=DEV)
        for _ in range(L):
            api.selective_scan_step(x[:, 0], delta[:, 0], a_log, one[:, 0], one[:, 0], None, None, None, h)
    else:
        h = api.selective_scan_forward(x, delta, a_log, one, one, keep=False)["hT"]
    dt = dt.to(DEV)
    e = -torch.exp(a_log.double()) * dt
    want = dt * torch.expm1(L * e) / torch.expm1(e)
    off = (h[0].double() / want - 1) * -torch.expm1(e)
    if step:
        spacing = (torch.nextafter(h[0], torch.full_like(h[0], math.inf)) - h[0]).double()
        off = off + spacing / (2 * h[0].double())
    assert abs(float(off.mean())) <= 2.0 ** -26
