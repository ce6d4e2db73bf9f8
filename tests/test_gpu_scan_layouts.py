"""The selective scan by the layout of b, c and a_log: copied two states at a time, read one at a time, rates and states four
at a time.  Every form against the definition in 64 bits, and against each other: they compute the same."""
import pytest
import torch

import ssm_reference as ref
from linear_recurrence_sequence_gb300 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32
GRADS = ("dx", "ddelta", "da_log", "db", "dc", "dd_skip", "ddelta_bias", "dgate", "dh0")


def _placed(t, offset):
    """t's values `offset` elements behind a 256-byte boundary."""
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device=DEV)
    v = buf[offset:].view(t.shape)
    v.copy_(t)
    return v


def _inputs(B, L, D, N, seed):
    gen = torch.Generator().manual_seed(seed)

    def r(*shape, s=1.0, d=BF):
        return (torch.randn(*shape, generator=gen) * s).to(d).to(DEV)

    i = {"x": r(B, L, D), "delta": r(B, L, D, s=0.7), "a_log": r(D, N, s=0.7, d=F) + 0.5, "b": r(B, L, N), "c": r(B, L, N),
         "d_skip": r(D, d=F), "delta_bias": r(D, d=F) - 2.5, "gate": r(B, L, D), "h0": r(B, D, N, d=F),
         "reset": (torch.rand(B, L, generator=gen) < 0.02).to(torch.uint8).to(DEV)}
    return i, r(B, L, D, s=0.3), r(B, D, N, s=0.3, d=F)


def _run(i, dy, dhT):
    f = api.selective_scan_forward(**i)
    g = api.selective_scan_backward(dy, dhT, *i.values(), f["saved"], grad_fp32=True)
    return {"y": f["y"], "hT": f["hT"], **{k: g[k] for k in GRADS}}


def _forms(i):
    """The same inputs: b and c a value at a time; in words; a_log off the 16-byte boundaries."""
    yield {**i, "b": _placed(i["b"], 1), "c": _placed(i["c"], 3)}
    yield {**i, "b": _placed(i["b"], 2), "c": _placed(i["c"], 6)}
    yield {**i, "a_log": _placed(i["a_log"], 1)}
    yield {**i, "a_log": _placed(i["a_log"], 2), "b": _placed(i["b"], 1)}


# as many states as each number of lanes a channel takes, and fewer; even, odd, multiples of four
@pytest.mark.parametrize("N", [1, 2, 4, 6, 7, 8, 10, 12, 16, 18, 24, 29, 30, 32, 34, 48, 50, 63, 64])
@pytest.mark.parametrize("B,L,D", [(2, 77, 136)])
def test_every_width_of_b_and_c(B, L, D, N):
    i, dy, dhT = _inputs(B, L, D, N, seed=N)
    assert i["b"].data_ptr() % 16 == 0 and i["a_log"].data_ptr() % 16 == 0
    got = _run(i, dy, dhT)
    ref.check(got, ref.scan(**i, dy=dy, dhT=dhT))
    for j in _forms(i):
        same = _run(j, dy, dhT)
        for k in got:
            assert torch.equal(got[k], same[k]), k


@pytest.mark.parametrize("B,L,D,N", [(8, 2390, 8, 24), (8, 2432, 16, 64), (2, 1500, 40, 32), (1, 3000, 72, 8), (1, 2000, 520, 4)])
def test_several_chunks(B, L, D, N):
    i, dy, dhT = _inputs(B, L, D, N, seed=N)
    got = _run(i, dy, dhT)
    ref.check(got, ref.scan(**i, dy=dy, dhT=dhT))
    for j in _forms(i):
        same = _run(j, dy, dhT)
        for k in got:
            assert torch.equal(got[k], same[k]), k


@pytest.mark.parametrize("N", [1, 3, 4, 5, 8, 12, 16, 20, 24, 32, 36, 48, 61, 64])
@pytest.mark.parametrize("B,D", [(37, 136), (700, 24)])
def test_step(B, D, N):
    """From the smallest grid of the step to several turns a CTA, in words of four states and one at a time."""
    i, _, _ = _inputs(B, 1, D, N, seed=N)
    want = ref.scan(**i)
    first = None
    for j in (i, *_forms(i)):
        s = {k: v if k in ("a_log", "d_skip", "delta_bias", "h0") else v[:, 0] for k, v in j.items()}
        s["reset"] = s["reset"].contiguous()
        state = s.pop("h0").clone()
        reset = s.pop("reset")
        o = api.selective_scan_step(*s.values(), state, reset)
        ref.check({"y": o["y"][:, None], "hT": state}, want)
        if first is None:
            first = o["y"].clone(), state
        assert torch.equal(o["y"], first[0]) and torch.equal(state, first[1])


def test_step_of_more_sequences_than_the_grid_takes_at_once():
    B, D, N = 3000, 2048, 8
    i, _, _ = _inputs(B, 1, D, N, seed=5)
    s = {k: v if k in ("a_log", "d_skip", "delta_bias", "h0") else v[:, 0] for k, v in i.items()}
    reset = s.pop("reset").contiguous()
    state = s.pop("h0")
    before = state.clone()
    o = api.selective_scan_step(*s.values(), state, reset)
    for k in (slice(0, 5), slice(1490, 1500), slice(2990, 3000)):
        part = {n: v[k] if n in ("x", "delta", "b", "c", "gate") else v for n, v in i.items()}
        ref.check({"y": o["y"][k, None], "hT": state[k]}, ref.scan(**{**part, "h0": before[k], "reset": i["reset"][k]}))
