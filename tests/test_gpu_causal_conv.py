"""The causal convolution (causal_conv_forward / _step / _backward) against its definition in 64 bits; the bounds are
those of ssm_reference."""
import math

import pytest
import torch

import ssm_reference as ref
from linear_recurrence_sequence_gb300 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


def _inputs(B, L, D, W, seed, bias=True, state=True, resets=0.0):
    gen = torch.Generator().manual_seed(seed)

    def r(*shape, s=1.0, d=BF):
        return (torch.randn(*shape, generator=gen) * s).to(d).to(DEV)

    f = torch.float32
    i = {"x": r(B, L, 2 * D + 8)[..., D:2 * D], "weight": r(W, D, s=0.6, d=f), "bias": r(D, s=0.5, d=f) if bias else None,
         "state": r(B, W - 1, D) if state else None,
         "reset": (torch.rand(B, L, generator=gen) < resets).to(torch.uint8).to(DEV) if resets else None}
    return i, r(B, L, D)


def _run(i, dy, silu, fp32):
    f = api.causal_conv_forward(**i, silu=silu)
    g = api.causal_conv_backward(dy, **i, silu=silu, grad_fp32=fp32)
    return {"y": f["y"], "state": f["state"], **{k: g[k] for k in ("dx", "dweight", "dbias", "dstate")}}


@pytest.mark.parametrize("B,L,D,W", [
    (1, 1, 8, 4), (2, 2, 64, 4), (1, 3, 256, 3), (3, 8, 264, 2), (2, 16, 136, 4), (1, 17, 128, 4), (2, 63, 72, 3),
    (1, 64, 520, 2), (2, 65, 24, 4), (1, 128, 1024, 4), (2, 129, 328, 4), (3, 1009, 328, 3), (1, 300, 2056, 4)])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("fp32", [False, True])
def test_matches_the_definition(B, L, D, W, silu, fp32):
    i, dy = _inputs(B, L, D, W, seed=B + L + D + W, resets=0.1)
    got = _run(i, dy, silu, fp32)
    ref.check(got, ref.conv(*i.values(), silu_=silu, dy=dy))
    assert got["dx"].dtype == got["dstate"].dtype == (torch.float32 if fp32 else BF)


@pytest.mark.parametrize("B,L,D,W", [(600, 318, 16, 4), (600, 320, 16, 3), (1100, 250, 8, 2)])
@pytest.mark.parametrize("resets", [0.0, 0.02])
def test_long_runs(B, L, D, W, resets):
    """Batch enough for runs of up to 80 tokens, the last one shorter; starts on either side of a run's ends."""
    i, dy = _inputs(B, L, D, W, seed=W, resets=resets)
    if resets:
        i["reset"][::2, 75:85] = 1
        i["reset"][1::2, 80] = 1
    ref.check(_run(i, dy, True, True), ref.conv(*i.values(), dy=dy))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("state", [False, True])
def test_missing_inputs(bias, state):
    i, dy = _inputs(2, 50, 64, 4, seed=1, bias=bias, state=state)
    got = _run(i, dy, True, True)
    ref.check(got, ref.conv(*i.values(), dy=dy))
    assert (got["dbias"] is not None) == bias and (got["dstate"] is not None) == state


@pytest.mark.parametrize("W", [2, 3, 4])
def test_resets_at_every_place(W):
    i, dy = _inputs(4, 140, 64, W, seed=W)
    reset = torch.zeros(4, 140, dtype=torch.uint8, device=DEV)
    reset[0] = 1
    reset[1, [0, 139]] = 3
    reset[2, [1, 2, 7, 8, 9, 15, 16, 63, 64, 65, 127, 128, 137]] = 1
    reset[3, 138] = 255
    i["reset"] = reset
    got = _run(i, dy, True, True)
    ref.check(got, ref.conv(*i.values(), dy=dy))
    assert float(got["dstate"][:2].abs().max()) == 0


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
def test_steps_are_the_forward(W, silu):
    i, _ = _inputs(5, 40, 264, W, seed=7, resets=0.15)
    whole = api.causal_conv_forward(**i, silu=silu)
    head = api.causal_conv_forward(i["x"][:, :9], i["weight"], i["bias"], i["state"], i["reset"][:, :9].contiguous(), silu=silu)
    assert torch.equal(head["y"], whole["y"][:, :9])
    state = head["state"]
    for t in range(9, 40):
        o = api.causal_conv_step(i["x"][:, t], i["weight"], i["bias"], state, i["reset"][:, t].contiguous(), silu=silu)
        assert o["state"].data_ptr() == state.data_ptr()
        assert torch.equal(o["y"], whole["y"][:, t]), t
    assert torch.equal(state, whole["state"])


def test_what_lies_ahead_of_a_start_stays_there():
    i, dy = _inputs(2, 60, 64, 4, seed=9)
    i["x"][0, :21] = math.nan
    i["x"][1, :21] = math.inf
    i["state"][:] = math.nan
    i["reset"] = torch.zeros(2, 60, dtype=torch.uint8, device=DEV)
    i["reset"][:, 21] = 1
    got = _run(i, dy, True, True)
    want = ref.conv(i["x"][:, 21:], i["weight"], i["bias"], None, None, dy=dy[:, 21:])
    ref.check({"y": got["y"][:, 21:], "state": got["state"], "dx": got["dx"][:, 21:]}, want)


def test_strides_streams_and_bits():
    i, dy = _inputs(2, 200, 136, 4, seed=15, resets=0.02)
    first = _run(i, dy, True, False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        wide = torch.full((2, 200, 3 * 136), 5.0, dtype=BF, device=DEV)
        dx = wide[..., 136:2 * 136]
        g = api.causal_conv_backward(dy, **i, out={"dx": dx})
        again = _run({k: v if v is None else v.contiguous() for k, v in i.items()}, dy, True, False)
    side.synchronize()
    for k in first:
        assert torch.equal(first[k], again[k]), k
    assert torch.equal(dx, first["dx"]) and torch.equal(g["dweight"], first["dweight"])
    assert bool((wide[..., :136] == 5).all()) and bool((wide[..., 2 * 136:] == 5).all())


def test_gradients_against_differences():
    i, dy = _inputs(2, 40, 16, 4, seed=25, resets=0.05)
    got = _run(i, dy, True, True)
    gen = torch.Generator(device=DEV).manual_seed(3)
    for k, g in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("state", "dstate")):
        v = torch.randn(i[k].shape, generator=gen, device=DEV, dtype=torch.float64)
        e = 1e-5
        loss = [float((ref.conv(*{**i, k: i[k].double() + s * e * v}.values())["y"][0] * dy.double()).sum()) for s in (1, -1)]
        slope, mine = (loss[0] - loss[1]) / (2 * e), got[g].double() * v
        assert abs(float(mine.sum()) - slope) <= 1e-3 * float(mine.abs().sum()) / math.sqrt(v.numel()) + 1e-6 * abs(slope), k


def test_a_captured_step():
    i, dy = _inputs(2, 100, 64, 4, seed=31)
    want = _run(i, dy, True, False)
    scratch = torch.empty(api.causal_conv_workspace_bytes(2, 100, 64, 4), dtype=torch.uint8, device=DEV)
    out = {k: torch.zeros_like(v) for k, v in want.items()}
    state = i["state"].clone()
    x1 = i["x"][:, 0]

    def step():
        api.causal_conv_forward(**i, out=out)
        api.causal_conv_backward(dy, **i, out=out, scratch=scratch)
        return api.causal_conv_step(x1, i["weight"], i["bias"], state)["y"]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1 = step()
    for v in out.values():
        v.zero_()
    scratch.fill_(0xff)
    state.copy_(i["state"])
    graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(out[k], want[k]), k
    assert torch.equal(y1, want["y"][:, 0])
    assert torch.equal(state, torch.cat([i["state"][:, 1:], x1[:, None]], 1))
    assert api.device_status(scratch) == 0   # (it held 0xff)


def test_more_than_2_31_values():
    L, D = 270336, 8000
    assert L * D > 1 << 31
    x = torch.empty(1, L, D, dtype=BF, device=DEV).normal_()
    w = torch.randn(4, D, device=DEV)
    f = api.causal_conv_forward(x, w)
    ref.check({"y": f["y"][:, -9:], "state": f["state"]}, ref.conv(x[:, -9:], w, None, x[:, -12:-9]))
    g = api.causal_conv_backward(f["y"], x, w)
    tail = ref.conv(x[:, -20:], w, None, x[:, -23:-20], dy=f["y"][:, -20:])
    ref.check({"dx": g["dx"][:, -9:]}, {"dx": tuple(v[:, -9:] for v in tail["dx"])})
