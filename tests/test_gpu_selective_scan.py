"""The selective scan (selective_scan_forward / _step / _backward) against its definition in 64 bits, token after token;
its gradients against differences too.  The bounds are those of ssm_reference."""
import math

import pytest
import torch

import ssm_reference as ref
from linear_recurrence_sequence_gb300 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
GRADS = ("dx", "ddelta", "da_log", "db", "dc", "dd_skip", "ddelta_bias", "dgate", "dh0")


def _inputs(B, L, D, N, seed, gate=True, skip=True, bias=True, h0=True, resets=0.0, strided=True):
    gen = torch.Generator().manual_seed(seed)

    def r(*shape, s=1.0, d=BF):
        return (torch.randn(*shape, generator=gen) * s).to(d).to(DEV)

    f = torch.float32
    proj, small = r(B, L, 2 * D), r(B, L, 3 + 2 * N)
    i = {"x": proj[..., :D], "delta": r(B, L, D, s=0.7), "a_log": r(D, N, s=0.7, d=f) + 0.5, "b": small[..., 3:3 + N],
         "c": small[..., 3 + N:], "d_skip": r(D, d=f) if skip else None,
         "delta_bias": (r(D, s=1.0, d=f) - 2.5) if bias else None, "gate": proj[..., D:] if gate else None,
         "h0": r(B, D, N, d=f) if h0 else None,
         "reset": (torch.rand(B, L, generator=gen) < resets).to(torch.uint8).to(DEV) if resets else None}
    if not strided:
        i = {k: v if v is None else v.contiguous() for k, v in i.items()}
    return i, r(B, L, D, s=0.3), r(B, D, N, s=0.3, d=f)


def _run(i, dy, dhT, fp32=False):
    f = api.selective_scan_forward(**i)
    g = api.selective_scan_backward(dy, dhT, *i.values(), f["saved"], grad_fp32=fp32)
    return {"y": f["y"], "hT": f["hT"], **{k: g[k] for k in GRADS}}


SHAPES = [
    (1, 1, 8, 1), (2, 7, 64, 16), (3, 100, 72, 5), (2, 257, 136, 16), (1, 300, 264, 12), (2, 129, 24, 64),
    (1, 65, 520, 33), (4, 33, 1040, 8), (1, 40, 2056, 4), (5, 16, 128, 17), (2, 1023, 32, 2),
    (900, 70, 8, 4),     # batch enough for one chunk of more than 64 tokens
]


@pytest.mark.parametrize("B,L,D,N", SHAPES)
@pytest.mark.parametrize("fp32", [False, True])
def test_matches_the_definition(B, L, D, N, fp32):
    i, dy, dhT = _inputs(B, L, D, N, seed=B + 3 * L + 5 * D + 7 * N, resets=0.03)
    got = _run(i, dy, dhT, fp32)
    want = ref.scan(**i, dy=dy, dhT=dhT)
    ref.check(got, want)
    for k in ("dx", "ddelta", "db", "dc", "dgate"):
        assert got[k].dtype == (torch.float32 if fp32 else BF)


@pytest.mark.parametrize("B,L,D,N", [(8, 2390, 8, 5), (8, 2432, 40, 16), (8, 2390, 16, 64), (19, 1024, 256, 16),
                                     (8, 2690, 40, 16), (8, 2710, 8, 3), (8, 2700, 72, 30)])
@pytest.mark.parametrize("resets", [0.0, 0.002])
def test_chunks_of_several_tiles(B, L, D, N, resets):
    """Chunks of 64 tokens and of 72, whose reverse maps are those of their halves (of 32, of 40 and 32 tokens); at 2390 and
    2690 tokens the last chunk has one half."""
    i, dy, dhT = _inputs(B, L, D, N, seed=N, resets=resets)
    i["delta_bias"] = i["delta_bias"] - 2.0   # states that reach over several chunks
    ref.check(_run(i, dy, dhT), ref.scan(**i, dy=dy, dhT=dhT))


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("skip,bias", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("h0", [False, True])
def test_missing_inputs(gate, skip, bias, h0):
    i, dy, dhT = _inputs(2, 90, 88, 16, seed=11, gate=gate, skip=skip, bias=bias, h0=h0)
    dhT = dhT if h0 else None
    got = _run(i, dy, dhT, True)
    ref.check(got, ref.scan(**i, dy=dy, dhT=dhT))
    for k, there in (("dgate", gate), ("dd_skip", skip), ("ddelta_bias", bias), ("dh0", h0)):
        assert (got[k] is not None) == there
    f = api.selective_scan_forward(**i, keep=False)
    assert f["saved"] is None and torch.equal(f["y"], got["y"]) and torch.equal(f["hT"], got["hT"])


def test_resets_at_every_place():
    """Every token a start; starts at the first and last tokens, at tile and chunk ends."""
    i, dy, dhT = _inputs(4, 200, 64, 16, seed=5)
    reset = torch.zeros(4, 200, dtype=torch.uint8, device=DEV)
    reset[0] = 1
    reset[1, [0, 199]] = 7
    reset[2, [7, 8, 15, 16, 17, 31, 32, 47, 48, 63, 64, 95, 96, 127, 128]] = 1
    i["reset"] = reset
    got = _run(i, dy, dhT, True)
    ref.check(got, ref.scan(**i, dy=dy, dhT=dhT))
    # nothing of the carried state gets past a start
    for k in range(2):
        assert float(got["dh0"][k].abs().max()) == 0


@pytest.mark.parametrize("D,N", [(64, 16), (8, 3), (136, 8), (1024, 16), (40, 64), (96, 30), (2048, 1), (24, 41)])
def test_step_is_the_forward_of_one_token(D, N):
    B = 37
    i, _, _ = _inputs(B, 1, D, N, seed=D + N, resets=0.3)
    want = ref.scan(**i)
    s = {k: v if v is None or k in ("a_log", "d_skip", "delta_bias", "h0") else v[:, 0] for k, v in i.items()}
    s["reset"] = i["reset"].view(B)
    state = s.pop("h0").clone()
    at = state.data_ptr()
    o = api.selective_scan_step(*[s[k] for k in ("x", "delta", "a_log", "b", "c", "d_skip", "delta_bias", "gate")], state,
                                s["reset"])
    assert o["state"].data_ptr() == at
    ref.check({"y": o["y"][:, None], "hT": o["state"]}, want)


def test_steps_go_on_where_the_prompt_ended():
    i, _, _ = _inputs(3, 150, 264, 16, seed=3, resets=0.05)
    want = ref.scan(**i)

    def part(a, b):
        return {k: v if v is None or k in ("a_log", "d_skip", "delta_bias", "h0") else v[:, a:b] for k, v in i.items()}

    p = part(0, 100)
    p["reset"] = p["reset"].contiguous()
    f = api.selective_scan_forward(**p, keep=False)
    ys, state = [f["y"]], f["hT"]
    for t in range(100, 150):
        s = part(t, t + 1)
        o = api.selective_scan_step(*[None if s[k] is None else s[k] if k in ("a_log", "d_skip", "delta_bias") else s[k][:, 0]
                                      for k in ("x", "delta", "a_log", "b", "c", "d_skip", "delta_bias", "gate")], state,
                                    s["reset"][:, 0].contiguous())
        ys.append(o["y"][:, None])
    ref.check({"y": torch.cat(ys, 1), "hT": state}, want)


def test_padding():
    """A token with delta = -inf leaves the state as it is; what lies ahead of a start, NaN and infinity too, reaches
    neither the sequence nor its state."""
    i, dy, dhT = _inputs(2, 120, 64, 16, seed=8)
    i["delta"][:, 80:] = -math.inf
    f = api.selective_scan_forward(**i)
    cut = {k: v if v is None or k in ("a_log", "d_skip", "delta_bias", "h0") else v[:, :80] for k, v in i.items()}
    want = ref.scan(**cut, dy=dy[:, :80], dhT=dhT)
    ref.check({"y": f["y"][:, :80], "hT": f["hT"]}, want)
    dy[:, 80:] = 0
    g = api.selective_scan_backward(dy, dhT, *i.values(), f["saved"], grad_fp32=True)
    ref.check({k: g[k] if k in ("da_log", "dd_skip", "ddelta_bias", "dh0") else g[k][:, :80] for k in GRADS}, want)
    for k in ("dx", "ddelta", "db", "dgate"):
        assert float(g[k][:, 80:].abs().max()) == 0, k

    i, dy, dhT = _inputs(2, 120, 64, 16, seed=9, strided=False)
    for k in ("x", "delta", "b", "c", "gate"):
        i[k][0, :37] = math.nan
        i[k][1, :37] = math.inf
    i["h0"][:] = math.nan
    i["reset"] = torch.zeros(2, 120, dtype=torch.uint8, device=DEV)
    i["reset"][:, 37] = 1
    f = api.selective_scan_forward(**i)
    tail = {k: v if v is None or k in ("a_log", "d_skip", "delta_bias") else v[:, 37:] for k, v in i.items()}
    tail["h0"] = None
    ref.check({"y": f["y"][:, 37:], "hT": f["hT"]}, ref.scan(**tail))
    g = api.selective_scan_backward(dy, dhT, *i.values(), f["saved"], grad_fp32=True)
    want = ref.scan(**tail, dy=dy[:, 37:], dhT=dhT)
    ref.check({k: g[k][:, 37:] for k in ("dx", "ddelta", "db", "dc", "dgate")}, want)


def test_extreme_steps():
    """dt from 0 to hundreds, rates from 1e-6 to 1e6: states that keep everything, and nothing."""
    i, dy, dhT = _inputs(2, 64, 64, 16, seed=13)
    i["delta"][:, ::3] *= 60
    i["a_log"] *= 9
    got = _run(i, dy, dhT, True)
    ref.check(got, ref.scan(**i, dy=dy, dhT=dhT))


def test_gradients_against_differences():
    """The loss sum(dy y) + sum(dhT hT), in the definition's 64 bits, along random directions."""
    i, dy, dhT = _inputs(2, 50, 24, 6, seed=21, resets=0.05)
    got = _run(i, dy, dhT, True)

    def loss(j):
        o = ref.scan(**j)
        return float((o["y"][0] * dy.double()).sum() + (o["hT"][0] * dhT.double()).sum())

    gen = torch.Generator(device=DEV).manual_seed(2)
    for k, g in (("x", "dx"), ("delta", "ddelta"), ("a_log", "da_log"), ("b", "db"), ("c", "dc"), ("d_skip", "dd_skip"),
                 ("delta_bias", "ddelta_bias"), ("gate", "dgate"), ("h0", "dh0")):
        v = torch.randn(i[k].shape, generator=gen, device=DEV, dtype=torch.float64)
        e = 1e-5
        up, down = ({**i, k: i[k].double() + s * e * v} for s in (1, -1))
        slope = (loss(up) - loss(down)) / (2 * e)
        mine = float((got[g].double() * v).sum())
        # the difference's own error is of the order e^2; the gradient's is far below 1e-3 of its terms
        assert abs(mine - slope) <= 1e-3 * float((got[g].double() * v).abs().sum()) / math.sqrt(v.numel()) + 1e-6 * abs(slope), k


def test_same_bits_every_time_and_on_any_stream():
    i, dy, dhT = _inputs(2, 500, 328, 16, seed=31, resets=0.01)
    first = _run(i, dy, dhT)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = _run(i, dy, dhT)
    side.synchronize()
    for k in first:
        assert torch.equal(first[k], second[k]), k


def test_outputs_as_halves_of_the_projections_gradient():
    B, L, D = 2, 70, 64
    i, dy, dhT = _inputs(B, L, D, 16, seed=41)
    want = _run(i, dy, dhT)
    wide = torch.full((B, L + 3, 2 * D + 8), 5.0, dtype=BF, device=DEV)
    dx, dgate = wide[:, :L, :D], wide[:, :L, D:2 * D]
    f = api.selective_scan_forward(**i)
    g = api.selective_scan_backward(dy, dhT, *i.values(), f["saved"], out={"dx": dx, "dgate": dgate})
    assert g["dx"].data_ptr() == wide.data_ptr()
    assert torch.equal(dx, want["dx"]) and torch.equal(dgate, want["dgate"]) and torch.equal(g["ddelta"], want["ddelta"])
    assert bool((wide[:, L:] == 5).all()) and bool((wide[:, :, 2 * D:] == 5).all())


def test_inputs_shared_by_the_batch():
    """Batch stride 0 (an expanded tensor) reads like copies."""
    i, dy, dhT = _inputs(3, 40, 64, 8, seed=43)
    for k in ("x", "b", "gate"):
        i[k] = i[k][:1].expand(3, *i[k].shape[1:])
    got = _run(i, dy, dhT)
    want = _run({k: v if v is None else v.contiguous() for k, v in i.items()}, dy, dhT)
    for k in got:
        assert torch.equal(got[k], want[k]), k


def test_a_captured_training_step_and_its_workspaces():
    i, dy, dhT = _inputs(2, 300, 128, 16, seed=51)
    want = _run(i, dy, dhT)
    n = api.selective_scan_workspace_bytes(2, 300, 128, 16)
    saved, scratch = (torch.empty(k, dtype=torch.uint8, device=DEV) for k in (n[0], max(n[1:])))
    out = {k: torch.zeros_like(v) for k, v in want.items()}

    def step():
        api.selective_scan_forward(**i, saved=saved, scratch=scratch, out=out)
        api.selective_scan_backward(dy, dhT, *i.values(), saved, scratch=scratch, out=out)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in out.values():
        v.zero_()
    saved.fill_(0xff)
    scratch.fill_(0xff)
    graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(out[k], want[k]), k
    # other inputs in the same buffers
    j, dy2, dhT2 = _inputs(2, 300, 128, 16, seed=52)
    for k, v in i.items():
        if v is not None:
            v.copy_(j[k])
    dy.copy_(dy2)
    dhT.copy_(dhT2)
    graph.replay()
    again = _run(j, dy2, dhT2)
    for k in again:
        assert torch.equal(out[k], again[k]), k


@pytest.mark.parametrize("B,L,D,N", [(900, 8, 8, 4), (2, 300, 128, 16)])
def test_status_word(B, L, D, N):
    """Whatever the scratch held before: one chunk and several."""
    i, dy, dhT = _inputs(B, L, D, N, seed=5)
    n = api.selective_scan_workspace_bytes(B, L, D, N)
    scratch = torch.full((max(n[1:]),), 0xff, dtype=torch.uint8, device=DEV)
    saved = api.selective_scan_forward(**i, scratch=scratch)["saved"]
    assert api.device_status(scratch) == 0
    scratch.fill_(0xff)
    api.selective_scan_backward(dy, dhT, *i.values(), saved, scratch=scratch)
    assert api.device_status(scratch) == 0


def test_state_in_place():
    """hT may be h0 (a server's slot): one chunk and several."""
    for L in (40, 400):
        i, _, _ = _inputs(2, L, 64, 16, seed=L)
        want = api.selective_scan_forward(**i, keep=False)
        slot = i["h0"].clone()
        got = api.selective_scan_forward(**{**i, "h0": slot}, keep=False, out={"hT": slot})
        assert torch.equal(got["y"], want["y"]) and torch.equal(slot, want["hT"])


def test_more_than_2_31_values():
    """One long sequence whose x, delta and y have more than 2^31 values: its last tokens are those of the tail alone."""
    L, D, N, tail = 270336, 8000, 4, 100
    assert L * D > 1 << 31
    gen = torch.Generator(device=DEV).manual_seed(7)

    def r(*shape, s=1.0):
        t = torch.empty(*shape, dtype=BF, device=DEV)
        return t.normal_(generator=gen).mul_(s)

    i = {"x": r(1, L, D), "delta": r(1, L, D, s=0.5), "a_log": torch.rand(D, N, generator=gen, device=DEV), "b": r(1, L, N),
         "c": r(1, L, N)}
    f = api.selective_scan_forward(**i, keep=False)
    # one state forgets within 2000 tokens (rate 1 and dt about 0.7: 1e-600): the tail from any state before
    part = {k: v if k == "a_log" else v[:, L - 2000 - tail:] for k, v in i.items()}
    got = api.selective_scan_forward(**part, keep=False)
    ref.check({"y": f["y"][:, -tail:], "hT": f["hT"]},
              ref.scan(**{k: v if k == "a_log" else v[:, -tail:] for k, v in i.items()},
                       h0=api.selective_scan_forward(**{k: v if k == "a_log" else v[:, L - 2000 - tail:L - tail]
                                                        for k, v in i.items()}, keep=False)["hT"]))
    assert float((f["hT"] - got["hT"]).abs().max()) <= 2.0 ** -15 * float(got["hT"].abs().max())
