"""The AdamW step over many tensors (adamw_plan / adamw_step) against its
definition in 64 bits, started from the same states.

Tolerances (u = 2^-24).  The gradients' norm is an FP32 sum of squares, at most
64 of them in a thread and then pairwise or in short rows: relative 2^-18 with
the clipping factor.  m and v are two products and a sum: within 4 u of their
absolute terms plus the factor's error (twice for v); the step m / sqrt(v)
within 2^-17 of the same with m's absolute terms; p within 2 u |p| more.
BF16 copies: 2^-8 of the value.  8-bit states: E4M3 has 4 significant bits, so
a code is within 2^-4 of its value, or within 2^-10 of the scale below the
smallest normal code; a root that is not zero is at least 2^-9 of the scale.
Over several steps the errors of one step add (the factors are below 1).
"""
import pytest
import torch

from linear_recurrence_sequence_gb300 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
B1, B2, EPS = 0.9, 0.95, 1e-8
SIZES = (1, 3, 127, 255, 256, 257, 2047, 2048, 2049, 5000, 70001)


def _tensors(sizes, seed, bits=32, master=True, grad=torch.float32, fresh=False, gscale=1e-2):
    gen = torch.Generator().manual_seed(seed)
    ts = []
    for i, n in enumerate(sizes):
        p = torch.randn(n, generator=gen) * 0.05
        t = {"grad": (torch.randn(n, generator=gen) * gscale * 4.0 ** (i % 3)).to(grad).to(DEV),
             "weight_decay": 0.1 * (i % 2)}
        if master:
            t["master"], t["param"] = p.to(DEV), p.to(torch.bfloat16).to(DEV)
        else:
            t["param"] = p.to(DEV)
        t |= api.adamw_state(t["param"], bits)
        if not fresh:
            m, r = torch.randn(n, generator=gen) * gscale, torch.rand(n, generator=gen) * gscale
            if bits == 32:
                t["m"].copy_(m)
                t["v"].copy_(r * r)
            else:
                for k, a in (("m", m), ("v", r)):
                    pad = torch.zeros(-(-n // 256) * 256)
                    pad[:n] = a
                    s = pad.view(-1, 256).abs().amax(1) / 448
                    t[k + "_scale"].copy_(s)
                    t[k].copy_((pad.view(-1, 256) / s[:, None]).to(torch.float8_e4m3fn).view(-1)[:n])
        ts.append(t)
    return ts


def _spread(scale, n):
    return scale.double().repeat_interleave(256)[:n]


def _moments(t):
    """m and v of a tensor in 64 bits."""
    if t.get("m_scale") is None:
        return t["m"].double(), t["v"].double()
    n = t["param"].numel()
    return (t["m"].float().double() * _spread(t["m_scale"], n),
            (t["v"].float().double() * _spread(t["v_scale"], n)) ** 2)


def _expected(ts, t, lr, max_norm):
    norm = sum(float(x["grad"].double().square().sum()) for x in ts) ** 0.5
    k = max_norm / norm if 0 < max_norm < norm else 1.0
    out = []
    for x in ts:
        m, v = _moments(x)
        g = x["grad"].double() * k
        p = (x["param"] if x.get("master") is None else x["master"]).double()
        ma = B1 * m.abs() + (1 - B1) * g.abs()
        m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
        den = torch.sqrt(v / (1 - B2 ** t)) + EPS
        c1 = 1 - B1 ** t
        out.append({"p": p * (1 - lr * x["weight_decay"]) - lr * m / c1 / den, "m": m, "v": v, "ma": ma,
                    "step": lr * ma / c1 / den, "g": g})
    return norm, out


def _check(ts, exp, before):
    u = 2.0 ** -24
    for t, e, b in zip(ts, exp, before):
        p = t["param"] if t.get("master") is None else t["master"]
        off = (p.double() - e["p"]).abs() - (2 * u * (b["p"].abs() + e["p"].abs()) + 2.0 ** -17 * e["step"])
        assert float(off.max()) <= 0, float(off.max())
        if t.get("master") is not None:
            assert torch.equal(t["param"], t["master"].to(torch.bfloat16))
        em = 4 * u * e["ma"] + 2.0 ** -18 * (1 - B1) * e["g"].abs()
        ev = 4 * u * e["v"] + 2.0 ** -17 * (1 - B2) * e["g"] ** 2
        if t.get("m_scale") is None:
            assert float(((t["m"].double() - e["m"]).abs() - em).max()) <= 0
            assert float(((t["v"].double() - e["v"]).abs() - ev).max()) <= 0
            continue
        n = p.numel()
        m, v = _moments(t)
        for got, ref, err, s, low in ((m, e["m"], em, t["m_scale"], 2.0 ** -10),
                                      (v.sqrt(), e["v"].sqrt(), ev / e["v"].sqrt().clamp(min=1e-30), t["v_scale"], 2.0 ** -9)):
            s = _spread(s, n)
            most = torch.maximum(2.0 ** -4 * ref.abs(), low * s) * (1 + 2.0 ** -10) + 2 * err
            assert float(((got - ref).abs() - most).max()) <= 0
        assert bool(((v > 0) == (e["v"] > 0)).all())
        top = torch.zeros(-(-n // 256) * 256, dtype=torch.float64, device=DEV)
        top[:n] = e["m"].abs()
        top = top.view(-1, 256).amax(1) / 448
        assert float(((t["m_scale"].double() - top).abs() - 2.0 ** -16 * top).max()) <= 0


def _before(ts):
    return [{"p": (t["param"] if t.get("master") is None else t["master"]).double()} for t in ts]


def _scalars(step, lr=1e-2):
    return (torch.full((1,), step, dtype=torch.int32, device=DEV), torch.full((1,), lr, device=DEV))


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("master", [True, False])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6])
def test_one_step(bits, master, grad, max_norm):
    ts = _tensors(SIZES, 1, bits, master, grad)
    step, lr = _scalars(7)
    norm, exp = _expected(ts, 8, float(lr), max_norm)
    before = _before(ts)
    o = api.adamw_step(api.adamw_plan(ts), step, lr, beta1=B1, beta2=B2, eps=EPS, max_norm=max_norm)
    torch.cuda.synchronize()
    assert int(step) == 8
    if max_norm:
        assert abs(float(o["norm"]) - norm) <= 2.0 ** -18 * norm
    _check(ts, exp, before)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps_from_zero_states(bits):
    ts = _tensors(SIZES, 2, bits, fresh=True)
    ts[3]["grad"].zero_()   # a tensor that never gets a gradient keeps its value (but for its decay)
    step, lr = _scalars(0)
    plan = api.adamw_plan(ts)
    for k in range(1, 4):
        _, exp = _expected(ts, k, float(lr), 1.0)
        before = _before(ts)
        api.adamw_step(plan, step, lr, beta1=B1, beta2=B2, eps=EPS, max_norm=1.0)
        torch.cuda.synchronize()
        _check(ts, exp, before)
    assert int(step) == 3 and not ts[3]["m"].float().any() and not ts[3]["v"].float().any()


@pytest.mark.parametrize("count", [14, 32, 33, 400, 401, 900])
def test_lists_of_every_length(count):
    """The list's two sizes in the kernel's parameters, and more tensors than one launch takes."""
    sizes = [(i * 37) % 300 + 1 for i in range(count)]
    ts = _tensors(sizes, 3, gscale=1e-1)
    step, lr = _scalars(3)
    norm, exp = _expected(ts, 4, float(lr), 0.1)
    before = _before(ts)
    o = api.adamw_step(api.adamw_plan(ts), step, lr, beta1=B1, beta2=B2, eps=EPS, max_norm=0.1)
    assert abs(float(o["norm"]) - norm) <= 2.0 ** -18 * norm and int(step) == 4
    _check(ts, exp, before)
    # without clipping the step is advanced once
    _, exp = _expected(ts, 5, float(lr), 0.0)
    before = _before(ts)
    api.adamw_step(api.adamw_plan(ts), step, lr, beta1=B1, beta2=B2, eps=EPS)
    assert int(step) == 5
    _check(ts, exp, before)


def test_mixed_states_and_types_in_one_list():
    ts = _tensors(SIZES, 4, 8, True, torch.bfloat16) + _tensors(SIZES, 5, 32, False) + _tensors(SIZES, 6, 32, True)
    step, lr = _scalars(1)
    _, exp = _expected(ts, 2, float(lr), 0.3)
    before = _before(ts)
    api.adamw_step(api.adamw_plan(ts), step, lr, beta1=B1, beta2=B2, eps=EPS, max_norm=0.3)
    _check(ts, exp, before)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("count", [5, 500])
def test_a_norm_that_is_not_finite_changes_nothing(bad, count):
    ts = _tensors([64] * count, 7, 8)
    ts[count // 2]["grad"][13] = bad
    keys = ("param", "master", "m", "v", "m_scale", "v_scale")
    before = [[t[k].clone() for k in keys] for t in ts]
    step, lr = _scalars(9)
    o = api.adamw_step(api.adamw_plan(ts), step, lr, max_norm=1.0)
    assert not torch.isfinite(o["norm"]).any() and int(step) == 9
    for t, b in zip(ts, before):
        for k, x in zip(keys, b):
            assert torch.equal(t[k].view(torch.uint8), x.view(torch.uint8)), k


def test_small_and_uneven_blocks_in_8_bits():
    """Blocks that are tiny as a whole become zeros; a small root beside a large one stays above zero."""
    ts = _tensors([1024], 8, 8, fresh=True)
    g = ts[0]["grad"]
    g[:256] = 1e-38
    g[256:512] = 1e-6
    g[256] = 10.0
    g[512:768] = 0.0
    step, lr = _scalars(0)
    _, exp = _expected(ts, 1, float(lr), 0.0)
    before = _before(ts)
    api.adamw_step(api.adamw_plan(ts), step, lr, beta1=B1, beta2=B2, eps=EPS)
    torch.cuda.synchronize()
    m, v = _moments(ts[0])
    assert not m[:256].any() and not v[:256].any() and not m[512:768].any()
    assert bool((v[256:512] > 0).all())
    p = ts[0]["master"].double()
    off = (p - exp[0]["p"]).abs() - (2.0 ** -23 * (before[0]["p"].abs() + exp[0]["p"].abs()) + 2.0 ** -17 * exp[0]["step"])
    # v of the first block underflows in FP32 (1e-38 squared): its step is bounded by m / eps
    assert float(off[256:].max()) <= 0 and torch.isfinite(p).all()


def test_new_gradients_and_a_captured_graph():
    ts = _tensors(SIZES, 9)
    plan = api.adamw_plan(ts)
    step, lr = _scalars(0)
    # other gradient tensors, of the other type
    new = [(t["grad"] * 3).to(torch.bfloat16) for t in ts]
    plan.set_grads(new)
    ts2 = [{**t, "grad": g} for t, g in zip(ts, new)]
    _, exp = _expected(ts2, 1, float(lr), 1.0)
    before = _before(ts)
    api.adamw_step(plan, step, lr, beta1=B1, beta2=B2, eps=EPS, max_norm=1.0)
    torch.cuda.synchronize()
    _check(ts2, exp, before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.adamw_step(plan, step, lr, beta1=B1, beta2=B2, eps=EPS, max_norm=1.0)
    for k in (2, 3):
        lr.fill_(1e-2 / k)   # a schedule reaches a captured step
        for g in new:
            g.mul_(0.5)
        _, exp = _expected(ts2, k, float(lr), 1.0)
        before = _before(ts)
        graph.replay()
        torch.cuda.synchronize()
        assert int(step) == k
        _check(ts2, exp, before)


@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_past_32_bits(bits):
    """A tensor of more than 2^31 values: its end is updated like a tensor of its own."""
    n, tail = (1 << 31) + 5000, 4096 + 905
    start = n - tail
    gen = torch.Generator().manual_seed(13)

    def placed(values, dtype):
        t = torch.zeros(n, dtype=dtype, device=DEV)
        t[start:] = values.to(DEV)
        return t

    p = torch.randn(tail, generator=gen) * 0.05
    big = {"param": placed(p, torch.bfloat16), "master": placed(p, torch.float32), "weight_decay": 0.1,
           "grad": placed(torch.randn(tail, generator=gen) * 1e-2, torch.float32)}
    for k, a in (("m", torch.randn(tail, generator=gen) * 1e-2), ("v", torch.rand(tail, generator=gen) * 1e-2)):
        if bits == 32:
            big[k] = placed(a if k == "m" else a * a, torch.float32)
            continue
        blocks, at = -(-n // 256), start // 256 * 256
        pad = torch.zeros(blocks * 256 - at)
        pad[start - at:n - at] = a
        s = pad.view(-1, 256).abs().amax(1) / 448
        codes = (pad.view(-1, 256) / s[:, None]).to(torch.float8_e4m3fn).view(-1)
        big[k] = torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        big[k].view(torch.uint8)[at:] = codes.view(torch.uint8)[:n - at].to(DEV)
        big[k + "_scale"] = torch.zeros(blocks, device=DEV)
        big[k + "_scale"][at // 256:] = s.to(DEV)

    def moments():
        if bits == 32:
            return big["m"][start:].double(), big["v"][start:].double()
        at = start // 256
        sp = [big[k + "_scale"][at:].double().repeat_interleave(256)[start % 256:start % 256 + tail] for k in ("m", "v")]
        return big["m"][start:].float().double() * sp[0], (big["v"][start:].float().double() * sp[1]) ** 2

    step, lr = _scalars(2)
    p0, g0 = big["master"][start:].double(), big["grad"][start:].double()
    m0, v0 = moments()
    norm = float(g0.square().sum()) ** 0.5
    o = api.adamw_step(api.adamw_plan([big]), step, lr, beta1=B1, beta2=B2, eps=EPS, max_norm=1e9)
    assert abs(float(o["norm"]) - norm) <= 2.0 ** -18 * norm
    m1, v1 = B1 * m0 + (1 - B1) * g0, B2 * v0 + (1 - B2) * g0 * g0
    ref = p0 * (1 - float(lr) * big["weight_decay"]) - \
        float(lr) * m1 / (1 - B1 ** 3) / (torch.sqrt(v1 / (1 - B2 ** 3)) + EPS)
    ma = B1 * m0.abs() + (1 - B1) * g0.abs()
    most = 2.0 ** -23 * (p0.abs() + ref.abs()) + \
        2.0 ** -17 * float(lr) * ma / (1 - B1 ** 3) / (torch.sqrt(v1 / (1 - B2 ** 3)) + EPS)
    assert float(((big["master"][start:].double() - ref).abs() - most).max()) <= 0
    assert not big["master"][:1 << 20].any() and not big["m"].view(torch.uint8)[:1 << 20].any()
    assert torch.equal(big["param"][start:], big["master"][start:].to(torch.bfloat16))


def test_repeats_bit_for_bit_on_another_stream():
    results = []
    for side in (torch.cuda.current_stream(), torch.cuda.Stream()):
        ts = _tensors(SIZES, 10, 8)
        step, lr = _scalars(5)
        plan = api.adamw_plan(ts)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            api.adamw_step(plan, step, lr, max_norm=0.2)
        side.synchronize()
        results.append([t[k].view(torch.uint8) for t in ts for k in ("param", "master", "m", "v", "m_scale", "v_scale")])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_refusals():
    ts = _tensors((300,), 11)
    step, lr = _scalars(0)
    plan = api.adamw_plan(ts)
    for kw in ({"beta1": 1.0}, {"beta2": -0.1}, {"eps": 0.0}, {"beta1": float("nan")}, {"max_norm": float("inf")}):
        with pytest.raises(api.LrsError) as e:
            api.adamw_step(plan, step, lr, **kw)
        assert e.value.status == 1
    assert int(step) == 0
    with pytest.raises(TypeError):
        api.adamw_step(plan, step.long(), lr)
    with pytest.raises(ValueError):
        api.adamw_plan([])
    with pytest.raises(TypeError):       # a BF16 parameter needs its master
        api.adamw_plan([{**ts[0], "master": None}])
    with pytest.raises(TypeError):
        api.adamw_plan([{**ts[0], "grad": ts[0]["grad"].half()}])
    with pytest.raises(ValueError):
        api.adamw_plan([{**ts[0], "grad": ts[0]["grad"][:5]}])
    with pytest.raises(ValueError):      # one scale without the other
        q = _tensors((300,), 12, 8)[0]
        api.adamw_plan([{**q, "v_scale": None}])
    with pytest.raises(ValueError):
        plan.set_grads([])
    with pytest.raises(ValueError):
        api.adamw_state(ts[0]["param"], 16)
    odd = torch.zeros(301, device=DEV)[1:]
    with pytest.raises(api.LrsError) as e:   # not 16-byte aligned
        api.adamw_step(api.adamw_plan([{**ts[0], "grad": odd}]), step, lr)
    assert e.value.status == 1


def _norm_of(ts, step=0):
    """The norm that a step reports (a bound that nothing reaches)."""
    count, lr = _scalars(step)
    return float(api.adamw_step(api.adamw_plan(ts), count, lr, max_norm=3e38)["norm"])


# The norm adds at most 32 squares in one FP32 chain, each addition within u of
# its partial sum (the products are fused), and the chains in two floats: 2^-19
# of the sum of squares, half of that of its root, and u twice for the two last
# roundings: within 2^-19 of the norm.
NORM_TOL = 2.0 ** -19


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 3, 8, 31, 255, 256, 1000, 2049, 70001, 3000017])
def test_norm_of_equal_and_of_random_gradients(n, grad):
    gen = torch.Generator().manual_seed(n)
    ts = _tensors((n,), 20, grad=grad)
    for g in (torch.full((n,), 0.1), torch.full((n,), 1.0 / 3), torch.randn(n, generator=gen)):
        ts[0]["grad"].copy_(g)
        exact = float(ts[0]["grad"].double().square().sum()) ** 0.5
        assert abs(_norm_of(ts) - exact) <= NORM_TOL * exact


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("large", [1e18, 1e20, 1e30, 1e38])
def test_gradients_whose_squares_overflow_are_clipped(large, bits, grad):
    """A finite norm of gradients above the root of FP32's range clips them like any other."""
    ts = _tensors(SIZES, 21, bits, True, grad, gscale=1.0)
    for k in (1, 6, 10):
        ts[k]["grad"][::7] *= large / 200
    step, lr = _scalars(7)
    norm, exp = _expected(ts, 8, float(lr), 1.0)
    assert norm < 3e38
    before = _before(ts)
    o = api.adamw_step(api.adamw_plan(ts), step, lr, beta1=B1, beta2=B2, eps=EPS, max_norm=1.0)
    assert int(step) == 8
    assert abs(float(o["norm"]) - norm) <= NORM_TOL * norm
    for t, e, b in zip(ts, exp, before):
        p = t["master"].double()
        most = 2.0 ** -23 * (b["p"].abs() + e["p"].abs()) + 2.0 ** -17 * e["step"]
        assert float(((p - e["p"]).abs() - most).max()) <= 0


def test_a_norm_past_the_range_changes_nothing():
    ts = _tensors([2048] * 3, 22)
    ts[1]["grad"].fill_(3e38)   # finite values, a norm of 1e40
    before = [t["master"].clone() for t in ts]
    step, lr = _scalars(4)
    o = api.adamw_step(api.adamw_plan(ts), step, lr, max_norm=1.0)
    assert float(o["norm"]) == float("inf") and int(step) == 4
    assert all(torch.equal(t["master"], b) for t, b in zip(ts, before))


@pytest.mark.parametrize("master", [True, False])
@pytest.mark.parametrize("gscale", [1e-19, 1e-20, 1e-21])
def test_tiny_gradients_with_a_tiny_eps(gscale, master):
    """Second moments below FP32's normal range still divide the step.  v is rounded to multiples of 2^-149 twice on
    its way (its square and its product): 2^-149 absolute, half of that relative to v in its root."""
    ts = _tensors((5000,), 23, 32, master, fresh=True)
    g = (1 + torch.rand(5000, generator=torch.Generator().manual_seed(24))) * gscale
    ts[0]["grad"].copy_(g * torch.where(torch.arange(5000) % 2 == 0, 1.0, -1.0))
    step, lr = _scalars(0)
    g = ts[0]["grad"].double()
    p0 = _before(ts)[0]["p"]
    api.adamw_step(api.adamw_plan(ts), step, lr, beta1=B1, beta2=B2, eps=1e-30)
    p = (ts[0]["master"] if master else ts[0]["param"]).double()
    v = (1 - B2) * g * g
    move = float(lr) * g / (torch.sqrt(v / (1 - B2)) + 1e-30)
    off = (p - (p0 * (1 - float(lr) * ts[0]["weight_decay"]) - move)).abs()
    most = 2.0 ** -23 * (p0.abs() + move.abs()) + move.abs() * (2.0 ** -149 / v + 2.0 ** -17)
    assert float((off - most).max()) <= 0
