"""The gated pre/post norm (gated_norm_forward / gated_norm_backward) against
its definition in 64 bits on the same inputs; its gradients against
differences too.

Tolerances.  Each result is an expression of a few tens of FP32 operations
(2^-24 each), row means of up to 8192 terms (16 in a thread, then pairwise
over 512 threads: below 2^-19 of the terms' absolute sum) and the GeLU (2^-20).
So it is within 2^-16 of the same expression with every term taken by its
absolute value, plus 2^-8 of itself (BF16 storage, 8 significant bits; times
1 + 2^-7).  A parameter gradient adds rows: within 2^-15 of its sum of
absolute terms.
"""
import math

import pytest
import torch

from linear_recurrence_sequence_gb300 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-6


def _inputs(T, D, seed, branch=True, gate=True, vectors=True):
    gen = torch.Generator().manual_seed(seed)

    def r(*shape, s=1.0, d=torch.bfloat16):
        return (torch.randn(*shape, generator=gen) * s).to(d).to(DEV)

    one = torch.float32
    i = {"x": r(T, D, s=2.0), "y": r(T, D, s=0.7) if branch else None, "gate": r(T, D) if gate else None,
         "gamma_post": 1 + r(D, s=0.2, d=one) if branch and vectors else None,
         "scale": 0.5 + r(D, s=0.2, d=one) if branch and vectors else None,
         "gamma_pre": 1 + r(D, s=0.2, d=one) if vectors else None}
    return i, r(T, D, s=0.1), r(T, D, s=0.1)


def _gelu(g):
    u = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(2 * u)
    return g * s, s + 2 * g * s * torch.sigmoid(-2 * u) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)


def _definition(i, dr, dh):
    """Every output in 64 bits, and the sums of absolute terms that bound its error."""
    x = i["x"].double()
    one = torch.ones(x.shape[-1], dtype=torch.float64, device=DEV)
    gpre, gpost, scale = (one if i[k] is None else i[k].double() for k in ("gamma_pre", "gamma_post", "scale"))
    dr = torch.zeros_like(x) if dr is None else dr.double()
    dh = dh.double()
    branch, gate = i["y"] is not None, i["gate"] is not None

    def mean(a):
        return a.mean(-1, keepdim=True)

    r, ra = x, x.abs()
    if branch:
        y = i["y"].double()
        rstd1 = 1 / torch.sqrt(mean(y * y) + EPS)
        p = y * rstd1
        n = p * gpost
        ge, dge = _gelu(i["gate"].double()) if gate else (torch.ones_like(x), torch.zeros_like(x))
        u = scale * ge * n
        r, ra = x + u, x.abs() + u.abs()
    rstd2 = 1 / torch.sqrt(mean(r * r) + EPS)
    q, qa = r * rstd2, ra * rstd2
    a = dh * gpre
    dx = dr + rstd2 * (a - q * mean(a * q))
    dxa = dr.abs() + rstd2 * (a.abs() + qa * mean(a.abs() * qa))
    out = {"r": (r, ra), "h": (q * gpre, qa * gpre.abs()), "dx": (dx, dxa)}
    sums = {"dgamma_pre": ((dh * q).sum(0), (dh.abs() * qa).sum(0))}
    if branch:
        dn, dna = dx * scale * ge, dxa * (scale * ge).abs()
        b, ba = dn * gpost, dna * gpost.abs()
        out["dy"] = (rstd1 * (b - p * mean(b * p)), rstd1 * (ba + p.abs() * mean(ba * p.abs())))
        sums["dscale"] = ((dx * ge * n).sum(0), (dxa * (ge * n).abs()).sum(0))
        sums["dgamma_post"] = ((dn * p).sum(0), (dna * p.abs()).sum(0))
        if gate:
            out["dgate"] = (dx * scale * n * dge, dxa * (scale * n).abs() * (dge.abs() + 1))
    else:
        del out["r"]
    return out, sums


def _check(i, dr, dh):
    f = api.gated_norm_forward(**i, eps=EPS)
    b = api.gated_norm_backward(dr, dh, *i.values(), f["saved"], eps=EPS)
    got = {**{k: f[k] for k in ("r", "h")}, **b}
    out, sums = _definition(i, dr, dh)
    for k, (ref, most) in out.items():
        assert got[k].dtype == torch.bfloat16
        off = (got[k].double() - ref).abs() - (2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs() + 2.0 ** -16 * most)
        assert float(off.max()) <= 0, (k, float(off.max()))
    for k, (ref, most) in sums.items():
        assert got[k].dtype == torch.float32
        off = (got[k].double() - ref).abs() - 2.0 ** -15 * most
        assert float(off.max()) <= 0, (k, float(off.max()))
    return f, b


@pytest.mark.parametrize("branch,gate", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("T,D", [(1, 8), (1, 2048), (2, 64), (5, 256), (33, 264), (7, 320), (700, 1024), (130, 2560),
                                 (9, 4096), (11, 4104), (3, 8192), (2000, 72)])
def test_against_the_definition(T, D, branch, gate):
    i, dr, dh = _inputs(T, D, T + D, branch, gate)
    _check(i, dr, dh)


@pytest.mark.parametrize("branch", [True, False])
def test_missing_vectors_are_ones_and_missing_dr_is_zero(branch):
    i, dr, dh = _inputs(37, 520, 3, branch, branch, vectors=False)
    _check(i, None, dh)


def test_many_rows_per_cta():
    i, dr, dh = _inputs(20011, 128, 4)
    _check(i, dr, dh)


def test_zero_rows_and_large_values():
    """A row of zeros has a norm of sqrt(eps), not 0; rows near the largest BF16 squares stay finite."""
    i, dr, dh = _inputs(6, 256, 5)
    i["x"][0] = 0
    i["y"][0] = 0
    i["x"][1] = 0
    i["y"][2] = 0
    i["gate"][3] = 60.0
    i["gate"][4] = -60.0
    i["x"][5] *= 1e12
    _check(i, dr, dh)


def test_a_bad_row_stays_in_its_row():
    i, dr, dh = _inputs(40, 512, 6)
    clean = api.gated_norm_forward(**i)
    i["y"][3, 5], i["x"][9, 7], i["gate"][11, 0] = float("nan"), float("inf"), float("nan")
    f = api.gated_norm_forward(**i)
    rest = [k for k in range(40) if k not in (3, 9, 11)]
    assert torch.equal(f["h"][rest], clean["h"][rest]) and torch.equal(f["r"][rest], clean["r"][rest])
    assert torch.isnan(f["h"][3]).all()


def test_gradient_against_differences():
    i, dr, dh = _inputs(3, 16, 7)
    f = api.gated_norm_forward(**i, eps=EPS)
    b = api.gated_norm_backward(dr, dh, *i.values(), f["saved"], eps=EPS)
    step = 2.0 ** -12
    zero = torch.zeros(3, 16, dtype=torch.bfloat16, device=DEV)

    def value(j):
        out, _ = _definition(j, zero, zero)
        return float((out["r"][0] * dr.double()).sum() + (out["h"][0] * dh.double()).sum())

    names = {"x": "dx", "y": "dy", "gate": "dgate", "gamma_post": "dgamma_post", "scale": "dscale",
             "gamma_pre": "dgamma_pre"}
    for k, d in names.items():
        rms = float(b[d].double().square().mean().sqrt())
        for e in (0, 5, i[k].numel() - 1):
            vals = []
            for s in (step, -step):
                j = dict(i)
                j[k] = i[k].double().clone()
                j[k].view(-1)[e] += s
                vals.append(value(j))
            diff = (vals[0] - vals[1]) / (2 * step)
            # differences: order step^2; the result: BF16, or FP32 sums of BF16-sized errors
            assert abs(diff - float(b[d].view(-1)[e])) <= 2.0 ** -7 * max(rms, abs(diff)), (k, e)


def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows of a large call agree with a call on them alone."""
    T, D = (1 << 31) // 2048 + 40, 2048
    i, dr, dh = _inputs(64, D, 10)
    big = {}
    for k in ("x", "y", "gate"):
        big[k] = torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)
        big[k][-64:] = i[k]
    bdr, bdh = torch.zeros_like(big["x"]), torch.zeros_like(big["x"])
    bdr[-64:], bdh[-64:] = dr, dh
    vectors = [i[k] for k in ("gamma_post", "scale", "gamma_pre")]
    f = api.gated_norm_forward(big["x"], big["y"], big["gate"], *vectors)
    b = api.gated_norm_backward(bdr, bdh, big["x"], big["y"], big["gate"], *vectors, f["saved"])
    g = api.gated_norm_forward(**i)
    c = api.gated_norm_backward(dr, dh, *i.values(), g["saved"])
    for k in ("r", "h"):
        assert torch.equal(f[k][-64:], g[k]) and not f[k][:-64].any()
    for k in ("dx", "dy", "dgate"):
        assert torch.equal(b[k][-64:], c[k]) and not b[k][:1 << 10].any()
    out, sums = _definition(i, dr, dh)
    for k, (ref, most) in sums.items():   # rows of zeros add nothing
        assert float(((b[k].double() - ref).abs() - 2.0 ** -15 * most).max()) <= 0, k


def test_repeats_bit_for_bit_on_another_stream():
    i, dr, dh = _inputs(3000, 1024, 8)
    f, b = _check(i, dr, dh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f2 = api.gated_norm_forward(**i, eps=EPS)
        b2 = api.gated_norm_backward(dr, dh, *i.values(), f2["saved"], eps=EPS)
    side.synchronize()
    assert torch.equal(f["h"], f2["h"]) and torch.equal(f["r"], f2["r"])
    for k in ("dx", "dy", "dgate", "dgamma_post", "dscale", "dgamma_pre"):
        assert torch.equal(b[k], b2[k])


def test_refusals():
    i, dr, dh = _inputs(4, 64, 9)
    saved = api.gated_norm_forward(**i)["saved"]
    with pytest.raises(TypeError):
        api.gated_norm_forward(i["x"].float())
    with pytest.raises(ValueError):
        api.gated_norm_forward(i["x"][:, ::2])
    with pytest.raises(ValueError):
        api.gated_norm_forward(i["x"], i["y"][:2])
    with pytest.raises(ValueError):
        api.gated_norm_backward(dr, dh, *i.values(), saved[:8])
    for bad in ({"eps": 0.0}, {"eps": float("nan")}, {"eps": 2.0}):
        with pytest.raises(api.LrsError) as e:
            api.gated_norm_forward(**i, **bad)
        assert e.value.status == 1
    with pytest.raises(api.LrsError) as e:   # a gate without a branch
        api.gated_norm_forward(i["x"], None, i["gate"])
    assert e.value.status == 1
    for D, status in ((12, 2), (8200, 2)):
        with pytest.raises(api.LrsError) as e:
            api.gated_norm_forward(torch.zeros(2, D, dtype=torch.bfloat16, device=DEV))
        assert e.value.status == status


def test_gates_far_outside_the_sigmoid():
    """Gates whose cube leaves FP32's range: the derivative there is 1 or 0."""
    i, dr, dh = _inputs(9, 256, 20)
    for row, g in enumerate((1e12, -1e12, 1e13, -1e13, 1e14, -1e14, -3e38)):
        i["gate"][row, 3 * row] = g
    i["gate"][7] = -1e30
    _, b = _check(i, dr, dh)
    assert not b["dgate"][1, 3].any() and not b["dgate"][7].any()
    # a gate at the end of the range overflows its row's norm (h is 0 or not finite), not its own derivative
    i["gate"][8, 5] = 3e38
    f = api.gated_norm_forward(**i, eps=EPS)
    b = api.gated_norm_backward(dr, None if dh is None else torch.zeros_like(dh), *i.values(), f["saved"], eps=EPS)
    p = i["y"][8].double() / torch.sqrt(i["y"][8].double().square().mean() + EPS)
    ref = (dr[8].double() * i["scale"].double() * i["gamma_post"].double() * p)[5]
    assert abs(float(b["dgate"][8, 5]) - float(ref)) <= 2.0 ** -7 * abs(float(ref))
