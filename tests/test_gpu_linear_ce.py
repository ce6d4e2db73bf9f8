"""The vocabulary loss (linear_ce_forward / linear_ce_backward) against its
definition in 64 bits on the same BF16 inputs.

Tolerances.  With u = 2^-24 the FP32 half-ulp:
  - a logit is a sum of D exact BF16 products accumulated in FP32, and
    e^{z - lse} is formed at arguments of size |z| + |lse|: both move z' by at
    most a few u (sum |h_i w_i| + |z| + |lse|).  The inputs keep that sum below
    2^7, so |loss - exact| and |lse - exact| <= 2^7 * 8 u = 6.1e-5, and the
    relative error of e^{z - lse} is of the same size.
  - gradients, element by element: with dz's relative rounding r (2^-8 as one
    BF16 number: 8 significant bits, to nearest; 2^-16 as two), an FP32
    accumulation of K terms in steps of 16 (each at most 2^-23 of the sum of the
    absolute terms) and the error above of p = e^{z - lse}, an element is within
      (r + 2^-23 (K / 16 + 4)) (|dz| |w|) + 6.1e-5 (|p dloss| |w|) + r_out |dh|
    (times 1 + 2^-7 for the products of two errors) of the exact one (r_out =
    2^-8 for a BF16 result, 2^-24 for FP32), dw alike:
    a bound that holds through cancellation, which a bound by the result's own
    size does not;
  - over a tensor the roundings are independent: relative L2 error <= 2^-8
    (BF16) and <= 2^-16 + 6.1e-5 (FP32).
  - against differences: the loss is evaluated in 64 bits at w +- e for single
    entries; central differences with step 2^-10 have an error of order step^2
    (1e-6) beside the FP32 gradient's 1e-5: within 1e-4 of the larger of the
    entry and the tensor's RMS.
"""
import numpy as np
import pytest
import torch

from linear_recurrence_sequence_gb300 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TOL_ROW = 6.1e-5


def _inputs(T, V, D, seed, ignored=0.0, std=2.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, D, generator=g).to(torch.bfloat16)
    w = (torch.randn(V, D, generator=g) * (std / D ** 0.5)).to(torch.bfloat16)
    t = torch.randint(0, V, (T,), generator=g)
    t[torch.rand(T, generator=g) < ignored] = -100
    return h.to(DEV), w.to(DEV), t.to(DEV)


def _exact(h, w, t, dloss=None, softcap=0.0, bounds=None):
    """loss, lse, dh, dw in 64 bits on the CPU (and the bounds on dh and dw)."""
    h, w, t = h.double().cpu().numpy(), w.double().cpu().numpy(), t.cpu().numpy()
    z = h @ w.T
    if softcap:
        z = softcap * np.tanh(z / softcap)
    m = z.max(1, keepdims=True)
    lse = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
    ok = (t >= 0) & (t < w.shape[0])
    at = np.where(ok, t, 0)
    rows = np.arange(len(t))
    loss = np.where(ok, lse - z[rows, at], 0.0)
    d = np.where(ok, 1.0 / max(ok.sum(), 1) if dloss is None else dloss.double().cpu().numpy(), 0.0)
    p = np.exp(z - lse[:, None])
    p[rows, at] -= 1.0
    dz = p * d[:, None]
    if softcap:
        dz = dz * (1 - (z / softcap) ** 2)
    if not bounds:
        return loss, lse, dz @ w, dz.T @ h
    pd, dz1 = np.abs(np.exp(z - lse[:, None]) * d[:, None]), np.abs(dz)

    def bound(x, y, k, out, r, r_out):
        return (1 + 2.0 ** -7) * ((r + 2.0 ** -23 * (k / 16 + 4)) * (dz1 @ x if y is None else dz1.T @ y) +
                                  TOL_ROW * (pd @ x if y is None else pd.T @ y) + r_out * np.abs(out))

    r, r_out = (2.0 ** -16, 2.0 ** -24) if bounds == "fp32" else (2.0 ** -8, 2.0 ** -8)
    dh, dw = dz @ w, dz.T @ h
    return (loss, lse, dh, dw, bound(np.abs(w), None, w.shape[0], dh, r, r_out),
            bound(None, np.abs(h), h.shape[0], dw, r, r_out))


def _rel(a, b):
    n = np.linalg.norm(b)
    return float(np.linalg.norm(a - b) / n) if n else float(np.abs(a).max(initial=0.0))


def _f64(t):
    return t.detach().double().cpu().numpy()


def _check(h, w, t, softcap=0.0, dloss=None, fp32=False):
    f = api.linear_ce_forward(h, w, t, softcap=softcap)
    b = api.linear_ce_backward(h, w, t, f["lse"], dloss, total=f["total"], softcap=softcap, grad_fp32=fp32)
    torch.cuda.synchronize()
    assert api.device_status(f["scratch"]) == 0 and api.device_status(b["scratch"]) == 0
    loss, lse, dh, dw, bh, bw = _exact(h, w, t, dloss, softcap, "fp32" if fp32 else "bf16")
    np.testing.assert_allclose(_f64(f["lse"]), lse, rtol=0, atol=TOL_ROW)
    np.testing.assert_allclose(_f64(f["loss"]), loss, rtol=0, atol=TOL_ROW)
    n = int((t >= 0).sum())
    assert float(f["total"][1]) == n
    assert abs(float(f["total"][0]) - loss.sum()) <= TOL_ROW * max(n, 1) + 2.0 ** -23 * abs(loss.sum())
    for got, ref, most in ((b["dh"], dh, bh), (b["dw"], dw, bw)):
        assert got.dtype == (torch.float32 if fp32 else torch.bfloat16)
        e = _rel(_f64(got), ref)
        assert e <= (2.0 ** -16 + TOL_ROW if fp32 else 2.0 ** -8), e
        off = np.abs(_f64(got) - ref) - most
        assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    return f, b


SIZES = [(1, 1, 8), (1, 2, 8), (1, 4099, 64), (3, 257, 72), (127, 300, 320), (128, 256, 64), (129, 255, 256),
         (255, 513, 136), (257, 1000, 64), (300, 31, 520), (1000, 130, 24), (2, 20001, 1024), (640, 2048, 128)]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_loss_and_gradients(T, V, D, fp32):
    _check(*_inputs(T, V, D, seed=T + V + D, ignored=0.1 if T > 8 else 0.0), fp32=fp32)


@pytest.mark.parametrize("T,V,D", [(5, 700, 64), (200, 1111, 136)])
@pytest.mark.parametrize("fp32", [False, True])
def test_softcap_and_weights(T, V, D, fp32):
    h, w, t = _inputs(T, V, D, 3, ignored=0.25, std=4.0)
    g = torch.Generator().manual_seed(9)
    dloss = torch.rand(T, generator=g).to(DEV) / T
    _check(h, w, t, softcap=5.0, dloss=dloss, fp32=fp32)
    _check(h, w, t, softcap=30.0, fp32=fp32)


def test_long_token_axis_is_split():
    """Many tokens against a small vocabulary: dw is split over the tokens and joined in order."""
    _check(*_inputs(20000, 40, 64, 5))
    _check(*_inputs(9000, 40, 64, 6), fp32=True)


def test_pieces_of_the_vocabulary():
    """More tokens x vocabulary than one piece of logit gradients holds: the pieces' rows of dw and sums of dh."""
    T, V, D = 70000, 5000, 8
    assert T * V * 2 > 512 << 20
    h, w, t = _inputs(T, V, D, 7)
    keep = torch.randperm(T, generator=torch.Generator().manual_seed(1))[:300].to(DEV)
    # only 300 tokens are counted, so that the 64-bit definition needs only those
    t2 = torch.full_like(t, -1)
    t2[keep] = t[keep]
    keep = torch.sort(keep).values
    for fp32 in (False, True):
        f = api.linear_ce_forward(h, w, t2)
        b = api.linear_ce_backward(h, w, t2, f["lse"], total=f["total"], grad_fp32=fp32)
        loss, lse, dh, dw = _exact(h[keep], w, t2[keep])
        np.testing.assert_allclose(_f64(f["loss"][keep]), loss, rtol=0, atol=TOL_ROW)
        tol = 2.0 ** -16 + TOL_ROW if fp32 else 2.0 ** -8
        assert _rel(_f64(b["dh"][keep]), dh) <= tol
        assert _rel(_f64(b["dw"]), dw) <= tol
        rest = torch.ones(T, dtype=torch.bool, device=DEV)
        rest[keep] = False
        assert not b["dh"][rest].any()


def test_no_token_counts():
    h, w, t = _inputs(130, 300, 64, 11)
    t = torch.full_like(t, -100)
    f = api.linear_ce_forward(h, w, t)
    b = api.linear_ce_backward(h, w, t, f["lse"], total=f["total"])
    assert not f["loss"].any() and not f["total"].any() and not b["dh"].any() and not b["dw"].any()
    np.testing.assert_allclose(_f64(f["lse"]), _exact(h, w, t)[1], rtol=0, atol=TOL_ROW)


def test_rows_that_do_not_count_may_hold_anything():
    """NaN and infinities in the rows of tokens that are not counted reach no gradient and no other row."""
    h, w, t = _inputs(150, 600, 64, 12)
    t[::3] = -1
    clean = api.linear_ce_forward(h, w, t)
    grads = api.linear_ce_backward(h, w, t, clean["lse"], total=clean["total"])
    bad = h.clone()
    bad[0], bad[3], bad[147] = float("nan"), float("inf"), float("-inf")
    f = api.linear_ce_forward(bad, w, t)
    b = api.linear_ce_backward(bad, w, t, f["lse"], total=f["total"])
    live = t >= 0
    assert torch.equal(f["loss"][live], clean["loss"][live]) and not f["loss"][~live].any()
    assert torch.equal(f["total"], clean["total"])
    assert torch.equal(b["dh"], grads["dh"]) and torch.equal(b["dw"], grads["dw"])
    dloss = torch.full((150,), 0.01, device=DEV)
    x = api.linear_ce_backward(h, w, t, clean["lse"], dloss)
    y = api.linear_ce_backward(bad, w, t, f["lse"], dloss)
    assert torch.equal(x["dh"], y["dh"]) and torch.equal(x["dw"], y["dw"])


def test_extreme_logits():
    """Logits of several hundred: one entry carries the whole mass, and the sum never overflows."""
    T, V, D = 9, 700, 64
    h, w, t = _inputs(T, V, D, 13)
    w[5] = h[2] * 8   # row 2: a logit of about 8 |h|^2
    f = api.linear_ce_forward(h, w, t)
    loss, lse, _, _ = _exact(h, w, t)
    np.testing.assert_allclose(_f64(f["lse"]), lse, rtol=1e-5, atol=TOL_ROW)
    assert torch.isfinite(f["loss"]).all()


def test_target_past_the_vocabulary_is_reported():
    h, w, t = _inputs(40, 100, 64, 14)
    t[7], t[9] = 100, 1 << 40
    f = api.linear_ce_forward(h, w, t)
    assert api.device_status(f["scratch"]) == 1          # LRS_ERR_ARG
    assert float(f["loss"][7]) == 0.0 and float(f["loss"][9]) == 0.0 and float(f["total"][1]) == 38
    b = api.linear_ce_backward(h, w, t, f["lse"], total=f["total"])
    loss, _, dh, dw = _exact(h, w, t)
    assert _rel(_f64(b["dh"]), dh) <= 2.0 ** -8 and _rel(_f64(b["dw"]), dw) <= 2.0 ** -8
    assert not b["dh"][7].any() and not b["dh"][9].any()


def test_gradient_against_differences():
    T, V, D = 12, 50, 16
    h, w, t = _inputs(T, V, D, 15)
    f = api.linear_ce_forward(h, w, t, softcap=6.0)
    b = api.linear_ce_backward(h, w, t, f["lse"], total=f["total"], softcap=6.0, grad_fp32=True)
    step = 2.0 ** -10

    def mean_loss(hh, ww):
        return _exact(hh, ww, t, softcap=6.0)[0].mean()

    for x, g, other in ((h.double(), b["dh"], "w"), (w.double(), b["dw"], "h")):
        rms = float(g.double().square().mean().sqrt())
        for i in (0, 37, x.numel() - 1):
            lo, hi = x.clone(), x.clone()
            lo.view(-1)[i] -= step
            hi.view(-1)[i] += step
            args = [(a, w.double()) if other == "w" else (h.double(), a) for a in (hi, lo)]
            diff = (mean_loss(*args[0]) - mean_loss(*args[1])) / (2 * step)
            assert abs(diff - float(g.view(-1)[i])) <= 1e-4 * max(rms, abs(diff))


def test_offsets_past_32_bits():
    """w and dw of more than 2^31 values: the loss knows the last rows, and dw has them."""
    D, V = 2048, (1 << 31) // 2048 + 300
    T = 12
    gen = torch.Generator().manual_seed(20)
    h = torch.randn(T, D, generator=gen).to(torch.bfloat16).to(DEV)
    w = torch.zeros(V, D, dtype=torch.bfloat16, device=DEV)
    tail = (torch.randn(300, D, generator=gen) * (4.0 / D ** 0.5)).to(torch.bfloat16).to(DEV)
    w[-300:] = tail
    t = (V - 300 + torch.randint(0, 300, (T,), generator=gen)).to(DEV)
    f = api.linear_ce_forward(h, w, t)
    b = api.linear_ce_backward(h, w, t, f["lse"], total=f["total"])
    # in 64 bits: V - 300 logits of zero beside the 300
    z = h.double() @ tail.double().T
    lse = torch.log(torch.exp(z).sum(1) + (V - 300))
    at = t - (V - 300)
    rows = torch.arange(T, device=DEV)
    np.testing.assert_allclose(_f64(f["lse"]), _f64(lse), rtol=0, atol=TOL_ROW)
    np.testing.assert_allclose(_f64(f["loss"]), _f64(lse - z[rows, at]), rtol=0, atol=TOL_ROW)
    p = torch.exp(z - lse[:, None])
    p[rows, at] -= 1
    dz = p / T
    assert _rel(_f64(b["dh"]), _f64(dz @ tail.double())) <= 2.0 ** -8
    assert _rel(_f64(b["dw"][-300:]), _f64(dz.T @ h.double())) <= 2.0 ** -8
    rest = (torch.exp(-lse)[:, None] / T * h.double()).sum(0)   # every other row's gradient is the same
    for k in (0, 1 << 19, V - 301):
        assert _rel(_f64(b["dw"][k]), _f64(rest)) <= 2.0 ** -7


def test_repeats_bit_for_bit_on_another_stream():
    h, w, t = _inputs(400, 3001, 264, 16, ignored=0.1)
    f, b = _check(h, w, t, fp32=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f2 = api.linear_ce_forward(h, w, t)
        b2 = api.linear_ce_backward(h, w, t, f2["lse"], total=f2["total"], grad_fp32=True)
    side.synchronize()
    for k in ("loss", "lse", "total"):
        assert torch.equal(f[k], f2[k])
    assert torch.equal(b["dh"], b2["dh"]) and torch.equal(b["dw"], b2["dw"])


def test_captured_in_a_graph():
    h, w, t = _inputs(200, 900, 64, 17)
    api.linear_ce_forward(h, w, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = api.linear_ce_forward(h, w, t)
        b = api.linear_ce_backward(h, w, t, f["lse"], total=f["total"])
    h2, _, t2 = _inputs(200, 900, 64, 18)
    h.copy_(h2)
    t.copy_(t2)
    graph.replay()
    torch.cuda.synchronize()
    loss, _, dh, _ = _exact(h, w, t)
    np.testing.assert_allclose(_f64(f["loss"]), loss, rtol=0, atol=TOL_ROW)
    assert _rel(_f64(b["dh"]), dh) <= 2.0 ** -8


def test_leading_shape_and_refusals():
    h, w, t = _inputs(24, 90, 64, 19)
    f = api.linear_ce_forward(h.view(2, 12, 64), w, t.view(2, 12))
    assert f["loss"].shape == (2, 12)
    assert torch.equal(f["loss"].view(-1), api.linear_ce_forward(h, w, t)["loss"])
    with pytest.raises(TypeError):
        api.linear_ce_forward(h.float(), w, t)
    with pytest.raises(TypeError):
        api.linear_ce_forward(h, w, t.int())
    with pytest.raises(ValueError):
        api.linear_ce_forward(h[:, ::2], w[:, ::2], t)
    with pytest.raises(ValueError):
        api.linear_ce_forward(h, w, t[:5])
    with pytest.raises(ValueError):
        api.linear_ce_backward(h, w, t, f["lse"].view(-1))
    with pytest.raises(ValueError):
        api.linear_ce_forward(h, w, t, scratch=torch.empty(16, dtype=torch.uint8, device=DEV))
    for kw in ({"softcap": -1.0}, {"softcap": float("nan")}, {"softcap": float("inf")}):
        with pytest.raises(api.LrsError) as e:
            api.linear_ce_forward(h, w, t, **kw)
        assert e.value.status == 1
    with pytest.raises(api.LrsError) as e:
        api.linear_ce_forward(h[:, :12].contiguous(), w[:, :12].contiguous(), t)
    assert e.value.status == 2


@pytest.mark.parametrize("T,D", [(1, 24320), (1, 24328), (1, 24576), (1, 24584), (2, 12032), (2, 12040), (2, 12288),
                                 (2, 12296), (3, 8016), (3, 8024), (3, 8192), (3, 8200), (4, 6016), (4, 6024),
                                 (4, 6144), (4, 6152)])
def test_few_tokens_of_wide_models(T, D):
    """Either side of where a few tokens' rows of h stop fitting in shared memory (the inputs' sum of absolute terms
    stays below 2^7 at a quarter of the weights' spread elsewhere)."""
    _check(*_inputs(T, 300, D, seed=T + D, std=0.25))


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
def test_few_capped_tokens(T, fp32):
    _check(*_inputs(T, 4099, 64, seed=30 + T, std=4.0), softcap=5.0, fp32=fp32)


def _leave_in_shared_memory(value):
    """Fills every SM's operand slots with a value: what a later launch finds where it has not written."""
    h = torch.full((256, 1024), value, dtype=torch.bfloat16, device=DEV)
    w = torch.full((40000, 1024), value, dtype=torch.bfloat16, device=DEV)
    api.linear_ce_forward(h, w, torch.zeros(256, dtype=torch.int64, device=DEV))


@pytest.mark.parametrize("T", [5, 20, 40, 60, 70, 100, 120, 333])
def test_capped_results_do_not_depend_on_what_ran_before(T):
    h, w, t = _inputs(T, 1000, 256, 40 + T, ignored=0.1 if T > 8 else 0.0)
    results = []
    for value in (0.0, 3e4, -3e4):
        _leave_in_shared_memory(value)
        f = api.linear_ce_forward(h, w, t, softcap=30.0)
        _leave_in_shared_memory(value)
        b = [api.linear_ce_backward(h, w, t, f["lse"], total=f["total"], softcap=30.0, grad_fp32=k) for k in (False, True)]
        results.append([f["loss"], f["lse"], f["total"]] + [x[k] for x in b for k in ("dh", "dw")])
    for r in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], r))


def test_capped_rows_do_not_depend_on_their_neighbours():
    """Rows whose logits reach the cap leave the other rows as they are, bit for bit."""
    h, w, t = _inputs(96, 700, 136, 50)
    big = h.clone()
    big[::2] *= 64
    dloss = torch.full((96,), 0.01, device=DEV)
    for fp32 in (False, True):
        got = []
        for x in (h, big):
            f = api.linear_ce_forward(x, w, t, softcap=30.0)
            b = api.linear_ce_backward(x, w, t, f["lse"], dloss, softcap=30.0, grad_fp32=fp32)
            got.append([f["loss"], f["lse"], b["dh"]])
        assert all(torch.equal(x[1::2], y[1::2]) for x, y in zip(*got))
    _check(big, w, t, softcap=30.0)


@pytest.mark.parametrize("fp32", [False, True])
def test_capped_rows_that_do_not_count_may_hold_anything(fp32):
    h, w, t = _inputs(150, 600, 64, 51)
    t[::3] = -1
    bad = h.clone()
    bad[0], bad[3], bad[6], bad[147] = float("nan"), float("inf"), 1e4, float("-inf")
    got = []
    for x in (h, bad):
        f = api.linear_ce_forward(x, w, t, softcap=30.0)
        b = api.linear_ce_backward(x, w, t, f["lse"], total=f["total"], softcap=30.0, grad_fp32=fp32)
        got.append([f["loss"][t >= 0], f["total"], b["dh"], b["dw"]])
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("T,V,D", [(3, 257, 72), (200, 1111, 136)])
def test_weights_of_either_sign(T, V, D, fp32):
    h, w, t = _inputs(T, V, D, 60, ignored=0.2 if T > 8 else 0.0)
    _check(h, w, t, dloss=torch.randn(T, generator=torch.Generator().manual_seed(61)).to(DEV) / T, fp32=fp32)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_weight_that_is_not_finite_stays_in_its_row(bad, fp32):
    """dh of the other tokens is what it is without that token; dw, a sum over all of them, has no finite value."""
    h, w, t = _inputs(150, 600, 64, 62)
    t[5] = -1
    dloss = torch.rand(150, generator=torch.Generator().manual_seed(63)).to(DEV) / 150
    f = api.linear_ce_forward(h, w, t)
    dloss[17] = 0.0
    clean = api.linear_ce_backward(h, w, t, f["lse"], dloss, grad_fp32=fp32)
    dloss[17] = bad
    got = api.linear_ce_backward(h, w, t, f["lse"], dloss, grad_fp32=fp32)
    rest = torch.arange(150, device=DEV) != 17
    assert torch.equal(got["dh"][rest], clean["dh"][rest])
    assert not torch.isfinite(got["dh"][17]).any() and not torch.isfinite(got["dw"]).any()
    # where no weight but that one is other than zero
    dloss.zero_()
    dloss[17] = bad
    got = api.linear_ce_backward(h, w, t, f["lse"], dloss, grad_fp32=fp32)
    assert not got["dh"][rest].any() and not torch.isfinite(got["dh"][17]).any()
    # of a token that is not counted it reaches nothing
    dloss.fill_(0.01)
    clean = api.linear_ce_backward(h, w, t, f["lse"], dloss, grad_fp32=fp32)
    dloss[5] = bad
    got = api.linear_ce_backward(h, w, t, f["lse"], dloss, grad_fp32=fp32)
    assert torch.equal(got["dh"], clean["dh"]) and torch.equal(got["dw"], clean["dw"])


@pytest.mark.parametrize("T,grad_fp32", [(3, False), (70, False), (333, True)])
def test_rows_of_a_longer_batch(T, grad_fp32):
    """The next token's targets as a view of the tokens, and a batch's rows from the second on: contiguous, and
    aligned to their elements only."""
    h, w, t = _inputs(T + 1, 900, 64, 70 + T, ignored=0.1 if T > 8 else 0.0)
    dloss = torch.rand(T + 1, generator=torch.Generator().manual_seed(71)).to(DEV) / T
    whole = api.linear_ce_forward(h, w, t)
    assert t[1:].data_ptr() % 16 and dloss[1:].data_ptr() % 16 and whole["lse"][1:].data_ptr() % 16
    f = api.linear_ce_forward(h[1:], w, t[1:])
    g = api.linear_ce_forward(h[1:], w, t[1:].clone())
    assert all(torch.equal(f[k], g[k]) for k in ("loss", "lse", "total"))
    pair = torch.stack([torch.zeros_like(g["total"]), g["total"]]).view(-1)[1:3]   # a total of 4-byte alignment
    pair.copy_(g["total"])
    for weights, total in ((dloss[1:], None), (None, pair)):
        lse = torch.cat([g["lse"][:1], g["lse"]])[1:]
        b = api.linear_ce_backward(h[1:], w, t[1:], lse, weights, total=total, grad_fp32=grad_fp32)
        c = api.linear_ce_backward(h[1:], w, t[1:].clone(), g["lse"], None if weights is None else weights.clone(),
                                   total=g["total"], grad_fp32=grad_fp32)
        assert torch.equal(b["dh"], c["dh"]) and torch.equal(b["dw"], c["dw"])


@pytest.mark.parametrize("fp32", [False, True])
def test_pieces_of_the_vocabulary_with_weights_and_a_cap(fp32):
    T, V, D = 70000, 5000, 8
    assert T * V * 2 > 512 << 20
    h, w, t = _inputs(T, V, D, 80, std=4.0)
    keep = torch.sort(torch.randperm(T, generator=torch.Generator().manual_seed(81))[:300]).values.to(DEV)
    # only 300 tokens are counted, so that the 64-bit definition needs only those
    t2 = torch.full_like(t, -1)
    t2[keep] = t[keep]
    dloss = torch.randn(T, generator=torch.Generator().manual_seed(82)).to(DEV) / 300
    f = api.linear_ce_forward(h, w, t2, softcap=5.0)
    b = api.linear_ce_backward(h, w, t2, f["lse"], dloss, softcap=5.0, grad_fp32=fp32)
    loss, _, dh, dw, bh, bw = _exact(h[keep], w, t2[keep], dloss[keep], 5.0, "fp32" if fp32 else "bf16")
    np.testing.assert_allclose(_f64(f["loss"][keep]), loss, rtol=0, atol=TOL_ROW)
    for got, ref, most in ((b["dh"][keep], dh, bh), (b["dw"], dw, bw)):
        assert (np.abs(_f64(got) - ref) - most).max() <= 0
        assert _rel(_f64(got), ref) <= (2.0 ** -16 + TOL_ROW if fp32 else 2.0 ** -8)
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[keep] = False
    assert not b["dh"][rest].any()


@pytest.mark.parametrize("T,V,D", [(3, 3000, 4096), (200, 1000, 4096), (300, 5000, 256), (2000, 300, 64), (9000, 40, 64),
                                   (256, 3000, 2056)])
def test_fp32_results_are_fp32(T, V, D):
    """Relative L2 errors of everything that is FP32 stay below 1e-6.  The tensor cores truncate their sums, about
    2e-8 of the value a step of 16 products; a chain of a logit has 64 steps (1.3e-6 of a number that lse and the
    exponentials see with the same error), a chain of a gradient 24 (5e-7); dz is held to 24 bits (6e-8); FP32 and the
    fast exponentials add 2e-7."""
    h, w, t = _inputs(T, V, D, 90 + D, ignored=0.1 if T > 8 else 0.0)
    dloss = torch.rand(T, generator=torch.Generator().manual_seed(91)).to(DEV) / T
    f = api.linear_ce_forward(h, w, t)
    b = api.linear_ce_backward(h, w, t, f["lse"], dloss, grad_fp32=True)
    exact = _exact(h, w, t, dloss)
    for got, ref in zip((f["loss"], f["lse"], b["dh"], b["dw"]), exact):
        assert _rel(_f64(got), ref) <= 1e-6


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("softcap", [1e-44, 1e-39, 1e-38, 1e20, 2.5e38, 3e38])
def test_caps_at_the_ends_of_their_range(T, softcap):
    """Next to nothing (every capped logit is 0 to FP32: the loss is log V) and next to no cap at all.  (A tiny cap's
    gradient is 0 where its logit is not.)"""
    h, w, t = _inputs(T, 300, 64, 100)
    softcap = float(np.float32(softcap))
    _check(h, w, t, softcap=softcap)
    _check(h, w, t, softcap=softcap, fp32=True)
    h[0] = 0   # logits of exactly 0
    f = api.linear_ce_forward(h, w, t, softcap=softcap)
    b = api.linear_ce_backward(h, w, t, f["lse"], total=f["total"], softcap=softcap)
    assert abs(float(f["loss"][0]) - np.log(300)) <= TOL_ROW
    assert torch.isfinite(b["dh"]).all() and torch.isfinite(b["dw"]).all()


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("softcap", [0.0, 5.0, 30.0])
@pytest.mark.parametrize("T,V,D", [(70, 600, 1032), (260, 300, 2112), (4, 515, 1088)])
def test_logits_of_more_than_one_chain(T, V, D, softcap, fp32):
    h, w, t = _inputs(T, V, D, 110 + D, ignored=0.1 if T > 8 else 0.0)
    dloss = torch.rand(T, generator=torch.Generator().manual_seed(111)).to(DEV) / T
    _check(h, w, t, softcap=softcap, fp32=fp32)
    _check(h, w, t, softcap=softcap, dloss=dloss, fp32=fp32)
