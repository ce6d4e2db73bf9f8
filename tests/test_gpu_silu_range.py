"""SiLU and its slope over all of FP32's range of e^-r: in the convolution, and of the scan's gate.

sigmoid(r) = 1 / (1 + 2^t), t = -r log2 e.  t is rounded once (2^-24 of it) from a rounded log2 e (2^-26), which is
|r| (2^-24 + 2^-26) < 2^-23 |r| of 2^t, and of the sigmoid where r is far below 0; ex2 and the reciprocal add 2^-22 and
2^-23, sums and products 2^-24 each: together below 2^-20 + 2^-23 max(-r, 0).  A sigmoid below 2^-126 is 0.  SiLU is one product
more; its slope s (1 + r (1 - s)) has terms of both signs: 2^-19 of their absolute values, and the same 2^-23 max(-r, 0).
The convolution's argument has an error of its own, 2^-22 of its absolute terms (up to five of them, each sum and product
2^-24), which the results feel by their derivatives: SiLU by its slope, the slope by s (1 - s) (2 + |r|)."""
import pytest
import torch

import ssm_reference as ref
from linear_recurrence_sequence_gb300 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32
LOST = 2.0 ** -126
ARGUMENTS = (-120.0, -95.0, -90.0, -88.0, -87.5, -87.0, -86.0, -80.0, -60.0, -40.0, -20.0, -12.0, -8.0, -3.0, -1.0, 0.0,
             1.0, 3.0, 8.0, 20.0, 60.0, 90.0, 120.0, 1000.0)


def _far(r):
    return 2.0 ** -23 * torch.clamp(-r, min=0)


@pytest.mark.parametrize("W", [2, 3, 4])
def test_convolution(W):
    B, L, D = 2, 37, 8 * len(ARGUMENTS)
    gen = torch.Generator().manual_seed(W)

    def r(*shape, s=1.0, d=F):
        return (torch.randn(*shape, generator=gen) * s).to(d).to(DEV)

    x, w, dy = r(B, L, D, d=BF), r(W, D, s=0.05), r(B, L, D, d=BF)
    bias = torch.tensor(ARGUMENTS, device=DEV).repeat_interleave(8).contiguous()
    y = api.causal_conv_forward(x, w, bias)["y"]
    g = api.causal_conv_backward(dy, x, w, bias, grad_fp32=True)

    past = torch.cat([torch.zeros(B, W - 1, D, dtype=torch.float64, device=DEV), x.double()], 1)
    taps = [past[:, W - 1 - j:L + W - 1 - j] for j in range(W)]
    pre = bias.double() + sum(w[j].double() * taps[j] for j in range(W))
    off = 2.0 ** -22 * (bias.double().abs() + sum((w[j].double() * taps[j]).abs() for j in range(W)))
    v, slope, slope_abs = ref.silu(pre)
    s = torch.sigmoid(pre)
    most = v.abs() * (2.0 ** -20 + _far(pre)) + LOST * pre.abs() + 1.1 * off * slope_abs
    dslope = slope_abs * (2.0 ** -19 + _far(pre)) + LOST * (1 + pre.abs()) + 1.1 * off * s * (1 - s) * (2 + pre.abs())
    d, de = dy.double() * slope, dy.double().abs() * (dslope + 2.0 ** -24 * slope.abs())
    want = {"y": (v, most)}
    dx, dxe = torch.zeros_like(past), torch.zeros_like(past)
    dw, dwe = [], []
    for j in range(W):
        dx[:, W - 1 - j:L + W - 1 - j] += w[j].double() * d
        dxe[:, W - 1 - j:L + W - 1 - j] += w[j].double().abs() * (de + 2.0 ** -22 * d.abs())
        dw.append((d * taps[j]).sum((0, 1)))
        dwe.append((taps[j].abs() * (de + ref.LONG * d.abs())).sum((0, 1)))
    want |= {"dx": (dx[:, W - 1:], dxe[:, W - 1:]), "dweight": (torch.stack(dw), torch.stack(dwe)),
             "dbias": (d.sum((0, 1)), (de + ref.LONG * d.abs()).sum((0, 1)))}
    ref.check({"y": y, "dx": g["dx"], "dweight": g["dweight"], "dbias": g["dbias"]}, want)


def test_scans_gate():
    B, L, D, N = 2, 20, 8 * len(ARGUMENTS), 5
    gen = torch.Generator().manual_seed(1)

    def r(*shape, s=1.0, d=BF):
        return (torch.randn(*shape, generator=gen) * s).to(d).to(DEV)

    gate = (torch.tensor(ARGUMENTS).repeat_interleave(8) * (1 + 0.01 * torch.randn(B, L, D, generator=gen))).to(BF).to(DEV)
    i = {"x": r(B, L, D), "delta": r(B, L, D), "a_log": r(D, N, d=F), "b": r(B, L, N), "c": r(B, L, N), "d_skip": r(D, d=F),
         "delta_bias": None, "gate": gate, "h0": None, "reset": None}
    dy = r(B, L, D)
    f = api.selective_scan_forward(**i)
    g = api.selective_scan_backward(dy, None, *i.values(), f["saved"], grad_fp32=True)
    want = ref.scan(**i, dy=dy)
    mixed = ref.scan(**{**i, "gate": None})["y"][0]
    z = gate.double()
    v, slope, slope_abs = ref.silu(z)
    y, ye = want["y"]
    ref.check({"y": f["y"]}, {"y": (y, ye + mixed.abs() * (v.abs() * _far(z) + LOST * z.abs()))})
    q, qe = want["dgate"]
    more = (dy.double() * mixed).abs() * (slope_abs * _far(z) + LOST * (1 + z.abs()))
    ref.check({"dgate": g["dgate"]}, {"dgate": (q, qe + more)})
