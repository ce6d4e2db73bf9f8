"""The causal convolution and the selective scan in 64 bits, each result with a bound on the error of its evaluation
in FP32: the same expression with every term taken by its absolute value, times the errors of the steps below it.

What the bounds take (2^-24 is FP32's rounding): dt = softplus within 2^-21, ex2 within 2^-22, its argument within
2^-24 of itself.  e^r is 2^(r log2 e) of a product rounded once (2^-24 of it) with a rounded log2 e (2^-26): its exponent
is off by at most |r| log2 e (2^-24 + 2^-26), which is |r| (2^-24 + 2^-26) of the result, below 2^-23 |r|; dt at r << 0 and
sigmoid(r) have that error too (`far` below; next to 2^-21 it counts from |r| = 8 on).  Below 2^-126 the GPU's fast
functions give 0: LOST more.  So a step keeps its state within 2^-20 (1 + rate dt), and multiplies and adds within 2^-22
more.
SiLU and its slope within 2^-19 of their terms (ex2, a reciprocal, arguments of up to 8).  Sums over a token's states or
channels run in trees and short runs: 2^-18 of their absolute terms.  Sums over tokens: 2^-15."""
import torch

STEP, TREE, LONG, LOST = 2.0 ** -20, 2.0 ** -18, 2.0 ** -15, 2.0 ** -126


def silu(z):
    s = torch.sigmoid(z)
    return z * s, s * (1 + z * (1 - s)), s * (1 + z.abs() * (1 - s))   # value, slope, the slope's absolute terms


def scan(x, delta, a_log, b, c, d_skip=None, delta_bias=None, gate=None, h0=None, reset=None, dy=None, dhT=None):
    """{name: (value, bound)} of y, hT and, given dy, of every gradient."""
    dev = x.device
    x, delta, a_log, b, c = (t.double() for t in (x, delta, a_log, b, c))
    B, L, D = x.shape
    N = a_log.shape[1]
    zero = torch.zeros(D, dtype=torch.float64, device=dev)
    skip = zero if d_skip is None else d_skip.double()
    raw = delta + (zero if delta_bias is None else delta_bias.double())
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    far = 2.0 ** -23 * torch.clamp(-raw, min=0)
    far = torch.where(torch.isfinite(far), far, 0.0)   # dt is 0 at -inf
    rate = -torch.exp(a_log)
    if gate is None:
        act = slope = slope_abs = torch.ones_like(x)
        act_err = torch.zeros_like(x)
    else:
        act, slope, slope_abs = silu(gate.double())
        act_err = 2 * STEP * act.abs()
    h = torch.zeros(B, D, N, dtype=torch.float64, device=dev) if h0 is None else h0.double()
    ha, he = h.abs(), torch.zeros_like(h)
    put = dt * x
    mixed, ya, ye = (torch.empty_like(x) for _ in range(3))
    before = []
    for t in range(L):
        a = torch.exp(dt[:, t, :, None] * rate)
        if reset is not None:
            cut = (reset[:, t] != 0)[:, None, None]
            a, h, ha, he = (torch.where(cut, 0.0, v) for v in (a, h, ha, he))
        before.append((a, h, ha, he))
        add = put[:, t, :, None] * b[:, t, None]
        h, ha = a * h + add, a * ha + add.abs()
        he = a * he + (STEP + far[:, t, :, None]) * (1 + rate.abs() * dt[:, t, :, None]) * ha
        he = he + LOST * x[:, t, :, None].abs() * b[:, t, None].abs()
        mixed[:, t] = (h * c[:, t, None]).sum(2)
        ya[:, t] = (ha * c[:, t, None].abs()).sum(2)
        ye[:, t] = (he * c[:, t, None].abs()).sum(2)
    mixed, ya = mixed + skip * x, ya + (skip * x).abs()
    ye = ye + TREE * ya
    out = {"y": (mixed * act, ye * act.abs() + ya * act_err), "hT": (h, he)}
    if dy is None:
        return out
    dy = dy.double()
    if gate is not None:
        out["dgate"] = (dy * mixed * slope, dy.abs() * (ye * slope.abs() + 4 * STEP * ya * slope_abs))
    dp, dpa = dy * act, (dy * act).abs()
    u = torch.zeros_like(h) if dhT is None else dhT.double()
    ua, ue = u.abs(), torch.zeros_like(h)
    dx, dxe, dd, dde = (torch.empty_like(x) for _ in range(4))
    db, dbe, dc, dce = (torch.empty_like(b) for _ in range(4))
    dA, dAe, dAa = (torch.zeros_like(h) for _ in range(3))
    sig = torch.sigmoid(raw)
    for t in range(L - 1, -1, -1):
        a, hp, hpa, hpe = before[t]
        ct, bt, pt, dtt = c[:, t, None], b[:, t, None], put[:, t, :, None], dt[:, t, :, None]
        add = pt * bt
        ht, hta = a * hp + add, a * hpa + add.abs()
        ft = far[:, t, :, None]
        hte = a * hpe + (STEP + ft) * (1 + rate.abs() * dtt) * hta + LOST * x[:, t, :, None].abs() * bt.abs()
        dc[:, t] = (dp[:, t, :, None] * ht).sum(1)
        dce[:, t] = (dpa[:, t, :, None] * (hte + TREE * hta)).sum(1)
        G, Ga = dp[:, t, :, None] * ct + u, dpa[:, t, :, None] * ct.abs() + ua
        Ge = ue + 4 * STEP * Ga
        db[:, t] = (pt * G).sum(1)
        dbe[:, t] = (pt.abs() * (Ge + (TREE + ft) * Ga) + LOST * x[:, t, :, None].abs() * Ga).sum(1)
        s1, s1a, s1e = (G * bt).sum(2), (Ga * bt.abs()).sum(2), ((Ge + TREE * Ga) * bt.abs()).sum(2)
        u, ua = a * G, a * Ga
        ue = a * (Ge + (STEP + ft) * (1 + rate.abs() * dtt) * Ga)
        r, ra = u * hp, ua * hpa
        re = ue * hpa + ua * hpe + 4 * STEP * ra
        q, qe = (rate * r).sum(2), (rate.abs() * (re + TREE * ra)).sum(2)
        dx[:, t] = s1 * dt[:, t] + skip * dp[:, t]
        dxe[:, t] = (s1e + far[:, t] * s1a) * dt[:, t] + LOST * s1a + 4 * STEP * (skip * dp[:, t]).abs()
        dd[:, t] = (s1 * x[:, t] + q) * sig[:, t]
        dde[:, t] = (s1e * x[:, t].abs() + qe) * sig[:, t] + ((4 * STEP + far[:, t]) * sig[:, t] + LOST) * (
            s1a * x[:, t].abs() + (rate.abs() * ra).sum(2))
        dA, dAa, dAe = dA + dtt * r, dAa + dtt * ra, dAe + dtt * (re + ft * ra) + LOST * ra
    out |= {"dx": (dx, dxe), "ddelta": (dd, dde), "db": (db, dbe), "dc": (dc, dce),
            "da_log": ((rate * dA).sum(0), (rate.abs() * (dAe + LONG * dAa)).sum(0)),
            "ddelta_bias": (dd.sum((0, 1)), (dde + LONG * dd.abs()).sum((0, 1))),
            "dd_skip": ((dp * x).sum((0, 1)), LONG * (dp * x).abs().sum((0, 1))), "dh0": (u, ue)}
    return out


def conv(x, weight, bias=None, state=None, reset=None, silu_=True, dy=None):
    """{name: (value, bound)} of y, the state after x (exact) and, given dy, of every gradient."""
    x, weight = x.double(), weight.double()
    B, L, D = x.shape
    W = weight.shape[0]
    before = torch.zeros(B, W - 1, D, dtype=torch.float64, device=x.device) if state is None else state.double()
    past = torch.cat([before, x], 1)
    start = torch.zeros(B, L + W - 1, dtype=torch.bool, device=x.device)
    if reset is not None:
        start[:, W - 1:] = reset != 0
    seq = start.cumsum(1)
    pre = torch.zeros_like(x) + (0 if bias is None else bias.double())
    prea = pre.abs()
    taps = []
    for j in range(W):
        at = slice(W - 1 - j, L + W - 1 - j)
        live = (seq[:, at] == seq[:, W - 1:])[..., None].double()
        taps.append((live, torch.where(live > 0, past[:, at], 0.0), at))
        pre, prea = pre + weight[j] * taps[j][1], prea + (weight[j] * taps[j][1]).abs()
    pree = 2.0 ** -22 * prea
    if silu_:
        y, slope, slope_abs = silu(pre)
        ye = 1.1 * pree + 4 * STEP * y.abs()
        # the slope's own slope is within 1/2
        dslope = 0.5 * pree + 4 * STEP * slope_abs
    else:
        y, ye, slope, dslope = pre, pree, torch.ones_like(pre), torch.zeros_like(pre)
    after = torch.where((seq == seq[:, -1:])[..., None], past, 0.0)[:, L:]
    out = {"y": (y, ye), "state": (after, torch.zeros_like(after))}
    if dy is None:
        return out
    dy = dy.double()
    d, de = dy * slope, dy.abs() * (dslope + 2.0 ** -23 * slope.abs())
    dp, dpe = torch.zeros_like(past), torch.zeros_like(past)
    dw, dwe = torch.zeros_like(weight), torch.zeros_like(weight)
    for j, (live, v, at) in enumerate(taps):
        dp[:, at] += live * weight[j] * d
        dpe[:, at] += live * weight[j].abs() * (de + 2.0 ** -22 * d.abs())
        dw[j] = (d * v).sum((0, 1))
        dwe[j] = (v.abs() * (de + LONG * d.abs())).sum((0, 1))
    out |= {"dx": (dp[:, W - 1:], dpe[:, W - 1:]), "dstate": (dp[:, :W - 1], dpe[:, :W - 1]), "dweight": (dw, dwe),
            "dbias": (d.sum((0, 1)), (de + LONG * d.abs()).sum((0, 1)))}
    return out


def check(got, want, keys=None):
    """Every result within its bound and, in BF16, half a step of BF16 (2^-8 of the value, 2^-134 near zero) more."""
    for k in keys or got:
        if got.get(k) is None or k not in want:
            continue
        ref, most = want[k]
        assert got[k].shape == ref.shape, k
        if got[k].dtype == torch.bfloat16:
            most = most * (1 + 2.0 ** -7) + 2.0 ** -8 * ref.abs() + 2.0 ** -134
        else:
            assert got[k].dtype == torch.float32, k
            most = most + 2.0 ** -23 * ref.abs() + 2.0 ** -126
        off = (got[k].double() - ref).abs() - most
        assert not bool(torch.isnan(off).any()), k
        worst = float((off / most.clamp(min=1e-300)).max()) if off.numel() else -1.0
        assert float(off.max()) <= 0, (k, float(off.max()), worst)
