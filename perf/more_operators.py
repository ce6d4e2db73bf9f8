"""Cases of the operators around a selective state space mixer: its short causal convolution, its scan (prompts,
training and single tokens) and the embedding lookup at the bottom of the stack with its gradient.

``run(state)`` is one pass: the plain form (elementary torch operations in 32 bits, rounded once at the end), or,
where ``own`` is true, the calls that a user makes of linear_recurrence_sequence_gb300.api.  ``exact`` is the
definition in 64 bits.
"""
import math

import torch

own = False

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def _api():
    from linear_recurrence_sequence_gb300 import api
    return api


# ----------------------------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------------------------
def _conv(name, kind, B, L, D, W=4, silu=True, bias=True, carried=False, reset=0.0, fp32=False):
    return {"name": name, "op": "conv", "kind": kind, "B": B, "L": L, "D": D, "W": W, "silu": silu, "bias": bias,
            "carried": carried, "reset": reset, "fp32": fp32}


def _scan(name, kind, B, L, D, N=16, gate=True, skip=True, carried=False, reset=0.0, fp32=False):
    return {"name": name, "op": "scan", "kind": kind, "B": B, "L": L, "D": D, "N": N, "gate": gate, "skip": skip,
            "carried": carried, "reset": reset, "fp32": fp32}


def _embed(name, kind, T, V, D, padding=0.0, scale=1.0, fp32=False, tied=False):
    return {"name": name, "op": "embed", "kind": kind, "T": T, "V": V, "D": D, "padding": padding, "scale": scale,
            "fp32": fp32, "tied": tied}


def listed():
    return [
        # one token of each of 64 sequences: the carried inputs move on by one
        _conv("conv_step", "step", 64, 1, 2048, carried=True),
        # the block benchmark's batch in training
        _conv("conv_train", "train", 4, 4096, 1024),
        # the block benchmark's wide prompt, continued from an earlier part
        _conv("conv_prompt", "prompt", 1, 8192, 2560, carried=True),
        # packed sequences of odd lengths, three taps, FP32 gradients
        _conv("conv_ragged", "train", 3, 1009, 328, W=3, carried=True, reset=1 / 100, fp32=True),
        # one token of each of 256 sequences: the decode benchmark's batch and width
        _scan("scan_step", "step", 256, 1, 2048, carried=True),
        # the wide prompt, continued from a carried state
        _scan("scan_prompt", "prompt", 1, 8192, 2560, carried=True),
        # packed sequences of odd lengths, 12 states a channel, FP32 gradients
        _scan("scan_ragged", "train", 3, 1009, 328, N=12, carried=True, reset=1 / 100, fp32=True),
        # the block benchmark's batch in training
        _scan("scan_train", "train", 4, 4096, 1024),
        # one long sequence in training, the mixer benchmark's own shape
        _scan("scan_train_long", "train", 1, 32768, 2048),
        # the tokens of one decoding step of 64 sequences
        _embed("embed_step", "lookup", 64, 32768, 1024),
        # a training step's batch (4 x 4096) against the vocabulary of the loss's benchmark
        _embed("embed_train", "train", 16384, 32768, 1024, scale=32.0, fp32=True),
        # a ragged batch with padding whose gradient joins that of a tied head
        _embed("embed_tied", "train", 5001, 50021, 2560, padding=0.1, tied=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 8, odd multiples among them."""
    return _log(rng, lo, hi) // 8 * 8


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "embed"])
    if op == "embed":
        kind = rng.choice(["lookup", "train", "train"])
        while True:
            T, V, D = _log(rng, 1, 65536), _log(rng, 100, 131072), _width(rng, 64, 4096)
            if T * D <= 1 << 26 and V * D <= 1 << 28:
                break
        c = _embed("", kind, T, V, D, rng.choice([0.0, 0.1, 0.5]), rng.choice([1.0, 32.0]),
                   kind == "train" and rng.random() < 0.5, kind == "train" and rng.random() < 0.4)
    else:
        kind = rng.choice(["step", "prompt", "train", "train"])
        while True:
            B, L, D = _log(rng, 1, 8), _log(rng, 1, 32768), _width(rng, 64, 4096)
            if kind == "step":
                B, L = _log(rng, 1, 1024), 1
            N = rng.choice([4, 8, 12, 16, 16, 16, 32, 64])
            if B * L * D <= 1 << 26 and (op == "conv" or B * L * D * N <= 1 << 30):
                break
        flags = {"carried": kind == "step" or rng.random() < 0.5, "reset": rng.choice([0.0, 0.0, 1 / 50, 1 / 1000]),
                 "fp32": kind == "train" and rng.random() < 0.4}
        if op == "conv":
            c = _conv("", kind, B, L, D, rng.choice([2, 3, 4, 4]), rng.random() < 0.8, rng.random() < 0.8, **flags)
        else:
            c = _scan("", kind, B, L, D, N, rng.random() < 0.75, rng.random() < 0.75, **flags)
    del c["name"]
    return c


# ----------------------------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _randn(gen, *shape, scale=1.0, dtype=F32):
    return torch.empty(shape, dtype=F32, device="cuda").normal_(generator=gen).mul_(scale).to(dtype)


def _uniform(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def prepare(case, seed):
    gen, s = _gen(seed), {"case": case}
    if case["op"] == "embed":
        return _prepare_embed(case, gen, s)
    B, L, D = case["B"], case["L"], case["D"]
    step = case["kind"] == "step"
    rows = (B,) if step else (B, L)
    # a projection's output: the branch and its gate, side by side
    s["proj"] = _randn(gen, *rows, 2 * D, dtype=BF)
    s["reset"] = (_uniform(gen, *rows) < case["reset"]).to(torch.uint8) if case["reset"] else None
    if case["op"] == "conv":
        W = case["W"]
        s["x"] = s["proj"][..., :D]
        s["weight"] = _randn(gen, W, D, scale=W ** -0.5)
        s["bias"] = _randn(gen, D, scale=0.1) if case["bias"] else None
        s["state"] = _randn(gen, B, W - 1, D, dtype=BF) if case["carried"] else None
    else:
        N = case["N"]
        x = s["proj"][..., :D].float()
        s["x"] = (x * torch.sigmoid(x)).to(BF)               # what the convolution leaves
        s["gate"] = s["proj"][..., D:] if case["gate"] else None
        s["delta"] = _randn(gen, *rows, D, scale=0.5, dtype=BF)
        dt = torch.exp(_uniform(gen, D) * math.log(100.0) + math.log(1e-3))   # steps of 1/1000 to 1/10
        s["delta_bias"] = dt + torch.log(-torch.expm1(-dt))
        s["a_log"] = torch.log(torch.arange(1, N + 1, device="cuda", dtype=F32)) + _randn(gen, D, N, scale=0.1)
        # the small projection of x: the step's low-rank part, then b and c
        s["small"] = _randn(gen, *rows, 64 + 2 * N, dtype=BF)
        s["b"], s["c"] = s["small"][..., 64:64 + N], s["small"][..., 64 + N:]
        s["d_skip"] = 1 + _randn(gen, D, scale=0.1) if case["skip"] else None
        s["h0"] = _randn(gen, B, D, N, scale=0.1) if case["carried"] else None
    if case["kind"] == "train":
        s["dy"] = _randn(gen, B, L, D, scale=0.01, dtype=BF)
        if case["op"] == "scan" and case["carried"]:
            s["dhT"] = _randn(gen, B, D, N, scale=0.01)
    return s


def _prepare_embed(case, gen, s):
    T, V, D = case["T"], case["V"], case["D"]
    # word frequencies: the k-th most common has a share of about 1 / k
    tokens = torch.exp(_uniform(gen, T).double() * math.log(V + 1.0)).long().clamp_(1, V) - 1
    if case["padding"]:
        tokens = torch.where(_uniform(gen, T) < case["padding"], torch.full_like(tokens, -1), tokens)
    s["tokens"] = tokens
    s["w"] = _randn(gen, V, D, scale=D ** -0.5, dtype=BF)
    if case["kind"] == "train":
        s["dy"] = _randn(gen, T, D, scale=0.01, dtype=BF)
        if case["tied"]:   # the head's gradient, which this one joins
            s["dw"] = _randn(gen, V, D, scale=0.01, dtype=F32 if case["fp32"] else BF)
    return s


# ----------------------------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "conv":
        return _conv_own(state) if own else _conv_plain(state)
    if op == "scan":
        return _scan_own(state) if own else _scan_plain(state)
    return _embed_own(state) if own else _embed_plain(state)


def _given(d, keys):
    return {k: d[k] for k in keys if d[k] is not None}


# the convolution ------------------------------------------------------------------------------------------------
def _conv_own(s):
    api, c = _api(), s["case"]
    if c["kind"] == "step":
        o = api.causal_conv_step(s["x"], s["weight"], s["bias"], s["state"], s["reset"], silu=c["silu"])
        return {"y": o["y"], "state": o["state"]}
    f = api.causal_conv_forward(s["x"], s["weight"], s["bias"], s["state"], s["reset"], silu=c["silu"])
    out = {"y": f["y"], "state": f["state"]}
    if c["kind"] == "train":
        b = api.causal_conv_backward(s["dy"], s["x"], s["weight"], s["bias"], s["state"], s["reset"], silu=c["silu"],
                                     grad_fp32=c["fp32"])
        out |= _given(b, ("dx", "dweight", "dbias", "dstate"))
    return out


def _conv_plain(s):
    c = s["case"]
    step = c["kind"] == "step"
    x = s["x"].float()
    x, reset = (x[:, None], None if s["reset"] is None else s["reset"][:, None]) if step else (x, s["reset"])
    B, L, D = x.shape
    W = c["W"]
    before = torch.zeros(B, W - 1, D, device="cuda") if s["state"] is None else s["state"].float()
    past = torch.cat([before, x], 1)                       # position t + W - 1 holds x[t]
    w = s["weight"]
    pos = torch.arange(L, device="cuda")[:, None] + torch.arange(W - 1, -1, -1, device="cuda")   # [L, W]: where tap j reads
    taps = past[:, pos]                                    # [B, L, W, D]
    live = None
    if reset is not None:
        seg = torch.cat([torch.zeros(B, W - 1, device="cuda"), reset.float().cumsum(1)], 1)
        live = (seg[:, pos] == seg[:, W - 1:, None])[..., None]
        taps = torch.where(live, taps, torch.zeros_like(taps))
        past = torch.where((seg == seg[:, -1:])[..., None], past, torch.zeros_like(past))
    pre = (taps * w).sum(2)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    sig = torch.sigmoid(pre)
    y = pre * sig if c["silu"] else pre
    after = past[:, L:].to(BF)
    if step:
        s["state"].copy_(after)
        return {"y": y[:, 0].to(BF), "state": s["state"]}
    out = {"y": y.to(BF), "state": after}
    if c["kind"] == "train":
        kind = F32 if c["fp32"] else BF
        d = s["dy"].float()
        if c["silu"]:
            d = d * sig * (1 + pre * (1 - sig))
        dt = d[:, :, None] * w                             # [B, L, W, D]: to what tap j read
        if live is not None:
            dt = torch.where(live, dt, torch.zeros_like(dt))
        dpast = torch.zeros(B, L + W - 1, D, device="cuda").index_add_(1, pos.flatten(), dt.flatten(1, 2))
        out["dx"] = dpast[:, W - 1:].to(kind)
        out["dweight"] = (d[:, :, None] * taps).sum((0, 1))
        if s["bias"] is not None:
            out["dbias"] = d.sum((0, 1))
        if s["state"] is not None:
            out["dstate"] = dpast[:, :W - 1].to(kind)
    return out


# the scan -------------------------------------------------------------------------------------------------------
def _scan_own(s):
    api, c = _api(), s["case"]
    a = (s["x"], s["delta"], s["a_log"], s["b"], s["c"], s["d_skip"], s["delta_bias"], s["gate"], s["h0"], s["reset"])
    if c["kind"] == "step":
        o = api.selective_scan_step(*a)
        return {"y": o["y"], "state": o["state"]}
    f = api.selective_scan_forward(*a, keep=c["kind"] == "train")
    out = {"y": f["y"], "hT": f["hT"]}
    if c["kind"] == "train":
        g = api.selective_scan_backward(s["dy"], s.get("dhT"), *a, f["saved"], grad_fp32=c["fp32"])
        out |= _given(g, ("dx", "ddelta", "da_log", "db", "dc", "dd_skip", "ddelta_bias", "dgate", "dh0"))
    return out


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1 from h = 0: pairs first, then what lies between them."""
    L = b.shape[1]
    if L == 1:
        return b
    odd = _recur(a[:, 1::2] * a[:, :L - 1:2], a[:, 1::2] * b[:, :L - 1:2] + b[:, 1::2])
    h = torch.empty_like(b)
    h[:, 1::2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, :(L - 1) // 2] + b[:, 2::2]
    return h


def _scan_plain(s):
    c = s["case"]
    step = c["kind"] == "step"

    def rows(t):
        return None if t is None else (t[:, None] if step else t).float()

    x, delta, b, cc, gate, reset = (rows(s[k]) for k in ("x", "delta", "b", "c", "gate", "reset"))
    raw = delta + s["delta_bias"]
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    rate = -torch.exp(s["a_log"])                                       # [D, N]
    keep = torch.exp(dt[..., None] * rate)                              # [B, L, D, N]
    if reset is not None:
        keep = torch.where(reset[:, :, None, None] != 0, torch.zeros_like(keep), keep)
    add = (dt * x)[..., None] * b[:, :, None]
    if s["h0"] is not None:
        add[:, 0] += keep[:, 0] * s["h0"]
    h = _recur(keep, add)
    del add
    mixed = (h * cc[:, :, None]).sum(3)
    if s["d_skip"] is not None:
        mixed = mixed + s["d_skip"] * x
    sig = None if gate is None else torch.sigmoid(gate)
    y = mixed if gate is None else mixed * gate * sig
    if step:
        s["h0"].copy_(h[:, 0])
        return {"y": y[:, 0].to(BF), "state": s["h0"]}
    out = {"y": y.to(BF), "hT": h[:, -1].contiguous()}
    if c["kind"] == "train":
        kind = F32 if c["fp32"] else BF
        dy = s["dy"].float()
        if gate is not None:
            out["dgate"] = (dy * mixed * sig * (1 + gate * (1 - sig))).to(kind)
            dy = dy * gate * sig
        out["dc"] = torch.einsum("bld,bldn->bln", dy, h).to(kind)
        # the adjoint g_t = dy_t c_t + keep_{t+1} g_{t+1}
        push = dy[..., None] * cc[:, :, None]
        if "dhT" in s:
            push[:, -1] += s["dhT"]
        after = torch.cat([keep[:, 1:], torch.zeros_like(keep[:, :1])], 1)
        g = _recur(after.flip(1), push.flip(1)).flip(1)
        del push, after
        if s["h0"] is not None:
            out["dh0"] = keep[:, 0] * g[:, 0]
        before = torch.cat([torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None], h[:, :-1]], 1)
        q = g * keep * before                                           # d / d (dt rate)
        del keep, before, h
        gb = torch.einsum("bldn,bln->bld", g, b)
        out["db"] = torch.einsum("bldn,bld->bln", g, dt * x).to(kind)
        del g
        dx = gb * dt
        if s["d_skip"] is not None:
            dx = dx + dy * s["d_skip"]
            out["dd_skip"] = (dy * x).sum((0, 1))
        out["dx"] = dx.to(kind)
        out["da_log"] = (q * dt[..., None]).sum((0, 1)) * rate
        ddelta = (gb * x + (q * rate).sum(3)) * torch.sigmoid(raw)
        out["ddelta"] = ddelta.to(kind)
        out["ddelta_bias"] = ddelta.sum((0, 1))
    return out


# the embedding --------------------------------------------------------------------------------------------------
def _embed_own(s):
    api, c = _api(), s["case"]
    out = {"y": api.embedding_forward(s["tokens"], s["w"], scale=c["scale"])["y"]}
    if c["kind"] == "train":
        given = {"out": {"dw": s["dw"]}, "accumulate": True} if c["tied"] else {}
        out["dw"] = api.embedding_backward(s["dy"], s["tokens"], c["V"], scale=c["scale"], grad_fp32=c["fp32"],
                                           **given)["dw"]
    return out


def _embed_plain(s):
    c, t = s["case"], s["tokens"]
    live = (t >= 0)[:, None]
    at = t.clamp(min=0)
    y = torch.where(live, s["w"][at].float() * c["scale"], torch.zeros((), device="cuda"))
    out = {"y": y.to(BF)}
    if c["kind"] == "train":
        d = torch.where(live, s["dy"].float() * c["scale"], torch.zeros((), device="cuda"))
        dw = s["dw"].float() if c["tied"] else torch.zeros(c["V"], c["D"], device="cuda")
        dw = torch.index_add(dw, 0, at, d)
        if c["tied"]:
            s["dw"].copy_(dw)
            out["dw"] = s["dw"]
        else:
            out["dw"] = dw.to(F32 if c["fp32"] else BF)
    return out


# ----------------------------------------------------------------------------------------------------------------
# Work and the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "embed":
        T, V, D = case["T"], case["V"], case["D"]
        live = T * (1 - case["padding"])
        seen = V * (1 - math.exp(-live / V))                # rows that are looked up, at most
        n = 8 * T + 2 * T * D + 2 * min(live, seen) * D
        if case["kind"] == "train":
            size = 4 if case["fp32"] else 2
            n += 8 * T + 2 * live * D + (2 * seen if case["tied"] else V) * size * D
        return {"bytes": n, "flops": 2 * T * D}
    B, L, D = case["B"], case["L"], case["D"]
    n, grad = B * L * D, 4 if case["fp32"] else 2
    if case["op"] == "conv":
        W = case["W"]
        taps = B * (W - 1) * D * 2
        moved = 4 * n + 4 * (W + 1) * D + taps * (1 + case["carried"])
        if case["kind"] == "train":
            moved += n * (2 + grad) + 4 * (W + 1) * D + B * (W - 1) * D * grad * case["carried"]
        return {"bytes": moved, "flops": n * (2 * W + 6) * (3 if case["kind"] == "train" else 1)}
    N = case["N"]
    streams = 2 + case["gate"]                              # x, delta and the gate
    params = 4 * D * (N + 2)
    state = 4 * B * D * N
    moved = n * 2 * (streams + 1) + 4 * B * L * N + params + state * (1 + case["carried"])
    flops = 7 * n * N
    if case["kind"] == "train":
        moved += n * (2 + grad * streams) + 2 * grad * B * L * N + params + 2 * state * case["carried"]
        flops += 20 * n * N
    return {"bytes": moved, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _conv_exact, "scan": _scan_exact, "embed": _embed_exact}[case["op"]](case, s)


def _conv_exact(case, s):
    step, W, D = case["kind"] == "step", case["W"], case["D"]
    x = s["x"].double()
    x = x[:, None] if step else x
    B, L, _ = x.shape
    reset = torch.zeros(B, L, device="cuda") if s["reset"] is None else s["reset"].view(B, L)
    x.requires_grad_(True)
    before = torch.zeros(B, W - 1, D, dtype=F64, device="cuda") if s["state"] is None else s["state"].double()
    before.requires_grad_(True)
    weight = s["weight"].double().requires_grad_(True)
    bias = (torch.zeros(D, device="cuda") if s["bias"] is None else s["bias"]).double().requires_grad_(True)
    pre, lag, open_ = bias.expand(B, L, D), x, torch.ones(B, L, 1, dtype=F64, device="cuda")
    for j in range(W):
        if j:   # the input j tokens earlier, and whether no segment starts in between
            lag = torch.cat([before[:, W - 1 - j:], x[:, :max(0, L - j)]], 1)[:, :L]
            cut = torch.zeros(B, L, 1, dtype=F64, device="cuda")
            cut[:, j - 1:, 0] = (reset[:, :max(0, L - j + 1)] != 0).double()
            open_ = open_ * (1 - cut)
        pre = pre + weight[j] * lag * open_
    y = torch.nn.functional.silu(pre) if case["silu"] else pre
    rows = torch.cat([before, x], 1).detach()[:, L:].clone()
    for b in range(B) if case["reset"] else ():
        starts = torch.nonzero(reset[b] != 0)[:, 0].tolist()
        if starts and L - starts[-1] < W - 1:
            rows[b, :W - 1 - (L - starts[-1])] = 0
    if step:
        return {"y": y[:, 0].detach(), "state": rows}
    out = {"y": y.detach(), "state": rows}
    if case["kind"] == "train":
        g = torch.autograd.grad(y, (x, weight, bias, before), s["dy"].double(), allow_unused=True)
        g = [torch.zeros_like(v) if d is None else d for d, v in zip(g, (x, weight, bias, before))]
        out |= {"dx": g[0], "dweight": g[1]}
        if s["bias"] is not None:
            out["dbias"] = g[2]
        if s["state"] is not None:
            out["dstate"] = g[3]
    return out


def _scan_exact(case, s):
    """Token after token, then back."""
    B, L, D, N = case["B"], case["L"], case["D"], case["N"]
    train = case["kind"] == "train"
    if train and B * L * D * N > 1 << 30:
        return None

    def rows(k, n):
        return s[k].double().reshape(B, L, n)

    x, b, c = rows("x", D), rows("b", N), rows("c", N)
    raw = rows("delta", D) + s["delta_bias"].double()
    dt = torch.nn.functional.softplus(raw, threshold=700)
    rate = -s["a_log"].double().exp()
    start = torch.zeros(B, D, N, dtype=F64, device="cuda") if s["h0"] is None else s["h0"].double()
    cut = [False] * L
    if s["reset"] is not None:
        fresh = s["reset"].view(B, L) != 0
        cut = fresh.any(0).tolist()
    h, mixed = start, torch.empty(B, L, D, dtype=F64, device="cuda")
    kept = torch.empty(L, B, D, N, dtype=F64, device="cuda") if train else None
    for t in range(L):
        if train:
            kept[t] = h
        if cut[t]:
            h = torch.where(fresh[:, t, None, None], 0.0, h)
        h = torch.addcmul(torch.exp(dt[:, t, :, None] * rate) * h, (dt[:, t] * x[:, t])[..., None], b[:, t, None])
        mixed[:, t] = torch.matmul(h, c[:, t, :, None])[..., 0]
    skip = None if s["d_skip"] is None else s["d_skip"].double()
    if skip is not None:
        mixed += skip * x
    act = 1.0 if s["gate"] is None else torch.nn.functional.silu(rows("gate", D))
    y = mixed * act
    if case["kind"] == "step":
        return {"y": y[:, 0], "state": h}
    out = {"y": y, "hT": h}
    if not train:
        return out
    dy = s["dy"].double()
    if s["gate"] is not None:
        z = rows("gate", D)
        sg = torch.sigmoid(z)
        out["dgate"] = dy * mixed * (sg + z * sg * (1 - sg))
        dy = dy * act
    dx, ddt = torch.empty_like(x), torch.empty_like(x)
    db, dc = torch.empty_like(b), torch.empty_like(c)
    drate = torch.zeros_like(rate)
    g = torch.zeros_like(start) if "dhT" not in s else s["dhT"].double()
    for t in range(L - 1, -1, -1):
        a = torch.exp(dt[:, t, :, None] * rate)
        old = torch.where(fresh[:, t, None, None], 0.0, kept[t]) if cut[t] else kept[t]
        put = (dt[:, t] * x[:, t])[..., None]
        old = a * old                                       # what is left of the past
        dc[:, t] = torch.matmul(dy[:, t, None], old + put * b[:, t, None])[:, 0]
        g = torch.addcmul(g, dy[:, t, :, None], c[:, t, None])
        gb = torch.matmul(g, b[:, t, :, None])[..., 0]
        db[:, t] = torch.matmul(put.transpose(1, 2), g)[:, 0]
        q = g * old
        ddt[:, t] = gb * x[:, t] + (q * rate).sum(2)
        dx[:, t] = gb * dt[:, t]
        drate += (q * dt[:, t, :, None]).sum(0)
        g = g * a
        if cut[t]:
            g = torch.where(fresh[:, t, None, None], 0.0, g)
    if skip is not None:
        dx += dy * skip
        out["dd_skip"] = (dy * x).sum((0, 1))
    draw_ = ddt * torch.sigmoid(raw)
    out |= {"dx": dx, "ddelta": draw_, "ddelta_bias": draw_.sum((0, 1)), "db": db, "dc": dc, "da_log": drate * rate}
    if s["h0"] is not None:
        out["dh0"] = g
    return out


def _embed_exact(case, s):
    t, V = s["tokens"], case["V"]
    table = torch.cat([s["w"].double(), torch.zeros(1, case["D"], dtype=F64, device="cuda")])   # padding: the last row
    at = torch.where(t < 0, torch.full_like(t, V), t)
    out = {"y": table[at] * case["scale"]}
    if case["kind"] == "train":
        order = torch.argsort(at)
        dw = torch.zeros(V + 1, case["D"], dtype=F64, device="cuda").index_add_(0, at[order], s["dy"][order].double())
        dw = dw[:V] * case["scale"]
        out["dw"] = dw + s["dw"].double() if case["tied"] else dw
    return out
