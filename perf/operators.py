"""Cases of the training step's operators: the vocabulary loss with its gradient, the gated pre/post norm of a
residual branch, and the AdamW step over many tensors.

``run(state)`` is one pass: the plain form (elementary torch operations in 32 bits, rounded once at the end), or,
where ``own`` is true, the calls that a user makes of linear_recurrence_sequence_gb300.api.  ``exact`` is the
definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
ADAM = {"beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "max_norm": 1.0, "lr": 1e-4}
FP8_MAX = 448.0       # largest E4M3 value
FP8_TINY = 2.0 ** -9  # smallest positive E4M3 value
QUANT = 256           # values that share one scale
SMALL = 2.0 ** -100   # a block of states below this is stored as zeros


def _api():
    from linear_recurrence_sequence_gb300 import api
    return api


# ----------------------------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------------------------
def _ce(name, kind, T, D, V, ignored=0.0, softcap=0.0, fp32=False, weighted=False):
    return {"name": name, "op": "ce", "kind": kind, "T": T, "D": D, "V": V, "ignored": ignored, "softcap": softcap,
            "fp32": fp32, "weighted": weighted}


def _norm(name, kind, T, D, branch=True, gate=True):
    return {"name": name, "op": "norm", "kind": kind, "T": T, "D": D, "branch": branch, "gate": gate}


def _adamw(name, bits, blocks, Dm, D, V, grad="fp32"):
    return {"name": name, "op": "adamw", "bits": bits, "blocks": blocks, "Dm": Dm, "D": D, "V": V, "grad": grad}


def listed():
    return [
        # scoring one token while serving: one row against the whole vocabulary, bound by reading the head
        _ce("ce_score_one", "score", 1, 1024, 32768),
        # scoring a long document, nothing kept for a backward pass
        _ce("ce_score_long", "score", 32768, 1024, 32768),
        # a short ragged batch while fine-tuning, padding not counted, nothing a multiple of a tile
        _ce("ce_train_ragged", "train", 333, 328, 5003, ignored=0.2, weighted=True),
        # the head of a training step of a small model (4 sequences of 1024)
        _ce("ce_train_step", "train", 4096, 1024, 32768, ignored=0.02),
        # FP32 gradients and capped logits, an odd vocabulary
        _ce("ce_train_fp32", "train", 2048, 1024, 50021, softcap=30.0, fp32=True),
        # the block benchmark's long sequence (1 x 8192 at stream width 2048) against a large vocabulary
        _ce("ce_train_large", "train", 8192, 2048, 65536, ignored=0.01),
        # the norm of one decoding step of 16 sequences
        _norm("norm_decode", "forward", 16, 2048),
        # a training step of the block benchmark's batch (4 x 4096 at width 1024)
        _norm("norm_train", "train", 16384, 1024),
        # the norm ahead of the head, a ragged number of tokens: no branch
        _norm("norm_final_ragged", "train", 5001, 2560, branch=False, gate=False),
        # one small block: launches and latency
        _adamw("adamw_small", 32, 1, 256, 256, 0),
        # eight wide blocks and their vocabulary matrix, 32-bit states
        _adamw("adamw_large", 32, 8, 2048, 2560, 65536),
        # four wide blocks with 8-bit states and BF16 gradients, an odd vocabulary
        _adamw("adamw_8bit", 8, 4, 2048, 2560, 50021, grad="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: a multiple of 8, odd multiples among them."""
    n = _log(rng, lo, hi) // 8 * 8
    return n + 8 if n == 3072 else n


def draw(rng):
    op = rng.choice(["ce", "ce", "norm", "adamw"])
    if op == "ce":
        while True:
            T, D, V = _log(rng, 1, 32768), _width(rng, 64, 4096), _log(rng, 100, 131072)
            if 1e6 < T * D * V <= 8192 * 2048 * 65536 and T * V <= 1 << 30:
                break
        kind = rng.choice(["score", "train", "train"])
        c = _ce("", kind, T, D, V, ignored=rng.choice([0.0, 0.02, 0.3]), softcap=rng.choice([0.0, 0.0, 30.0]),
                fp32=kind == "train" and rng.random() < 0.3, weighted=kind == "train" and rng.random() < 0.4)
    elif op == "norm":
        branch = rng.random() < 0.75
        c = _norm("", rng.choice(["forward", "train"]), _log(rng, 1, 32768), _width(rng, 64, 4096), branch,
                  branch and rng.random() < 0.75)
    else:
        Dm, D = 256 * rng.randint(1, 8), 256 * rng.randint(1, 10)
        c = _adamw("", rng.choice([8, 32]), rng.randint(1, 6), Dm, D, rng.choice([0, _log(rng, 300, 65536)]),
                   grad=rng.choice(["fp32", "bf16"]))
    del c["name"]
    return c


# ----------------------------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(gen, *shape, scale=1.0, dtype=torch.float32):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=gen)
    return t.mul_(scale).to(dtype)


def _block_shapes(Dm, D):
    """The parameters of one recurrent block: matrices (decayed, BF16 with FP32 masters) and vectors (FP32)."""
    M, F = D // 2, 3 * Dm
    mats = [2 * D * Dm, Dm * D, 2 * F * Dm, Dm * F]
    vecs = [Dm, 4 * D, D, M, M, D + 1, D + 1, 1, 1, Dm]
    return mats, vecs


def _layout(case):
    """Sizes of the matrices and of the vectors of a model, in order."""
    mats, vecs = _block_shapes(case["Dm"], case["D"])
    mats, vecs = mats * case["blocks"], vecs * case["blocks"]
    if case["V"]:
        mats.append(case["V"] * case["Dm"])
        vecs.append(case["Dm"])
    return mats, vecs


def _padded(sizes):
    """Offsets of tensors laid one after another on 256-element boundaries, and the length of them all."""
    at, n = [], 0
    for s in sizes:
        at.append(n)
        n += -(-s // QUANT) * QUANT
    return at, n


def _mask(sizes, n):
    """Where the flat buffer holds a tensor's values (the gaps between tensors hold zeros)."""
    at, _ = _padded(sizes)
    start = torch.zeros(n + 1, dtype=torch.int32)
    start[torch.tensor(at)] += 1
    start[torch.tensor([a + s for a, s in zip(at, sizes)])] -= 1
    return start[:n].cuda().cumsum(0, dtype=torch.int32).bool()


def _pieces(flat, sizes):
    return [flat[a:a + s] for a, s in zip(_padded(sizes)[0], sizes)]


def _pieces_q(scales, sizes):
    return [scales[a // QUANT:(a + s + QUANT - 1) // QUANT] for a, s in zip(_padded(sizes)[0], sizes)]


def prepare(case, seed):
    gen = _gen(seed)
    s = {"case": case}
    if case["op"] == "ce":
        T, D, V = case["T"], case["D"], case["V"]
        s["h"] = _randn(gen, T, D, dtype=torch.bfloat16)
        s["w"] = _randn(gen, V, D, scale=2.5 / math.sqrt(D), dtype=torch.bfloat16)
        t = torch.randint(0, V, (T,), generator=gen, device="cuda")
        drop = torch.rand(T, generator=gen, device="cuda") < case["ignored"]
        s["target"] = torch.where(drop, torch.full_like(t, -100), t)
        s["dloss"] = torch.rand(T, generator=gen, device="cuda") / T if case["weighted"] else None
    elif case["op"] == "norm":
        T, D = case["T"], case["D"]
        b = torch.bfloat16
        s["x"] = _randn(gen, T, D, scale=2.0, dtype=b)
        s["gamma_pre"] = 1 + _randn(gen, D, scale=0.1)
        for k in ("y", "gate", "gamma_post", "scale"):
            s[k] = None
        if case["branch"]:
            s["y"] = _randn(gen, T, D, scale=0.6, dtype=b)
            s["gamma_post"] = 1 + _randn(gen, D, scale=0.1)
            s["scale"] = 0.5 + _randn(gen, D, scale=0.1)
        if case["gate"]:
            s["gate"] = _randn(gen, T, D, dtype=b)
        if case["kind"] == "train":
            s["dr"] = _randn(gen, T, D, scale=0.01, dtype=b)
            s["dh"] = _randn(gen, T, D, scale=0.01, dtype=b)
    else:
        mats, vecs = _layout(case)
        for part, sizes in (("mat", mats), ("vec", vecs)):
            n = _padded(sizes)[1]
            live = _mask(sizes, n)
            g = torch.bfloat16 if part == "mat" and case["grad"] == "bf16" else torch.float32
            total = sum(mats) + sum(vecs)
            std = 2.0 / math.sqrt(total)   # a norm of about 2 before clipping
            p = _randn(gen, n, scale=0.02) * live
            s[part + "_p"] = p
            s[part + "_g"] = (_randn(gen, n, scale=std) * live).to(g)
            m = _randn(gen, n, scale=0.2 * std) * live
            v = (_randn(gen, n, scale=std).square() + 0.1 * std * std) * live
            if part == "mat":
                s["mat_b"] = p.to(torch.bfloat16)
            if part == "mat" and case["bits"] == 8:
                s["mat_m"], s["mat_ms"] = _quantise(m, False)
                s["mat_v"], s["mat_vs"] = _quantise(v.sqrt(), True)
            else:
                s[part + "_m"], s[part + "_v"] = m, v
            del p, m, v, live
        s["step"] = torch.full((1,), 100, dtype=torch.int32, device="cuda")
        s["lr"] = torch.full((1,), ADAM["lr"], dtype=torch.float32, device="cuda")
        s["taken"] = 100
        if own:
            s["plan"] = _plan(s, mats, vecs)
    return s


def _plan(s, mats, vecs):
    """The list of tensors that a training program hands over once."""
    q = s["case"]["bits"] == 8
    parts = [_pieces(s["mat_" + k], mats) for k in ("p", "b", "g", "m", "v")]
    scales = [_pieces_q(s[k], mats) if q else [None] * len(mats) for k in ("mat_ms", "mat_vs")] if q else \
        [[None] * len(mats)] * 2
    tensors = [{"param": b, "master": p, "grad": g, "m": m, "v": v, "m_scale": ms, "v_scale": vs, "weight_decay": 0.1}
               for p, b, g, m, v, ms, vs in zip(*parts, *scales)]
    tensors += [{"param": p, "grad": g, "m": m, "v": v, "weight_decay": 0.0}
                for p, g, m, v in zip(*[_pieces(s["vec_" + k], vecs) for k in ("p", "g", "m", "v")])]
    return _api().adamw_plan(tensors)


# ----------------------------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "ce":
        return _ce_own(state) if own else _ce_plain(state)
    if op == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    return _adamw_own(state) if own else _adamw_plain(state)


def _ce_own(s):
    api, c = _api(), s["case"]
    f = api.linear_ce_forward(s["h"], s["w"], s["target"], softcap=c["softcap"])
    out = {"loss": f["loss"], "lse": f["lse"], "total": f["total"]}
    if c["kind"] == "train":
        b = api.linear_ce_backward(s["h"], s["w"], s["target"], f["lse"], s["dloss"], total=f["total"],
                                   softcap=c["softcap"], grad_fp32=c["fp32"])
        out["dh"], out["dw"] = b["dh"], b["dw"]
    return out


def _ce_plain(s):
    c, h, w, target = s["case"], s["h"].float(), s["w"].float(), s["target"]
    cap = c["softcap"]
    z = h @ w.t()
    if cap:
        z = torch.tanh(z / cap) * cap
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    counted = target >= 0
    at = target.clamp(min=0)[:, None]
    loss = torch.where(counted, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    count = counted.sum().float()
    out = {"loss": loss, "lse": lse, "total": torch.stack([loss.sum(), count])}
    if c["kind"] == "train":
        weight = s["dloss"] if s["dloss"] is not None else 1.0 / count
        weight = torch.where(counted, weight, torch.zeros_like(lse))[:, None]
        dz = e.div_(total)
        dz.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        dz.mul_(weight)
        if cap:
            dz = dz * (1 - (z / cap).square())
        kind = torch.float32 if c["fp32"] else torch.bfloat16
        out["dh"], out["dw"] = (dz @ w).to(kind), (dz.t() @ h).to(kind)
    return out


def _norm_own(s):
    api = _api()
    a = (s["x"], s["y"], s["gate"], s["gamma_post"], s["scale"], s["gamma_pre"])
    f = api.gated_norm_forward(*a, eps=EPS)
    out = {"r": f["r"], "h": f["h"]} if s["y"] is not None else {"h": f["h"]}
    if s["case"]["kind"] == "train":
        b = api.gated_norm_backward(s["dr"], s["dh"], *a, f["saved"])
        out |= {k: b[k] for k in ("dx", "dy", "dgate", "dgamma_post", "dscale", "dgamma_pre") if b[k] is not None}
    return out


def _gelu(g):
    """The block's GeLU (tanh form) and its derivative."""
    k, a = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(k * (g + a * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * a * g * g)


def _norm_plain(s):
    return _norm_form(s, torch.float32, torch.bfloat16)


def _norm_form(s, kind, act):
    x, gpre = s["x"].to(kind), s["gamma_pre"].to(kind)
    branch, out = s["y"] is not None, {}
    r = x
    if branch:
        y, gpost, scale = s["y"].to(kind), s["gamma_post"].to(kind), s["scale"].to(kind)
        rstd1 = 1 / torch.sqrt(y.square().mean(1, keepdim=True) + EPS)
        p = y * rstd1
        n = p * gpost
        if s["gate"] is not None:
            gl, dgl = _gelu(s["gate"].to(kind))
        else:
            gl, dgl = torch.ones_like(x), None
        r = x + scale * gl * n
        out["r"] = r.to(act)
    rstd2 = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + EPS)
    q = r * rstd2
    out["h"] = (q * gpre).to(act)
    if s["case"]["kind"] == "train":
        dr, dh = s["dr"].to(kind), s["dh"].to(kind)
        a = dh * gpre
        dx = dr + rstd2 * (a - q * (a * q).mean(1, keepdim=True))
        out["dx"], out["dgamma_pre"] = dx.to(act), (dh * q).sum(0)
        if branch:
            out["dscale"] = (dx * gl * n).sum(0)
            if dgl is not None:
                out["dgate"] = (dx * scale * n * dgl).to(act)
            dn = dx * scale * gl
            out["dgamma_post"] = (dn * p).sum(0)
            b = dn * gpost
            out["dy"] = (rstd1 * (b - p * (b * p).mean(1, keepdim=True))).to(act)
    return out


def _adamw_outputs(s, norm):
    keys = ["mat_p", "mat_b", "mat_m", "mat_v", "vec_p", "vec_m", "vec_v"]
    keys += ["mat_ms", "mat_vs"] if s["case"]["bits"] == 8 else []
    return {**{k: s[k] for k in keys}, "norm": norm, "step": s["step"]}


def _adamw_own(s):
    o = _api().adamw_step(s["plan"], s["step"], s["lr"], beta1=ADAM["beta1"], beta2=ADAM["beta2"], eps=ADAM["eps"],
                          max_norm=ADAM["max_norm"])
    return _adamw_outputs(s, o["norm"])


def _quantise(x, root):
    """E4M3 codes and scales of flat states, 256 to a scale (root: values >= 0 of which none above 0 rounds to 0)."""
    b = x.view(-1, QUANT)
    top = b.abs().amax(1, keepdim=True)
    live = top >= SMALL
    inv = torch.where(live, FP8_MAX / top, torch.zeros_like(top))
    q = b * inv
    if root:
        q = torch.where(q > 0, q.clamp(min=FP8_TINY), q)
    scale = torch.where(live, top / FP8_MAX, torch.zeros_like(top))
    return q.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def _dequantise(code, scale):
    return (code.float().view(-1, QUANT) * scale[:, None]).view(-1)


def _adamw_plain(s):
    b1, b2, lr = ADAM["beta1"], ADAM["beta2"], ADAM["lr"]
    norm = torch.sqrt(s["mat_g"].float().square().sum() + s["vec_g"].square().sum())
    clip = torch.clamp(ADAM["max_norm"] / norm, max=1.0)
    s["taken"] += 1
    s["step"] += 1
    q = s["case"]["bits"] == 8
    if q:
        m, root = _dequantise(s["mat_m"], s["mat_ms"]), _dequantise(s["mat_v"], s["mat_vs"])
        m, v = _update(s["mat_p"], s["mat_g"].float() * clip, m, root * root, 0.1, s["taken"], b1, b2, lr)
        code, scale = _quantise(m, False)
        s["mat_m"].copy_(code)
        s["mat_ms"].copy_(scale)
        code, scale = _quantise(v.sqrt(), True)
        s["mat_v"].copy_(code)
        s["mat_vs"].copy_(scale)
    else:
        m, v = _update(s["mat_p"], s["mat_g"].float() * clip, s["mat_m"], s["mat_v"], 0.1, s["taken"], b1, b2, lr)
        s["mat_m"].copy_(m)
        s["mat_v"].copy_(v)
    s["mat_b"].copy_(s["mat_p"])
    m, v = _update(s["vec_p"], s["vec_g"] * clip, s["vec_m"], s["vec_v"], 0.0, s["taken"], b1, b2, lr)
    s["vec_m"].copy_(m)
    s["vec_v"].copy_(v)
    return _adamw_outputs(s, norm)


def _update(p, g, m, v, decay, t, b1, b2, lr):
    """One step on p in place; the new m and v."""
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    step = (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + ADAM["eps"])
    p.mul_(1 - lr * decay).sub_(step * lr)
    return m, v


# ----------------------------------------------------------------------------------------------------------------
# Work and the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "ce":
        T, D, V = case["T"], case["D"], case["V"]
        inputs = 2 * T * D + 2 * V * D + 8 * T
        if case["kind"] == "score":
            return {"bytes": inputs + 8 * T, "flops": 2 * T * V * D}
        out = (4 if case["fp32"] else 2) * (T * D + V * D)
        return {"bytes": inputs + 8 * T + out, "flops": 6 * T * V * D}
    if case["op"] == "norm":
        n = case["T"] * case["D"]
        reads = 1 + case["branch"] + case["gate"]
        writes = 1 + case["branch"]
        if case["kind"] == "train":
            reads, writes = reads + 2, writes + 1 + case["branch"] + case["gate"]
        return {"bytes": 2 * n * (reads + writes), "flops": 30 * n}
    mats, vecs = _layout(case)
    a, b = sum(mats), sum(vecs)
    grad = 2 if case["grad"] == "bf16" else 4
    state = 2 * 2 * (1 + 4 / QUANT) if case["bits"] == 8 else 16
    return {"bytes": a * (grad + 8 + state + 2) + b * (4 + 8 + 16), "flops": 20 * (a + b)}


def exact(case, seed):
    if case["op"] == "ce":
        if 8 * case["T"] * case["V"] * case["D"] > 1.2e13:
            return None
        return _ce_exact(case, prepare(case, seed))
    if case["op"] == "norm":
        return _norm_exact(case, prepare(case, seed))
    return _adamw_exact(case, prepare(case, seed))


def _ce_exact(case, s):
    T, V, cap = case["T"], case["V"], case["softcap"]
    w = s["w"].double()
    n = int((s["target"] >= 0).sum())
    loss, lse = (torch.zeros(T, dtype=torch.float64, device="cuda") for _ in range(2))
    train = case["kind"] == "train"
    dh = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda") if train else None
    dw = torch.zeros(V, case["D"], dtype=torch.float64, device="cuda") if train else None
    step = max(1, (1 << 28) // V)
    for a in range(0, T, step):   # some tokens at a time
        h, t = s["h"][a:a + step].double(), s["target"][a:a + step]
        z = torch.mm(h, w.t())
        slope = None
        if cap:
            slope = 1 / torch.cosh(z / cap).square()
            z = cap * torch.tanh(z / cap)
        l = torch.logsumexp(z, dim=1)
        rows = torch.nonzero(t >= 0)[:, 0]
        lse[a:a + step] = l
        loss[a + rows] = l[rows] - z[rows, t[rows]]
        if train:
            weight = torch.zeros(len(t), dtype=torch.float64, device="cuda")
            weight[rows] = 1.0 / n if s["dloss"] is None else s["dloss"][a:a + step].double()[rows]
            d = torch.exp(z - l[:, None])
            d[rows, t[rows]] -= 1
            d *= weight[:, None]
            if cap:
                d *= slope
            dh[a:a + step] = d @ w
            dw += d.t() @ h
    out = {"loss": loss, "lse": lse, "total": torch.stack([loss.sum(), torch.tensor(float(n), device="cuda",
                                                                                   dtype=torch.float64)])}
    if train:
        out |= {"dh": dh, "dw": dw}
    return out


def _norm_exact(case, s):
    """The definition in 64 bits, the gradients by differentiating it."""
    names = ["x", "gamma_pre"] + (["y", "gamma_post", "scale"] if case["branch"] else []) + \
        (["gate"] if case["gate"] else [])
    v = {k: s[k].double().requires_grad_(True) for k in names}

    def rms(a, gamma):
        return a / torch.sqrt((a * a).mean(-1, keepdim=True) + EPS) * gamma

    r = v["x"]
    if case["branch"]:
        u = v["scale"] * rms(v["y"], v["gamma_post"])
        if case["gate"]:
            g = v["gate"]
            u = u * (g / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))))
        r = r + u
    h = rms(r, v["gamma_pre"])
    out = {"h": h.detach()} | ({"r": r.detach()} if case["branch"] else {})
    if case["kind"] == "train":
        # without a branch r is x itself, whose own cotangent dr is part of dx
        got = torch.autograd.grad([r * 1.0, h], [v[k] for k in names], [s["dr"].double(), s["dh"].double()])
        out |= {"d" + k: g for k, g in zip(names, got)}
    return out


def _adamw_exact(case, s):
    t, lr = 101, float(s["lr"])
    norm = math.sqrt(float(s["mat_g"].double().pow(2).sum() + s["vec_g"].double().pow(2).sum()))
    clip = min(1.0, ADAM["max_norm"] / norm)
    out = {"norm": torch.tensor([norm], dtype=torch.float64), "step": None, "mat_ms": None, "mat_vs": None}
    for part, decay in (("mat", 0.1), ("vec", 0.0)):
        g = s[part + "_g"].double() * clip
        m, v = s[part + "_m"].double(), s[part + "_v"].double()
        q = part == "mat" and case["bits"] == 8
        if q:
            m = (m.view(-1, QUANT) * s["mat_ms"].double()[:, None]).flatten()
            v = (v.view(-1, QUANT) * s["mat_vs"].double()[:, None]).flatten().pow(2)
        m = ADAM["beta1"] * m + (1 - ADAM["beta1"]) * g
        v = ADAM["beta2"] * v + (1 - ADAM["beta2"]) * g.pow(2)
        mh, vh = m / (1 - ADAM["beta1"] ** t), v / (1 - ADAM["beta2"] ** t)
        p = s[part + "_p"].double()
        p = p - lr * (decay * p + mh / (vh.sqrt() + ADAM["eps"]))
        out[part + "_p"] = p
        if part == "mat":
            out["mat_b"] = p
        if q:   # what the codes stand for, in units of their scales
            v = v.sqrt()
            mt, vt = (a.view(-1, QUANT).abs().amax(1) / FP8_MAX for a in (m, v))
            out["mat_ms"], out["mat_vs"] = mt, vt
            one = torch.ones_like(mt)
            out["mat_m"] = (m.view(-1, QUANT) / torch.where(mt > 0, mt, one)[:, None]).flatten()
            out["mat_v"] = (v.view(-1, QUANT) / torch.where(vt > 0, vt, one)[:, None]).flatten()
        else:
            out[part + "_m"], out[part + "_v"] = m, v
    if case["bits"] != 8:
        del out["mat_ms"], out["mat_vs"]
    return out
