"""A small selective state space language model, trained and served with the
library's operators from end to end:

    tokens -> embedding (shared with the head)
    layer:  [v | z] = h w_in^T;  u = SiLU(conv(v));  s = u w_small^T, of which b and c;  delta = s w_dt^T
            y = scan(u, delta, b, c; gate z)
            x <- x + scale RMSNorm(y; gamma_post),  h = RMSNorm(x; gamma_pre)
    loss:   softmax cross entropy of h against the embedding matrix
    step:   AdamW over every tensor at once, the gradients' norm clipped

Sequences may be packed into a row (`reset` marks their starts).  Serving goes
through a prompt once and then token by token: every layer carries the last
inputs of its convolution and the state of its scan, both updated in place.

    python examples/selective_lm.py --steps 60
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from examples.train_lm import text  # noqa: E402
from linear_recurrence_sequence_gb300 import api  # noqa: E402

WIDTH_SMALL = 256   # of s: b, c and what only delta reads
TAPS = 4
MATRICES = ("w_in", "w_small", "w_dt")
CONV = ("conv_w", "conv_b")
SCAN = ("a_log", "d_skip", "delta_bias")
NORM = ("gamma_post", "scale", "gamma_pre")


class Model:
    """Parameters, their gradients and the AdamW plan over them."""

    def __init__(self, V, D, N, layers, device, seed):
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, s):
            return (torch.randn(*shape, generator=gen) * s).to(device)

        self.V, self.D, self.N, self.device, self.layers = V, D, N, device, layers
        shapes = {"w_in": (2 * D, D), "w_small": (WIDTH_SMALL, D), "w_dt": (D, WIDTH_SMALL)}
        self.masters = {"embed": normal(V, D, s=D ** -0.5)}
        self.params = {}
        one = torch.ones(D, device=device)
        for i in range(layers):
            for k, shape in shapes.items():
                self.masters[f"{i}.{k}"] = normal(*shape, s=shape[1] ** -0.5)
            # steps of 1/100 to 1/10, rates of 1 to N
            dt = torch.exp(torch.rand(D, generator=gen) * math.log(10.0) + math.log(0.01))
            p = {"conv_w": normal(TAPS, D, s=TAPS ** -0.5), "conv_b": 0 * one, "d_skip": one.clone(),
                 "delta_bias": (dt + torch.log(-torch.expm1(-dt))).to(device),
                 "a_log": torch.log(torch.arange(1.0, N + 1)).expand(D, N).contiguous().to(device),
                 "gamma_post": one.clone(), "scale": one.clone(), "gamma_pre": one.clone()}
            self.params |= {f"{i}.{k}": v for k, v in p.items()}
        self.params |= {k: v.to(torch.bfloat16) for k, v in self.masters.items()}
        self.params["gamma_in"] = one.clone()
        tensors = []
        for name, p in self.params.items():
            matrix = name in self.masters
            tensors.append({"param": p, "master": self.masters.get(name), "grad": torch.zeros_like(p).float(),
                            "weight_decay": 0.1 if matrix else 0.0, **api.adamw_state(p)})
        self.plan = api.adamw_plan(tensors)
        self.step_count = torch.zeros(1, dtype=torch.int32, device=device)
        self.lr = torch.full((1,), 3e-3, device=device)

    def of(self, i, names):
        return [self.params[f"{i}.{k}"] for k in names]

    def _nt(self, a, w):
        """a w^T over the last dimension."""
        n, k = w.shape
        return api.dense_gemm(api.LRS_GEMM_NT, a.view(-1, k), w, a.numel() // k, n, k).view(*a.shape[:-1], n)

    def _scan_inputs(self, i, u, s, delta, z):
        """The scan's arguments up to its gate."""
        a_log, d_skip, delta_bias = self.of(i, SCAN)
        return u, delta, a_log, s[..., :self.N], s[..., self.N:2 * self.N], d_skip, delta_bias, z

    # training ---------------------------------------------------------------------------------------------------
    def forward(self, tokens, target, reset=None):
        """The loss and what the backward needs of each layer."""
        D = self.D
        x = api.embedding_forward(tokens, self.params["embed"], scale=math.sqrt(D))["y"]
        first = api.gated_norm_forward(x, gamma_pre=self.params["gamma_in"])
        h, kept = first["h"], []
        for i in range(self.layers):
            w_in, w_small, w_dt = self.of(i, MATRICES)
            p = self._nt(h, w_in)
            u = api.causal_conv_forward(p[..., :D], *self.of(i, CONV), None, reset)["y"]
            s = self._nt(u, w_small)
            args = (*self._scan_inputs(i, u, s, self._nt(s, w_dt), p[..., D:]), None, reset)
            m = api.selective_scan_forward(*args)
            n = api.gated_norm_forward(x, m["y"], None, *self.of(i, NORM))
            kept.append((x, h, p, u, s, args, m, n))
            x, h = n["r"], n["h"]
        loss = api.linear_ce_forward(h, self.params["embed"], target)
        return loss, (first, kept, h)

    def backward(self, tokens, target, loss, state, reset=None):
        """Gradients of the mean loss, one per parameter."""
        first, kept, h = state
        D, N, T = self.D, self.N, tokens.numel()
        embed = self.params["embed"]
        head = api.linear_ce_backward(h, embed, target, loss["lse"], total=loss["total"], grad_fp32=True)
        grads, dh, dx = {"embed": head["dw"]}, head["dh"].to(torch.bfloat16), None
        for i in reversed(range(self.layers)):
            x, h, p, u, s, args, m, nf = kept[i]
            w_in, w_small, w_dt = self.of(i, MATRICES)
            n = api.gated_norm_backward(dx, dh, x, m["y"], None, *self.of(i, NORM), nf["saved"])
            dx = n["dx"]
            dp = torch.empty_like(p)   # of [v | z], each half written where it belongs
            g = api.selective_scan_backward(n["dy"], None, *args, m["saved"], out={"dgate": dp[..., D:]})
            ds = api.dense_gemm(api.LRS_GEMM_NN, g["ddelta"].view(T, D), w_dt, T, WIDTH_SMALL, D).view_as(s)
            ds[..., :N] += g["db"]
            ds[..., N:2 * N] += g["dc"]
            du = g["dx"] + api.dense_gemm(api.LRS_GEMM_NN, ds.view(T, -1), w_small, T, D, WIDTH_SMALL).view_as(u)
            c = api.causal_conv_backward(du, p[..., :D], *self.of(i, CONV), None, reset, out={"dx": dp[..., :D]})
            dh = api.dense_gemm(api.LRS_GEMM_NN, dp.view(T, 2 * D), w_in, T, D, 2 * D).view_as(h)
            for k, a, b in (("w_in", dp, h), ("w_small", ds, u), ("w_dt", g["ddelta"], s)):
                rows, cols = a.shape[-1], b.shape[-1]
                grads[f"{i}.{k}"] = api.dense_gemm(api.LRS_GEMM_TN, a.view(T, rows), b.view(T, cols), rows, cols, T)
            grads |= {f"{i}.{k}": n["d" + k] for k in NORM} | {f"{i}.{k}": g["d" + k] for k in SCAN}
            grads |= {f"{i}.conv_w": c["dweight"], f"{i}.conv_b": c["dbias"]}
        x0 = kept[0][0]
        n = api.gated_norm_backward(dx, dh, x0, None, None, None, None, self.params["gamma_in"], first["saved"])
        grads["gamma_in"] = n["dgamma_pre"]
        # the embedding's share joins the head's
        api.embedding_backward(n["dx"], tokens, self.V, scale=math.sqrt(D), grad_fp32=True, accumulate=True,
                               out={"dw": grads["embed"]})
        return grads

    def train_step(self, tokens, target, reset=None):
        """One step; returns the mean loss and the gradients' norm (device tensors)."""
        loss, state = self.forward(tokens, target, reset)
        grads = self.backward(tokens, target, loss, state, reset)
        self.plan.set_grads([grads[k] for k in self.params])
        o = api.adamw_step(self.plan, self.step_count, self.lr, max_norm=1.0)
        return loss["total"][0] / loss["total"][1], o["norm"]

    # serving ----------------------------------------------------------------------------------------------------
    def prompt(self, tokens, reset=None):
        """Goes through [B, L] tokens.  Returns the hidden rows [B, L, D] and the layers' states.  Shorter prompts are
        padded on the left (token -1) with a reset at their first token."""
        D = self.D
        x = api.embedding_forward(tokens, self.params["embed"], scale=math.sqrt(D))["y"]
        h, states = api.gated_norm_forward(x, gamma_pre=self.params["gamma_in"])["h"], []
        for i in range(self.layers):
            w_in, w_small, w_dt = self.of(i, MATRICES)
            p = self._nt(h, w_in)
            c = api.causal_conv_forward(p[..., :D], *self.of(i, CONV), None, reset)
            s = self._nt(c["y"], w_small)
            m = api.selective_scan_forward(*self._scan_inputs(i, c["y"], s, self._nt(s, w_dt), p[..., D:]), None, reset,
                                           keep=False)
            n = api.gated_norm_forward(x, m["y"], None, *self.of(i, NORM))
            x, h = n["r"], n["h"]
            states.append((c["state"], m["hT"]))
        return h, states

    def step(self, tokens, states, reset=None):
        """One token [B] of each sequence; the states move on in place.  Returns the hidden rows [B, D]."""
        D = self.D
        x = api.embedding_forward(tokens, self.params["embed"], scale=math.sqrt(D))["y"]
        h = api.gated_norm_forward(x, gamma_pre=self.params["gamma_in"])["h"]
        for i, (carried, state) in enumerate(states):
            w_in, w_small, w_dt = self.of(i, MATRICES)
            p = self._nt(h, w_in)
            u = api.causal_conv_step(p[:, :D], *self.of(i, CONV), carried, reset)["y"]
            s = self._nt(u, w_small)
            y = api.selective_scan_step(*self._scan_inputs(i, u, s, self._nt(s, w_dt), p[:, D:]), state, reset)["y"]
            n = api.gated_norm_forward(x, y, None, *self.of(i, NORM))
            x, h = n["r"], n["h"]
        return h


def train(steps=60, V=1000, D=256, N=16, layers=2, B=16, L=256, successors=4, seed=0, device="cuda:0", log=print):
    """The model after the steps, and their losses (floats)."""
    device = torch.device(device)
    model = Model(V, D, N, layers, device, seed)
    losses = []
    for k in range(steps):
        loss, norm = model.train_step(*text(B, L, V, successors, seed * 1000 + k, device))
        losses.append(float(loss))
        if log and (k % 10 == 0 or k == steps - 1):
            log(f"step {k}: loss {losses[-1]:.3f}  gradient norm {float(norm):.3f}")
    if log:
        log(f"log V = {math.log(V):.3f}, log successors = {math.log(successors):.3f}")
    return model, losses


def generate(model, prompt, count):
    """The most likely next tokens [B, count] after prompt [B, L]."""
    h, states = model.prompt(prompt)
    h, out = h[:, -1], []
    for _ in range(count):
        out.append((h @ model.params["embed"].t()).argmax(1))
        h = model.step(out[-1], states)
    return torch.stack(out, 1)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description="Train a small selective state space language model on synthetic text, and let it go on.")
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--states", type=int, default=16)
    ap.add_argument("--vocabulary", type=int, default=1000)
    a = ap.parse_args()
    model, _ = train(a.steps, a.vocabulary, a.width, a.states, a.layers)
    prompt, _ = text(2, 32, a.vocabulary, 4, 1, model.device)
    print("goes on:", generate(model, prompt, 12).tolist())
