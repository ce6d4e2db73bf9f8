"""Trains a small recurrent language model on synthetic text with the library's
operators from end to end:

    tokens -> embedding
    layer:  g = h w_gate^T;  y = SAMU(x_sel = h, w = h)
            x <- x + scale GeLU(g) RMSNorm(y; gamma_post),  h = RMSNorm(x; gamma_pre)
    loss:   softmax cross entropy of h against the vocabulary matrix
    step:   AdamW over every tensor at once (matrices with 8-bit states, vectors
            with 32-bit ones), the gradients' norm clipped

The text is a random walk over a fixed table of successors, so a model that
has learnt the table predicts each token from the one before: the loss falls
from log V towards the logarithm of the number of successors.

    python examples/train_lm.py --steps 60
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_recurrence_sequence_gb300 import api  # noqa: E402

MIXER = ("nu", "theta", "w_phi", "w_r", "a_phi", "a_r")
NORM = ("gamma_post", "scale", "gamma_pre")


class Model:
    """Parameters, their gradients and the AdamW plan over them."""

    def __init__(self, V, D, layers, device, seed):
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, s):
            return (torch.randn(*shape, generator=gen) * s).to(device)

        M = D // 2
        self.V, self.D, self.device = V, D, device
        self.masters, self.params = {}, {}
        for name, shape, s in [("embed", (V, D), 1.0), ("head", (V, D), D ** -0.5)] + \
                [(f"{i}.w_gate", (D, D), D ** -0.5) for i in range(layers)]:
            self.masters[name] = normal(*shape, s=s)
            self.params[name] = self.masters[name].to(torch.bfloat16)
        one = torch.ones(D, device=device)
        self.layers = layers
        for i in range(layers):
            p = {"nu": 0.05 + normal(M, s=1.0).abs(), "theta": normal(M, s=1.0), "w_phi": normal(D + 1, s=1.0),
                 "w_r": normal(D + 1, s=1.0), "a_phi": normal(1, s=0.1), "a_r": normal(1, s=0.1),
                 "gamma_post": one.clone(), "scale": one.clone(), "gamma_pre": one.clone()}
            self.params |= {f"{i}.{k}": v for k, v in p.items()}
        self.params["gamma_in"] = one.clone()
        tensors = []
        for name, p in self.params.items():
            matrix = name in self.masters
            tensors.append({"param": p, "master": self.masters.get(name), "grad": torch.zeros_like(p).float(),
                            "weight_decay": 0.1 if matrix else 0.0, **api.adamw_state(p, 8 if matrix else 32)})
        self.plan = api.adamw_plan(tensors)
        self.step = torch.zeros(1, dtype=torch.int32, device=device)
        self.lr = torch.full((1,), 3e-3, device=device)

    def mixer(self, i):
        return [self.params[f"{i}.{k}"] for k in MIXER]

    def norm(self, i):
        return [self.params[f"{i}.{k}"] for k in NORM]

    def forward(self, tokens, target):
        """The loss and what the backward needs of each layer."""
        B, L = tokens.shape
        x = self.params["embed"][tokens]
        first = api.gated_norm_forward(x, gamma_pre=self.params["gamma_in"])
        h, kept = first["h"], []
        for i in range(self.layers):
            g = api.dense_gemm(api.LRS_GEMM_NT, h.view(B * L, self.D), self.params[f"{i}.w_gate"], B * L, self.D,
                               self.D).view(B, L, self.D)
            m = api.samu_forward(h, h, None, None, *self.mixer(i))
            n = api.gated_norm_forward(x, m["y"], g, *self.norm(i))
            kept.append((x, h, g, m["y"], m["saved"], n["saved"]))
            x, h = n["r"], n["h"]
        loss = api.linear_ce_forward(h, self.params["head"], target)
        return loss, (first, kept, h)

    def backward(self, tokens, target, loss, state):
        """Gradients of the mean loss, one per parameter."""
        first, kept, h = state
        B, L = tokens.shape
        out = api.linear_ce_backward(h, self.params["head"], target, loss["lse"], total=loss["total"])
        grads = {"head": out["dw"]}
        dh, dx = out["dh"], None
        for i in reversed(range(self.layers)):
            x, h, g, y, saved, nsaved = kept[i]
            n = api.gated_norm_backward(dx, dh, x, y, g, *self.norm(i), nsaved)
            dx = n["dx"]
            grads |= {f"{i}.{k}": n["d" + k] for k in NORM}
            m = api.samu_backward(n["dy"], None, h, h, None, None, *self.mixer(i), saved)
            grads |= {f"{i}.{k}": m["d" + k] for k in MIXER}
            dg, hh = n["dgate"].view(B * L, self.D), h.view(B * L, self.D)
            grads[f"{i}.w_gate"] = api.dense_gemm(api.LRS_GEMM_TN, dg, hh, self.D, self.D, B * L)
            through_gate = api.dense_gemm(api.LRS_GEMM_NN, dg, self.params[f"{i}.w_gate"], B * L, self.D, self.D)
            # h feeds the mixer twice (x_sel and w) and the gate
            dh = m["dx_sel"] + m["dw"] + through_gate.view(B, L, self.D)
        x0 = kept[0][0]
        n = api.gated_norm_backward(dx, dh, x0, None, None, None, None, self.params["gamma_in"], first["saved"])
        grads["gamma_in"] = n["dgamma_pre"]
        grads["embed"] = torch.zeros(self.V, self.D, device=self.device).index_add_(
            0, tokens.view(-1), n["dx"].view(-1, self.D).float())
        return grads

    def train_step(self, tokens, target):
        """One step; returns the mean loss and the gradients' norm (device tensors)."""
        loss, state = self.forward(tokens, target)
        grads = self.backward(tokens, target, loss, state)
        self.plan.set_grads([grads[k] for k in self.params])
        o = api.adamw_step(self.plan, self.step, self.lr, max_norm=1.0)
        return loss["total"][0] / loss["total"][1], o["norm"]


def text(B, L, V, successors, seed, device):
    """Token sequences of a random walk over a fixed successor table, and their next tokens (the last one's unknown)."""
    table = torch.randint(0, V, (V, successors), generator=torch.Generator().manual_seed(1))
    gen = torch.Generator().manual_seed(seed)
    walk = [torch.randint(0, V, (B,), generator=gen)]
    for _ in range(L - 1):
        walk.append(table[walk[-1], torch.randint(0, successors, (B,), generator=gen)])
    tokens = torch.stack(walk, 1)
    target = torch.full_like(tokens, -100)
    target[:, :-1] = tokens[:, 1:]
    return tokens.to(device), target.to(device)


def train(steps=60, V=1000, D=256, layers=2, B=16, L=256, successors=4, seed=0, device="cuda:0", log=print):
    """Losses of the steps (floats)."""
    device = torch.device(device)
    model = Model(V, D, layers, device, seed)
    losses = []
    for k in range(steps):
        loss, norm = model.train_step(*text(B, L, V, successors, seed * 1000 + k, device))
        losses.append(float(loss))
        if log and (k % 10 == 0 or k == steps - 1):
            log(f"step {k}: loss {losses[-1]:.3f}  gradient norm {float(norm):.3f}")
    if log:
        log(f"log V = {math.log(V):.3f}, log successors = {math.log(successors):.3f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description="Train a small recurrent language model on synthetic text.")
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--vocabulary", type=int, default=1000)
    a = ap.parse_args()
    train(a.steps, a.vocabulary, a.width, a.layers)
