"""The selective scan, the causal convolution, the embedding and the operators around them as one model
(examples/selective_lm.py): its gradients against the model in 64 bits, its prompt and its steps against its forward.

The model's 64-bit form is evaluated with the activations rounded to BF16 where the operators store them, so what is left
is the FP32 arithmetic and the roundings that it tips over.  A tipped rounding moves a value by one step of BF16 (2^-8
of it at most): with one in ten tipped on each of the 8 stores of a layer, a vector's relative error is
sqrt(8 layers' stores / 10) 2^-8, about 2^-8 for two layers; backward the same again.  Bound: 2^-5 of a gradient's norm,
and 2^-6 of the hidden rows'."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


class _Round(torch.autograd.Function):
    """BF16 storage: rounded forward and backward."""

    @staticmethod
    def forward(ctx, x):
        return x.to(BF).double()

    @staticmethod
    def backward(ctx, g):
        return g.to(BF).double()


def _model(V=97, D=256, N=16, layers=2, seed=3):
    from examples import selective_lm
    return selective_lm.Model(V, D, N, layers, DEV, seed)


def _definition(model, tokens, target, reset):
    """The loss of the model in 64 bits from leaves of its parameters; returns (mean loss, hidden rows, leaves)."""
    r = _Round.apply
    leaf = {k: v.double().requires_grad_(True) for k, v in model.params.items()}
    D, N = model.D, model.N
    B, L = tokens.shape

    def rms(a, g):
        return a / torch.sqrt((a * a).mean(-1, keepdim=True) + 1e-6) * g

    seq = torch.zeros_like(tokens) if reset is None else (reset != 0).long().cumsum(1)
    at = tokens.clamp(min=0)
    x = r(torch.where((tokens >= 0)[..., None], leaf["embed"][at] * math.sqrt(D), 0.0))
    h = r(rms(x, leaf["gamma_in"]))
    for i in range(model.layers):
        p = {k: leaf[f"{i}.{k}"] for k in ("w_in", "w_small", "w_dt", "conv_w", "conv_b", "a_log", "d_skip", "delta_bias",
                                           "gamma_post", "scale", "gamma_pre")}
        vz = r(h @ p["w_in"].t())
        v, z = vz[..., :D], vz[..., D:]
        pre = p["conv_b"].expand(B, L, D)
        for j in range(4):
            lag = torch.cat([torch.zeros(B, min(j, L), D, dtype=torch.float64, device=DEV), v[:, :max(0, L - j)]], 1)
            was = torch.cat([torch.full((B, min(j, L)), -1, device=DEV), seq[:, :max(0, L - j)]], 1)
            pre = pre + torch.where((was == seq)[..., None], p["conv_w"][j] * lag, 0.0)
        u = r(torch.nn.functional.silu(pre))
        s = r(u @ p["w_small"].t())
        delta = r(s @ p["w_dt"].t())
        dt = torch.nn.functional.softplus(delta + p["delta_bias"], threshold=700)
        rate = -torch.exp(p["a_log"])
        state, ys = torch.zeros(B, D, N, dtype=torch.float64, device=DEV), []
        for t in range(L):
            if reset is not None:
                state = torch.where((reset[:, t] != 0)[:, None, None], 0.0, state)
            state = torch.exp(dt[:, t, :, None] * rate) * state + (dt[:, t] * u[:, t])[..., None] * s[:, t, None, :N]
            ys.append((state * s[:, t, None, N:2 * N]).sum(2))
        y = r((torch.stack(ys, 1) + p["d_skip"] * u) * torch.nn.functional.silu(z))
        full = x + p["scale"] * rms(y, p["gamma_post"])
        x, h = r(full), r(rms(full, p["gamma_pre"]))
    logits = h @ leaf["embed"].t()
    counted = target >= 0
    losses = torch.logsumexp(logits, -1) - logits.gather(-1, target.clamp(min=0)[..., None])[..., 0]
    return (losses * counted).sum() / counted.sum(), h, leaf


def _batch(B, L, V, seed, packed):
    gen = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, V, (B, L), generator=gen).to(DEV)
    target = torch.randint(0, V, (B, L), generator=gen).to(DEV)
    target[:, -1] = -100
    reset = None
    if packed:
        reset = (torch.rand(B, L, generator=gen) < 0.05).to(torch.uint8).to(DEV)
        tokens[0, :3] = -1
    return tokens, target, reset


@pytest.mark.parametrize("packed", [False, True])
def test_every_gradient(packed):
    model = _model()
    tokens, target, reset = _batch(3, 70, model.V, 5, packed)
    loss, state = model.forward(tokens, target, reset)
    grads = model.backward(tokens, target, loss, state, reset)
    assert sorted(grads) == sorted(model.params)
    want, _, leaf = _definition(model, tokens, target, reset)
    ref = torch.autograd.grad(want, [leaf[k] for k in model.params])
    mean = float(want.detach())
    assert abs(float(loss["total"][0] / loss["total"][1]) - mean) <= 2.0 ** -6 * mean
    for k, g in zip(model.params, ref):
        off = float((grads[k].double() - g).norm() / g.norm())
        assert off <= 2.0 ** -5, (k, off)


def test_prompt_and_steps_are_the_forward():
    """Prompts of different lengths, padded on the left, then token by token."""
    model = _model(seed=4)
    B, L, more = 3, 40, 12
    tokens, _, _ = _batch(B, L + more, model.V, 6, False)
    lengths = (40, 33, 1)
    padded = torch.full((B, L), -1, device=DEV)
    reset = torch.zeros(B, L, dtype=torch.uint8, device=DEV)
    for b, n in enumerate(lengths):
        padded[b, L - n:] = tokens[b, :n]
        reset[b, L - n] = 1
    h, states = model.prompt(padded, reset)
    rows = [[h[b, L - n + k] for k in range(n)] for b, n in enumerate(lengths)]
    for k in range(more):
        nxt = torch.stack([tokens[b, n + k] for b, n in enumerate(lengths)])
        o = model.step(nxt, states)
        for b in range(B):
            rows[b].append(o[b])
    for b, n in enumerate(lengths):
        seq = tokens[b:b + 1, :n + more]
        _, want, _ = _definition(model, seq, seq, None)
        got = torch.stack(rows[b]).double()
        off = (got - want[0]).norm(dim=-1) / want[0].norm(dim=-1)
        assert float(off.max()) <= 2.0 ** -6, (b, float(off.max()))


def test_a_step_of_training_captured():
    """The whole training step as a graph does what the eager one does."""
    eager, model = _model(seed=8), _model(seed=8)
    tokens, target, reset = _batch(2, 64, model.V, 9, True)
    model.train_step(tokens, target, reset)   # buffers and launch attributes
    eager.train_step(tokens, target, reset)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, norm = model.train_step(tokens, target, reset)
    for seed in (10, 11):
        t, y, r = _batch(2, 64, model.V, seed, True)
        tokens.copy_(t)
        target.copy_(y)
        reset.copy_(r)
        graph.replay()
        want, wnorm = eager.train_step(t, y, r)
        assert float(loss) == float(want) and float(norm) == float(wnorm)
    for k in model.params:
        assert torch.equal(model.params[k], eager.params[k]), k


def test_the_example_runs():
    from examples import selective_lm
    model, losses = selective_lm.train(steps=3, V=101, D=256, layers=1, B=2, L=48, log=None)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
    out = selective_lm.generate(model, torch.randint(0, 101, (2, 9), device=DEV), 4)
    assert out.shape == (2, 4) and int(out.min()) >= 0 and int(out.max()) < 101
