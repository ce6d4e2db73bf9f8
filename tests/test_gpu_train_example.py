"""The operators together as a training program uses them: the example's model
learns its synthetic text, and its gradients agree with differences of the loss."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_loss_falls():
    import train_lm
    losses = train_lm.train(steps=60, log=None)
    assert abs(losses[0] - math.log(1000)) < 2.0        # random weights: near the uniform loss
    assert min(losses[-5:]) < 0.6 * losses[0]
    assert all(math.isfinite(x) for x in losses)


def test_step_follows_its_gradient():
    """A small step against the gradient of one batch lowers the mean loss by |gradient|^2 times its length, within
    the second order of the step and BF16 activations."""
    import train_lm
    dev = torch.device("cuda:0")
    model = train_lm.Model(300, 256, 1, dev, 3)
    tokens, target = train_lm.text(4, 64, 300, 4, 5, dev)
    loss, state = model.forward(tokens, target)
    grads = model.backward(tokens, target, loss, state)
    assert set(grads) == set(model.params)
    head = grads["head"].float()
    eta = 1e-2 / float(head.norm())
    mean = float(loss["total"][0] / loss["total"][1])
    expect = float(head.square().sum()) * eta
    model.params["head"].copy_((model.masters["head"] - eta * head).to(torch.bfloat16))
    after, _ = model.forward(tokens, target)
    fall = mean - float(after["total"][0] / after["total"][1])
    # the head's BF16 rounding moves each weight by up to 2^-9 of it; the linear term dominates
    assert 0.3 * expect < fall < 3.0 * expect, (fall, expect)


class _Bf16(torch.autograd.Function):
    """Rounds a value on the way forward and its gradient on the way back."""

    @staticmethod
    def forward(ctx, x):
        return x.to(torch.bfloat16).double()

    @staticmethod
    def backward(ctx, g):
        return g.to(torch.bfloat16).double()


def _norm(x, gamma):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma


def _gelu(g):
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


def _samu(x_sel, w, p):
    M = w.shape[-1] // 2
    x = torch.cat([x_sel, torch.ones_like(x_sel[..., :1])], -1)
    d = torch.tanh(p["a_phi"]) / math.sqrt(M) * torch.tanh(x @ (p["w_phi"] / p["w_phi"].norm()))
    r = torch.tanh(x @ (p["w_r"] / p["w_r"].norm()))
    rate = torch.exp(torch.tanh(p["a_r"]) / math.sqrt(M) * r / (1 + r * r))
    size, angle = torch.exp(-p["nu"] * rate[..., None]), p["theta"] + d[..., None]
    turn = torch.complex(size * torch.cos(angle), size * torch.sin(angle))
    b = torch.complex(w[..., :M], w[..., M:])
    z, out = torch.zeros_like(b[:, 0]), []
    for t in range(b.shape[1]):
        z = turn[:, t] * z + b[:, t]
        out.append(z)
    out = torch.stack(out, 1)
    return torch.cat([out.real, out.imag], -1)


def _loss64(params, layers, tokens, target, bf16=False, without=None):
    """The model's mean loss in 64 bits (bf16: its activations and their gradients rounded as the model keeps them);
    `without`: the use of a layer's input that is left out of the gradients."""
    kept = _Bf16.apply if bf16 else lambda a: a

    def use(a, name):
        return a.detach() if name == without else a

    x = params["embed"][tokens]
    h = kept(_norm(x, params["gamma_in"]))
    for i in range(layers):
        p = {k.split(".")[1]: v for k, v in params.items() if k.startswith(f"{i}.")}
        g = kept(use(h, "gate") @ p["w_gate"].T)
        y = kept(_samu(use(h, "x_sel"), use(h, "w"), p))
        r = use(x, "x") + p["scale"] * _gelu(g) * _norm(y, p["gamma_post"])
        x, h = kept(r), kept(_norm(r, p["gamma_pre"]))
    z = h @ params["head"].T
    counted = target >= 0
    return (torch.logsumexp(z, -1) - z.gather(-1, target.clamp(min=0)[..., None])[..., 0])[counted].mean()


def _gradients64(model, tokens, target, **kw):
    params = {k: v.detach().cpu().double().requires_grad_(True) for k, v in model.params.items()}
    loss = _loss64(params, model.layers, tokens.cpu(), target.cpu(), **kw)
    return float(loss.detach()), dict(zip(params, torch.autograd.grad(loss, list(params.values()))))


def test_every_gradient_against_the_model_in_64_bits():
    """Relative L2 errors of every parameter's gradient.  A path through the two layers meets about 24 roundings to
    BF16 (activations and gradients), each 2^-8 / sqrt(12) of the value: 2^-7.5 together where they are independent,
    so 2^-6 bounds a tensor's error, and 2^-4 that of the controllers' (w_phi, w_r, a_phi, a_r: sums over all tokens
    and modes that cancel).  The 64-bit model with those roundings stays within half of it, and leaving out any use of a layer's input moves
    embed's gradient by at least twice as much."""
    import train_lm
    dev = torch.device("cuda:0")
    model = train_lm.Model(300, 256, 2, dev, 3)
    for k, v in model.params.items():   # controllers that matter
        if k.endswith(("a_phi", "a_r")):
            v.fill_(3.0)
    tokens, target = train_lm.text(4, 64, 300, 4, 5, dev)
    exact, want = _gradients64(model, tokens, target)
    _, rounded = _gradients64(model, tokens, target, bf16=True)

    def off(a, k):
        return float((a.double().cpu() - want[k]).norm() / want[k].norm())

    def most(k):
        return 2.0 ** -4 if k.endswith(("w_phi", "w_r", "a_phi", "a_r")) else 2.0 ** -6

    assert all(off(rounded[k], k) <= most(k) / 2 for k in want)
    for name in ("gate", "x_sel", "w", "x"):
        _, missing = _gradients64(model, tokens, target, without=name)
        assert off(missing["embed"], "embed") >= 2 * most("embed"), name
    loss, state = model.forward(tokens, target)
    assert abs(float(loss["total"][0] / loss["total"][1]) - exact) <= 2.0 ** -9 * exact
    got = model.backward(tokens, target, loss, state)
    assert set(got) == set(want)
    for k in want:
        assert off(got[k], k) <= most(k), (k, off(got[k], k))
