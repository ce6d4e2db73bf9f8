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
