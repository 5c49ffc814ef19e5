"""The example's block: its gradients against differences, its training, and its token-by-token pass."""

import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    spec = importlib.util.spec_from_file_location("token_block", os.path.join(ROOT, "examples", "token_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("causal", [0, 1])
def test_gradients_against_differences(block, causal):
    """The derivative of sum(z * w) along a direction in every parameter and in x, at a fixed dropout seed."""
    g = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    x, p = normal(2, 37, 32), block.parameters(32)
    w = normal(2, 37, 32)
    args = dict(causal=causal, seed=9, ratio=0.2)
    z, saved = block.forward(x, p, **args)
    dx, grads = block.backward(w, saved, p, **args)
    h = 1e-2
    for name, at in list(p.items()) + [("x", x)]:
        grad = dx if name == "x" else grads[name]
        step = normal(*at.shape) * h / at.numel() ** 0.5 * at.norm().clamp_min(1.0)

        def value(sign):
            q, y = dict(p), x
            if name == "x":
                y = x + sign * step
            else:
                q[name] = at + sign * step
            return (block.forward(y, q, **args)[0].double() * w.double()).sum()

        got, want = (value(1) - value(-1)) / 2, (grad.double() * step.double()).sum()
        # third derivatives along the step, of order h^2 of its size; fp32 sums of 2368 terms of order one
        size = (grad.double() * step.double()).abs().sum()
        assert abs(got - want) <= 1e-3 * size + 2368 ** 0.5 * 2.0 ** -20, name


def test_training_lowers_the_loss(block):
    losses = block.train(steps=20)
    assert losses[-1] < 0.8 * losses[0]
    assert losses == block.train(steps=20)


def test_token_by_token_is_the_whole_sequence(block):
    x = torch.randn(3, 50, 32, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    p = block.parameters(32, seed=4)
    a, b = block.read_by_token(x, p), block.forward(x, p, causal=1)[0]
    # fp32 all through: some tens of roundings of values of order one
    assert (a - b).abs().max() <= 2.0 ** -24 * 256 * b.abs().max()
