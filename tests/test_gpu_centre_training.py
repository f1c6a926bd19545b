"""The example that runs the dense operators and the estimators together: both
of its gradients lower the loss, and a captured step goes as the eager one does."""

import importlib.util
import os

import pytest
import torch

from gpu_util import device

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "centre_training.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("centre_training", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_losses_fall(example):
    losses, es = example.main(["--steps", "120", "--width", "128", "--rows", "512", "--es-steps", "40"])
    assert losses[-1] < 0.2 * losses[0]
    assert es[-1] < es[0]


def test_gradients_of_the_whole_network(example):
    """The step's gradients against autograd in 64 bits on the same bf16 weights: within
    the bf16 roundings of the activations and gradients on the way (a few percent)."""
    d = device()
    x, target = example.data(96, 32, 10, d)
    centre = example.Centre(32, 64, 2, 10, d)
    weights = [centre.weight(i).detach().double().cpu().requires_grad_(True) for i in range(len(centre.params))]
    centre.step(x, target)
    h = x.double().cpu() @ weights[0].t() + weights[1]
    norm = torch.nn.functional.layer_norm
    for b in range(2):
        at = 2 + 6 * b
        n = norm(h, (64,), weights[at], weights[at + 1])
        a = torch.nn.functional.gelu(n @ weights[at + 2].t() + weights[at + 3])
        h = h + a @ weights[at + 4].t() + weights[at + 5]
    y = norm(h, (64,), weights[14], weights[15]) @ weights[16].t() + weights[17]
    (y - target.double().cpu()).square().mean().backward()
    for i, (g, w) in enumerate(zip(centre.grads, weights)):
        off = float((g.double().cpu() - w.grad).norm() / w.grad.norm())
        assert off < 0.03, (i, off)
