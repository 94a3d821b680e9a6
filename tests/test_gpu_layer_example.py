"""The example's training steps: replayed bit for bit with other work between, descending, and against autograd."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "layer_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("layer_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_replay_bit_for_bit(example):
    first, losses = example.train(6)
    assert len(set(first)) == 6
    torch.randn(1000, 1000, device="cuda") @ torch.randn(1000, 1000, device="cuda")  # other work between
    again, _ = example.train(6)
    assert first == again
    assert losses[-1] < losses[0]
    other, _ = example.train(1, seed=1)
    assert other[0] != first[0]


def test_step_equals_the_plain_gradient(example):
    # One step's gradients against autograd in 64 bits; each sum here has at
    # most 256 rows times 256 columns of terms: 2^-24 * (8 + 256) of their size
    # bounds a chain of 256, far above what its random signs leave.
    layer = example.Layer(seed=3)
    w, qg, kg = (t.double().clone().requires_grad_() for t in (layer.weight, layer.q_gain, layer.k_gain))
    y = (layer.x.double() @ w).view(layer.shape)
    n = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
    z = torch.cat((n[:, :, :8] * qg, n[:, :, 8:] * kg), 2)
    c, s = layer.cos.double()[:, None], layer.sin.double()[:, None]
    a, b = z.chunk(2, -1)
    loss = 0.5 * (torch.cat((a * c - b * s, b * c + a * s), -1) - layer.targets.double()).square().sum()
    loss.backward()
    grads = torch.cat([t.grad.flatten() for t in (w, qg, kg)])
    norm = grads.norm()
    want = grads * min(1.0, 1.0 / (norm.item() + 1e-6))
    layer.step()
    assert abs(layer.norm[0].item() - norm.item()) <= 264 * 2.0 ** -24 * norm.item()
    assert (layer.grad.double() - want).norm() <= 264 * 2.0 ** -24 * want.norm()
