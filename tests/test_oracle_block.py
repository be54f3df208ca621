"""The 64-bit norm, epilogue and experts against torch's own functions in 64 bits and against differences."""

import numpy as np
import pytest
import torch

from oracle import block

F64 = torch.float64


def test_norm_and_gradient():
    rng = np.random.default_rng(0)
    h, w, dy, dh = rng.normal(size=(5, 24)), rng.normal(size=24), rng.normal(size=(5, 24)), rng.normal(size=(5, 24))
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    want = torch.nn.functional.rms_norm(th, (24,), tw, eps=1e-3)
    v, rstd = block.rms_norm(h, w, 1e-3)
    assert np.allclose(v, want.detach().numpy(), rtol=1e-13)
    assert np.allclose(rstd, 1 / np.sqrt((h**2).sum(1) / 24 + 1e-3), rtol=1e-13)
    gx, gw = torch.autograd.grad((want * torch.tensor(dy)).sum() + (th * torch.tensor(dh)).sum(), (th, tw))
    dx, dw = block.rms_norm_bwd(dy, h, w, 1e-3, dh)
    assert np.allclose(dx, gx.numpy(), rtol=1e-12, atol=1e-13) and np.allclose(dw, gw.numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("kind", block.ACTS)
def test_activations(kind):
    z = np.linspace(-9, 9, 181) + 0.013
    t = torch.tensor(z, requires_grad=True)
    f = {"none": lambda a: a * 1, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda a: torch.nn.functional.gelu(a, approximate="tanh")}[kind](t)
    assert np.allclose(block.act(z, kind), f.detach().numpy(), rtol=1e-12, atol=1e-15)
    assert np.allclose(block.act_slope(z, kind), torch.autograd.grad(f.sum(), t)[0].numpy(), rtol=1e-11, atol=1e-13)
    d = 1e-5
    assert np.allclose(block.act_slope(z, kind), (block.act(z + d, kind) - block.act(z - d, kind)) / (2 * d), atol=1e-8)


def test_experts_by_hand():
    # one input, one inner unit: y = w * down * silu(gate x) * (up x)
    w1 = np.array([[[2.0], [3.0]], [[-1.0], [0.5]]])
    w2 = np.array([[[5.0]], [[7.0]]])
    y = block.experts([[0.5], [1.0]], np.array([[4, 5], [5, -1]]), np.array([[0.25, 0.75], [1.0, 9.0]]), w1, w2, first_expert=4)
    e = lambda x, g, u, d: d * (g * x / (1 + np.exp(-g * x))) * (u * x)  # noqa: E731
    assert np.allclose(y, [[0.25 * e(0.5, 2, 3, 5) + 0.75 * e(0.5, -1, 0.5, 7)], [e(1.0, -1, 0.5, 7)]], rtol=1e-13)
