"""Pins of oracle/activation.py that need no GPU: against torch's own functions in float64, and the
slopes against central differences."""
import numpy as np
import pytest
import torch

import oracle

Z = np.concatenate([np.linspace(-40, 40, 4001), [0.0, -0.0, 1e-30, -1e-30]])


@pytest.mark.parametrize("kind", ["none", "relu2", "gelu", "silu"])
def test_values_and_slopes(kind):
    z = torch.tensor(Z, requires_grad=True)
    f = {"none": lambda x: x, "relu2": lambda x: torch.relu(x) ** 2, "silu": torch.nn.functional.silu,
         "gelu": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}[kind](z)
    f.sum().backward()
    assert np.allclose(oracle.act64(Z, kind), f.detach().numpy(), rtol=1e-12, atol=1e-15)
    assert np.allclose(oracle.act_slope64(Z, kind), z.grad.numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("kind", ["none", "relu2", "gelu", "silu"])
def test_slopes_against_differences(kind):
    z, h = np.linspace(-12, 12, 2001) + 1e-3, 1e-5
    diff = (oracle.act64(z + h, kind) - oracle.act64(z - h, kind)) / (2 * h)
    # second-order term h^2 / 6 * |act'''| (< 10) and cancellation, eps |act| / h
    tol = 10 * h * h + 2.0 ** -50 * np.abs(oracle.act64(z, kind)) / h + 1e-11
    near = np.abs(z) < 2 * h if kind == "relu2" else np.zeros(z.shape, bool)
    assert np.all((np.abs(diff - oracle.act_slope64(z, kind)) <= tol) | near)
