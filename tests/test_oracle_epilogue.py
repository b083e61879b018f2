"""Pins of oracle/linear.py's nonlinearities (CPU): against torch in fp64, slopes and the bias's gradient against central
differences, and the limits."""
import numpy as np
import pytest
import torch

from oracle import linear as ol

TORCH = {None: lambda t: t, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}


@pytest.mark.parametrize("name", ol.ACTIVATIONS)
def test_against_torch(name):
    t = np.concatenate([np.linspace(-12, 12, 2001), np.random.default_rng(0).standard_normal(500)])
    want = TORCH[name](torch.from_numpy(t)).numpy()
    assert np.abs(ol.activation(t, name) - want).max() <= 1e-13
    x = torch.from_numpy(t).requires_grad_()
    TORCH[name](x).sum().backward()
    assert np.abs(ol.activation_slope(t, name) - x.grad.numpy()).max() <= 1e-13


@pytest.mark.parametrize("name", ol.ACTIVATIONS)
def test_slope_against_differences(name):
    t = np.random.default_rng(1).standard_normal(2000) * 3
    t = t[np.abs(t) > 1e-3]
    h = 1e-5
    d = (ol.activation(t + h, name) - ol.activation(t - h, name)) / (2 * h)
    assert np.abs(d - ol.activation_slope(t, name)).max() <= 1e-8       # h^2 of the third derivative, and 1e-16 / h


@pytest.mark.parametrize("name", ol.ACTIVATIONS[1:])
def test_limits(name):
    v = ol.activation(np.array([-np.inf, np.inf, np.nan, 0.0]), name)
    assert v[0] == 0 and v[1] == np.inf and np.isnan(v[2]) and v[3] == 0


@pytest.mark.parametrize("name", ol.ACTIVATIONS)
def test_layer_gradient_against_differences(name):
    rng = np.random.default_rng(2)
    a, b, bias, r, dh = (rng.standard_normal(s) for s in ((5, 7), (6, 7), (6,), (5, 6), (5, 6)))
    t, _ = ol.linear(a, b, bias, name, r)
    dt, dbias = ol.activation_backward(dh, t, name)
    d, h = rng.standard_normal(6), 1e-6

    def loss(v):
        return (dh * ol.linear(a, b, v, name, r)[1]).sum()

    assert abs((loss(bias + h * d) - loss(bias - h * d)) / (2 * h) - dbias @ d) <= 1e-7
