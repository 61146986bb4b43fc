"""The oracle's layer norm, activations and gradients against closed forms, torch's binary64 autograd
and central differences (CPU only)."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import training as tr


def _rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 17), (5, 64)])
def test_layer_norm_and_gradient_against_autograd(rows, cols, affine):
    g = _rng(rows + cols)
    x, dy = g.standard_normal((rows, cols)) * 3 + 1, g.standard_normal((rows, cols))
    w, b = (g.standard_normal(cols), g.standard_normal(cols)) if affine else (None, None)
    t = lambda a: None if a is None else torch.tensor(a, requires_grad=True)   # noqa: E731
    tx, tw, tb = t(x), t(w), t(b)
    y = torch.nn.functional.layer_norm(tx, (cols,), tw, tb, 1e-5)
    y.backward(torch.tensor(dy))
    got, mean, rstd, _ = tr.layer_norm(x, w, b, 1e-5)
    assert np.allclose(got, y.detach().numpy(), rtol=0, atol=1e-12)
    dx, dw, db, *_ = tr.layer_norm_backward(dy, x, mean, rstd, w)
    assert np.allclose(dx, tx.grad.numpy(), rtol=0, atol=1e-11)
    if affine:
        assert np.allclose(dw, tw.grad.numpy(), atol=1e-11) and np.allclose(db, tb.grad.numpy(), atol=1e-11)


def test_layer_norm_gradient_against_differences():
    g = _rng(1)
    x, dy, w, v = (g.standard_normal((4, 24)) for _ in range(4))
    w = w[0]
    _, mean, rstd, _ = tr.layer_norm(x, w)
    dx, dw, *_ = tr.layer_norm_backward(dy, x, mean, rstd, w)
    h = 1e-5
    up, down = (tr.layer_norm(x + s * h * v, w)[0] for s in (1, -1))
    assert abs(((up - down) * dy).sum() / (2 * h) - (dx * v).sum()) < 1e-8
    up, down = (tr.layer_norm(x, w + s * h * v[0])[0] for s in (1, -1))
    assert abs(((up - down) * dy).sum() / (2 * h) - (dw * v[0]).sum()) < 1e-8


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_activation_and_slope(act):
    u = np.linspace(-30, 30, 4001)
    t = torch.tensor(u, requires_grad=True)
    y = torch.nn.functional.gelu(t, approximate="tanh") if act == "gelu_tanh" else torch.nn.functional.silu(t)
    y.sum().backward()
    assert np.allclose(tr.activation(u, act)[0], y.detach().numpy(), rtol=1e-12, atol=1e-14)
    slope = tr.activation_slope(u, act)[0]
    assert np.allclose(slope, t.grad.numpy(), rtol=0, atol=1e-12)
    h = 1e-5
    diff = (tr.activation(u + h, act)[0] - tr.activation(u - h, act)[0]) / (2 * h)
    assert np.abs(diff - slope).max() < 1e-8
    # the checkpoint saturates where the slope is within the stated distance of its limits
    far = np.abs(u) >= tr.LIMITS[act]
    assert np.abs(slope - (u > 0))[far].max() < (4e-4 if act == "gelu_tanh" else 3e-3)


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_checkpoint_steps(act):
    """Half a step of at most L / 127 off inside the limits, whatever the outliers; saturated outside."""
    L = tr.LIMITS[act]
    u = (_rng(3).standard_normal((6, 64)) * 2).astype(np.float32)
    u[1, 5], u[2, 7], u[3, 9], u[4] = 1000.0, -np.inf, np.nan, 0.25
    codes, s = tr.activation_checkpoint(u, act)
    assert math.isnan(s[3]) and not codes[3].any()
    v = codes.astype(np.float64) * s[:, None]
    for r in (0, 1, 2, 4, 5):
        assert s[r] <= np.float32(L / 127) and np.abs(v[r] - np.clip(u[r], -L, L)).max() <= 0.5001 * s[r]
    assert codes[1, 5] == 127 and codes[2, 7] == -127 and s[4] == np.float32(0.25 / 127)


def test_grad_weight_small():
    dy = np.array([[1.0, 2.0], [-1.0, 0.5], [0.0, 4.0]])
    codes = np.array([[127, -3], [5, 0], [-128, 64]], dtype=np.int8)
    scales = np.array([0.5, 2.0, 0.25], dtype=np.float32)    # code * scale is exact in bf16
    dw, size = oracle.training.grad_weight_int8(dy, codes, scales)
    x = codes * scales[:, None].astype(np.float64)
    want = [[sum(dy[m, n] * x[m, k] for m in range(3)) for k in range(2)] for n in range(2)]
    assert dw.tolist() == want and (size >= np.abs(dw)).all()


def test_grad_weight_rounds_the_values_to_bf16():
    dw, _ = tr.grad_weight_int8([[1.0]], np.array([[127]], dtype=np.int8), np.array([0.1], dtype=np.float32))
    assert dw[0, 0] == 12.6875 and abs(dw[0, 0] - 12.7) <= 12.7 * 2.0 ** -8
