"""Layer norm and its gradient, the feed-forward activation with its 8-bit checkpoint, and the weight
gradient of the 8-bit product, in float64 (oracle; test infrastructure only), written from the definitions.

Beside a result, ``size`` arrays give the magnitudes that a kernel's roundings are relative to.
"""

import numpy as np

from .formats import bf16_bits_to_f64, f64_to_bf16_bits
from .int8 import dequantize_int8, quantize_int8

LIMITS = {"gelu_tanh": 4.0, "silu": 8.0}


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def layer_norm(x, w=None, b=None, eps=1e-6):
    """(y, mean, rstd, size) of rows: y = (x - mean) * rstd * w + b, size = |w| (1 + |xh|)."""
    x, w, b = _f64(x), _f64(w), _f64(b)
    mean = x.mean(axis=-1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=-1) + eps)
    xh = d * rstd[:, None]
    size = 1.0 + np.abs(xh)
    if w is not None:
        xh, size = xh * w, size * np.abs(w)
    return (xh if b is None else xh + b), mean, rstd, size


def layer_norm_backward(dy, x, mean, rstd, w=None):
    """(dx, dw, db, size of dx, of dw, of db) for the statistics that the forward pass left."""
    dy, x, mean, rstd, w = (_f64(t) for t in (dy, x, mean, rstd, w))
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    gx = g * xh
    dx = rstd[:, None] * (g - g.mean(axis=-1, keepdims=True) - xh * gx.mean(axis=-1, keepdims=True))
    size = rstd[:, None] * (np.abs(g) + np.abs(g).mean(axis=-1, keepdims=True)
                            + np.abs(xh) * np.abs(gx).mean(axis=-1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0), size, np.abs(dy * xh).sum(axis=0), np.abs(dy).sum(axis=0)


def _exponent(u, act):
    """z and dz/du of f(u) = u / (1 + exp(-z))."""
    if act == "silu":
        return u, np.ones_like(u)
    k = 2.0 * np.sqrt(2.0 / np.pi)
    return k * (u + 0.044715 * u ** 3), k * (1.0 + 3 * 0.044715 * u ** 2)


def _logistic(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def activation(u, act):
    """(f(u), |z|): the rounding of z shows in exp(-z) times its size."""
    u = _f64(u)
    z, _ = _exponent(u, act)
    return u * _logistic(z), np.abs(z)


def activation_slope(u, act):
    """(f'(u), |z|, the sum of the magnitudes of its two terms)."""
    u = _f64(u)
    z, dz = _exponent(u, act)
    s, t = _logistic(z), u * _logistic(z) * _logistic(-z) * dz
    return s + t, np.abs(z), s + np.abs(t)


def activation_checkpoint(u, act):
    """(codes, scales) of float32 values clamped to +-L; a row with a NaN: scale NaN and codes 0."""
    u = np.asarray(u, dtype=np.float32)
    return quantize_int8(np.clip(u, -LIMITS[act], LIMITS[act]))   # np.clip keeps a NaN


def grad_weight_int8(dy, codes, scales):
    """(dW, sum of |products|): dy^T times the bf16 values that the codes stand for."""
    dy = _f64(dy)
    x = bf16_bits_to_f64(f64_to_bf16_bits(dequantize_int8(codes, scales).astype(np.float64)))
    return dy.T @ x, np.abs(dy).T @ np.abs(x)
