"""Root-mean-square norm of heads with the position rotation, in float64 (oracle; test
infrastructure only).

y = x / sqrt(mean(x^2) + eps) * w over the last axis; the pairs of the first R elements,
(2i, 2i+1) or (i, i + R/2), are turned by the angle whose cosine and sine the tables give
in row position[token], column i.
"""

import numpy as np


def qk_norm_rope(x, w, cos, sin, positions=None, eps=1e-6, style="interleaved"):
    """x [T, H, D] -> (y, size): the result and, for each element, |a c| + |b s| of its rotation (|y| where nothing
    turns), the magnitude that a kernel's roundings are relative to."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    if w is not None:
        y = y * np.asarray(w, dtype=np.float64)
    size = np.abs(y)
    if cos is None:
        return y, size
    T = x.shape[0]
    p = np.arange(T) if positions is None else np.asarray(positions)
    ok = (p >= 0) & (p < cos.shape[0])
    c, s = np.full((T, cos.shape[1]), np.nan), np.full((T, cos.shape[1]), np.nan)
    c[ok], s[ok] = np.asarray(cos, np.float64)[p[ok]], np.asarray(sin, np.float64)[p[ok]]
    c, s = c[:, None, :], s[:, None, :]
    R = 2 * cos.shape[1]
    first = np.arange(0, R, 2) if style == "interleaved" else np.arange(R // 2)
    second = first + (1 if style == "interleaved" else R // 2)
    a, b = y[..., first], y[..., second]
    out, size = y.copy(), size.copy()
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    size[..., first], size[..., second] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return out, size
