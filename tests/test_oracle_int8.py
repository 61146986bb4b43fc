"""Pins for the oracle's 8-bit rule, product and head norm (CPU only), against exact
rational arithmetic, integer sums and invariants."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle


def _nearest32(exact):
    """The binary32 nearest to a rational, ties to even, by comparing neighbours."""
    c = np.float32(float(exact))
    cand = [np.nextafter(c, np.float32(-np.inf)), c, np.nextafter(c, np.float32(np.inf))]
    return min(cand, key=lambda v: (abs(Fraction(float(v)) - exact), int(np.float32(v).view(np.uint32)) & 1))


def test_scales_are_correctly_rounded_quotients():
    rng = np.random.default_rng(0)
    for amax in np.concatenate([rng.lognormal(0, 20, 200), [127.0, 1.0, 2.0 ** -118, 3e38]]).astype(np.float32):
        if float(amax) < 2.0 ** -118:
            continue
        s, inv = oracle.int8.int8_scales(np.array([amax]))
        assert s[0] == _nearest32(Fraction(float(amax)) / 127) and inv[0] == _nearest32(127 / Fraction(float(amax)))


def test_codes_are_the_nearest_integers_of_the_rounded_product():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((16, 64)) * np.exp(rng.standard_normal((16, 1)) * 4)).astype(np.float32)
    q, s = oracle.quantize_int8(x)
    for r in range(16):
        amax = float(np.abs(x[r]).max())
        inv = Fraction(float(_nearest32(127 / Fraction(amax))))
        for k in range(64):
            assert q[r, k] == round(Fraction(float(_nearest32(Fraction(float(x[r, k])) * inv))))   # round(): ties to even
    assert np.abs(q.astype(int)).max(axis=1).min() == 127
    # half a step of the exact quotient, plus the two roundings of x * inv (127 * 2^-23)
    assert np.all(np.abs(q.astype(np.float64) - x.astype(np.float64) / (np.abs(x).max(1, keepdims=True).astype(np.float64) / 127))
                  <= 0.5 + 127 * 2.0 ** -23)


def test_degenerate_rows():
    x = np.zeros((5, 16), np.float32)
    x[1, 3] = np.inf
    x[2, 3] = np.nan
    x[3, 3] = np.nextafter(np.float32(2.0 ** -118), np.float32(0))
    x[4, 3] = -2.0 ** -118
    q, s = oracle.quantize_int8(x)
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] == 0 and s[4] > 0
    assert not q[:4].any() and q[4, 3] == -127


def test_product_is_exact_and_scaled_once_per_factor():
    rng = np.random.default_rng(2)
    a, w = rng.integers(-128, 128, (5, 96)), rng.integers(-128, 128, (7, 96))
    sa, sw = rng.random(5, np.float32), rng.random(7, np.float32)
    v, exact = oracle.gemm_w8a8(a, sa, w, sw)
    for m in range(5):
        for n in range(7):
            acc = sum(int(x) * int(y) for x, y in zip(a[m], w[n]))
            t = _nearest32(Fraction(float(np.float32(acc))) * Fraction(float(sa[m])))
            assert v[m, n] == _nearest32(Fraction(float(t)) * Fraction(float(sw[n])))
            assert abs(exact[m, n] - float(acc * Fraction(float(sa[m])) * Fraction(float(sw[n])))) <= 1e-15 * abs(exact[m, n])


@pytest.mark.parametrize("style", ["interleaved", "halves"])
@pytest.mark.parametrize("R", [8, 24])
def test_head_norm_keeps_lengths_and_turns_by_the_angle(style, R):
    rng = np.random.default_rng(3)
    T, H, D = 4, 3, 24
    x = rng.standard_normal((T, H, D))
    ang = rng.random((9, R // 2)) * 6
    pos = np.array([8, 0, 3, 3])
    y, _ = oracle.qk_norm_rope(x, None, np.cos(ang), np.sin(ang), pos, eps=0.0, style=style)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-12)
    # the turn of every pair as one complex product
    n = x / np.sqrt((x * x).mean(-1, keepdims=True))
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if style == "interleaved" else (i, i + R // 2)
        z = (n[..., a] + 1j * n[..., b]) * np.exp(1j * ang[pos, i])[:, None]
        np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(y[..., R:], n[..., R:])


def test_head_norm_matches_torch_rms_norm():
    x = torch.randn(3, 2, 40, dtype=torch.float64, generator=torch.Generator().manual_seed(4))
    w = torch.rand(40, dtype=torch.float64, generator=torch.Generator().manual_seed(5))
    y, _ = oracle.qk_norm_rope(x.numpy(), w.numpy(), None, None, eps=1e-3)
    np.testing.assert_allclose(y, torch.nn.functional.rms_norm(x, (40,), w, 1e-3).numpy(), rtol=1e-12)
