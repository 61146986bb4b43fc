"""8-bit row quantization and the 8-bit product with token and channel scales (oracle; test
infrastructure only), written from the rule:

* a row's scale is s = fl32(amax / 127) and its multiplier inv = fl32(127 / amax), both
  correctly rounded; code = RNE(fl32(x * inv)).  Rows with amax below 2^-118 have s = 0 and
  codes 0; rows with an infinity or a NaN have s = NaN and codes 0.
* acc = sum of code products (exact); t = fl32(fl32(acc) * sa); v = fl32(t * sw), or
  t * sw + bias rounded once.

Products of two binary32 values are exact in float64, so each fl32() is one rounding.
"""

import numpy as np

TINY = 2.0 ** -118


def int8_scales(amax):
    """(s, inv) binary32 for an array of row maxima (NaN or inf: s = NaN, inv = 0)."""
    a = np.asarray(amax, dtype=np.float64)
    live = np.isfinite(a) & (a >= TINY)
    safe = np.where(live, a, 1.0)
    s = np.where(live, safe / 127.0, 0.0).astype(np.float32)
    inv = np.where(live, 127.0 / safe, 0.0).astype(np.float32)
    s[~np.isfinite(a)] = np.nan
    return s, inv


def quantize_int8(x):
    """(codes int8, scales float32) of the last axis of a float32 array."""
    x = np.asarray(x, dtype=np.float32).astype(np.float64)
    bad = ~np.isfinite(x).all(axis=-1)
    amax = np.abs(np.where(np.isfinite(x), x, 0.0)).max(axis=-1, initial=0.0)
    amax = np.where(bad, np.nan, amax)
    s, inv = int8_scales(amax)
    v = (np.where(bad[..., None], 0.0, x) * inv.astype(np.float64)[..., None]).astype(np.float32)
    return np.rint(v).astype(np.int8), s


def dequantize_int8(codes, scales):
    """fl32(code * scale) as float32 (round to bf16 for the library's output)."""
    return (np.asarray(codes, dtype=np.float64) * np.asarray(scales, dtype=np.float64)[..., None]).astype(np.float32)


def gemm_w8a8(a, a_scales, w, w_scales, bias=None):
    """(v, exact): the product as the rule rounds it, before the output type (float64 of binary32 values; with a
    bias the last sum is left in float64), and the unrounded float64 value of the same expression."""
    acc = np.asarray(a, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T   # below 2^53: exact
    sa, sw = np.asarray(a_scales, dtype=np.float64)[:, None], np.asarray(w_scales, dtype=np.float64)[None, :]
    t = (acc.astype(np.float32).astype(np.float64) * sa).astype(np.float32).astype(np.float64)
    exact = acc * sa * sw
    if bias is None:
        return (t * sw).astype(np.float32).astype(np.float64), exact
    b = np.asarray(bias, dtype=np.float64)[None, :]
    return t * sw + b, exact + b
