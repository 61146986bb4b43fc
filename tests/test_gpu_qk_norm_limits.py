"""The head norm where the sum of squares, a binary32 number, leaves its range: heads that overflow come out
as zeros; without eps, heads whose mean is subnormal are normed and those whose mean is 0 are not
finite.  No other head is touched."""

import pytest
import torch

from helpers import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [5, 600])
@pytest.mark.parametrize("heads", [3, 40])
@pytest.mark.parametrize("style", ["interleaved", "halves"])
def test_sums_of_squares_at_their_limits(gpu, T, heads, style):
    announce(f"qk_norm_rope limits of the sum T={T} heads={heads} {style}")
    D = 128
    g = torch.Generator("cuda").manual_seed(T + heads)
    x = torch.randn(T, heads, D, device="cuda", generator=g)
    ang = torch.rand(T, D // 2, device="cuda", generator=g) * 6
    args = (None, None, ang.cos(), ang.sin())
    ref, _ = gpu.qk_norm_rope(x, x[:, :0], *args, eps=0.0, style=style)
    signs = torch.where(torch.rand(D, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    unit, _ = gpu.qk_norm_rope(signs.expand(T, heads, D), x[:, :0], *args, eps=0.0, style=style)
    y = x.clone()
    y[0, 0] = 3e19 * signs             # 128 * 9e38: past the largest number
    y[1, 1] = 2.0 ** -70 * signs       # a mean of 2^-140: subnormal and exact
    y[2, 2] = 0.0
    y[3, 0] = 2.0 ** -76 * signs       # squares of 2^-152 round to 0
    out, _ = gpu.qk_norm_rope(y, x[:, :0], *args, eps=0.0, style=style)
    assert not out[0, 0].any()
    # the reciprocal root of a power of two and its product: two roundings, and three of the rotation
    assert bool(((out[1, 1] - unit[1, 1]).abs() <= 8 * 2.0 ** -24 * 2.0 ** 0.5).all())
    assert out[2, 2].isnan().all() and not out[3, 0].isfinite().any()
    codes, scales, _, _ = gpu.quantize_qk_norm_rope(y, x[:, :0], *args, eps=0.0, style=style)
    assert scales[0, 0] == 0 and not codes[0, 0].any()
    assert scales[2, 2].isnan() and scales[3, 0].isnan() and int(scales.isnan().sum()) == 2
    rest = torch.ones(T, heads, dtype=torch.bool, device="cuda")
    rest[0, 0] = rest[1, 1] = rest[2, 2] = rest[3, 0] = False
    assert torch.equal(out[rest], ref[rest])
