"""The sums over rows of the layer norm's gradient, asked for apart from the weight: a norm with a bias alone has a gradient
of its bias, and weights that are not trained cost none."""

import numpy as np
import pytest
import torch

from oracle import training as tr
from helpers import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,C", [(1, 64), (5, 96), (33, 1040), (1100, 272), (7, 9008)])
def test_bias_without_weight(gpu, T, C, dtype):
    announce(f"layer_norm_backward sums {T}x{C} {dtype}")
    g = torch.Generator().manual_seed(T + C)
    x, dy = (torch.randn(T, C, generator=g).to(dtype).cuda() for _ in "xy")
    b = torch.randn(C, generator=g).cuda()
    y, mean, rstd, xc, xs = gpu.layer_norm(x, None, b, save="int8")
    for src, scales in ((x, None), (xc, xs)):
        dx, dw, db = gpu.layer_norm_backward(dy, src, mean, rstd, x_scales=scales, sums=True)
        # weights of 1
        ones = gpu.layer_norm_backward(dy, src, mean, rstd, torch.ones(C, device="cuda"), x_scales=scales)
        assert all(torch.equal(a, o) for a, o in zip((dx, dw, db), ones))
        plain = gpu.layer_norm_backward(dy, src, mean, rstd, x_scales=scales)
        assert torch.equal(plain[0], dx) and plain[1] is None and plain[2] is None
    # fewer than 128 additions of each column, as in test_gpu_layer_norm
    _, _, ref, _, _, size = tr.layer_norm_backward(*(t.double().cpu().numpy() for t in (dy, x, mean, rstd)))
    assert np.all(np.abs(db.double().cpu().numpy() - ref) <= 2.0 ** -17 * size)


def test_weight_without_sums(gpu):
    announce("layer_norm_backward no sums")
    x, dy, w = torch.randn(50, 528, device="cuda"), torch.randn(50, 528, device="cuda"), torch.randn(528, device="cuda")
    _, mean, rstd = gpu.layer_norm(x, w, save="x")
    full, plain = gpu.layer_norm_backward(dy, x, mean, rstd, w), gpu.layer_norm_backward(dy, x, mean, rstd, w, sums=False)
    assert torch.equal(plain[0], full[0]) and plain[1] is None and plain[2] is None
    assert all(torch.equal(a, b) for a, b in zip(full, gpu.layer_norm_backward(dy, x, mean, rstd, w, sums=True)))


def test_sums_of_no_rows(gpu):
    e = torch.zeros(0, 64, device="cuda")
    dx, dw, db = gpu.layer_norm_backward(e, e, torch.zeros(0, device="cuda"), torch.zeros(0, device="cuda"), sums=True)
    assert dx.shape == (0, 64) and dw.shape == db.shape == (64,) and not dw.any() and not db.any()


def test_bias_against_differences(gpu):
    """sum(y * dy) is linear in the bias."""
    announce("layer_norm_backward bias differences")
    x, dy, b, v = torch.randn(8, 64, device="cuda"), torch.randn(8, 64, device="cuda"), torch.randn(64, device="cuda"), torch.randn(64, device="cuda")
    _, mean, rstd = gpu.layer_norm(x, None, b, save="x")
    db = gpu.layer_norm_backward(dy, x, mean, rstd, sums=True)[2]
    f = lambda t: (gpu.layer_norm(x, None, t).double() * dy.double()).sum().item()   # noqa: E731
    # y rounded to 2^-24 of at most 8, 512 terms of |dy| below 5
    assert abs((f(b + v) - f(b - v)) / 2 - (db.double() * v.double()).sum().item()) < 512 * 8 * 5 * 2.0 ** -24
