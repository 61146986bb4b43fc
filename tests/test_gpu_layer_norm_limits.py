"""Layer norm where its statistics could lose digits: rows of equal values, and means far from zero, at every width."""

import pytest
import torch

from oracle import training as tr
from helpers import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# rows that share a wave, a wave a row, 4 and 8 waves; counts that binary32 divides exactly and others
WIDTHS = [8, 24, 40, 64, 72, 120, 200, 248, 256, 264, 504, 776, 1016, 1360, 1536, 1544, 2040, 3000, 4104, 5120, 6136, 6152, 8192, 9000, 13824, 16376, 16384]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_values_are_the_bias(gpu, dtype, C):
    """Deviations of 0 from a mean that is the value itself, whatever the rounding of 1 / C: b, to the last bit."""
    announce(f"layer_norm equal values {C} {dtype}")
    g = torch.Generator("cuda").manual_seed(C)
    size = torch.exp(3 * torch.randn(400, 1, device="cuda", generator=g))
    x = (torch.randn(400, 1, device="cuda", generator=g) * size).to(dtype).expand(400, C).contiguous()
    w, b = torch.randn(C, device="cuda", generator=g), torch.randn(C, device="cuda", generator=g)
    y, mean, rstd = gpu.layer_norm(x, w, b, eps=1e-6, save="x")
    assert torch.equal(mean, x[:, 0].float()) and bool(((rstd - 1e3).abs() <= 1e3 * 2.0 ** -22).all())
    assert torch.equal(y, b.to(dtype).expand_as(y))
    if C % 16:
        return
    codes, s = gpu.quantize_layer_norm(x, w, b, eps=1e-6)
    want, ws = gpu.quantize_int8(b[None])
    assert torch.equal(codes, want.expand_as(codes)) and torch.equal(s, ws.expand_as(s))


@pytest.mark.parametrize("C", WIDTHS)
def test_means_far_from_zero(gpu, C):
    """Deviations of a few last digits of the mean: they are exact in binary32, so that y is as near as anywhere
    (the bounds of test_gpu_layer_norm)."""
    announce(f"layer_norm far means {C}")
    g = torch.Generator().manual_seed(C)
    far = torch.exp(4 * torch.rand(64, 1, generator=g)) * 100
    x = (far + torch.randn(64, C, generator=g) * far * 2.0 ** -18).cuda()
    ref, m, r, size = tr.layer_norm(x.double().cpu().numpy(), None, None, 1e-12)
    y, mean, rstd = gpu.layer_norm(x, eps=1e-12, save="x")
    assert bool((abs(y.double().cpu().numpy() - ref) <= 2.0 ** -18 * size + 2.0 ** -24 * abs(ref)).all())
    assert bool((abs(rstd.double().cpu().numpy() - r) <= 2.0 ** -18 * r).all())
    assert bool((abs(mean.double().cpu().numpy() - m) <= 2.0 ** -23 * abs(m) + 2.0 ** -18 / r).all())


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_equal_values_are_the_bias(gpu, dtype, C):
    """Also where the sum of the row, or the square of a last digit of its values, is past binary32."""
    announce(f"layer_norm large equal values {C} {dtype}")
    top = torch.finfo(dtype).max
    values = [top, -top, top * (1 - 2.0 ** -7), 2.0 ** 127, -(2.0 ** 120), 1e37, 3e30, -7e27, 1e26, 2.0 ** 118, 3.0, -1e-30]
    x = torch.tensor(values).to(dtype).cuda()[:, None].repeat(12, C)
    w, b = torch.randn(C, device="cuda"), torch.randn(C, device="cuda")
    y, mean, rstd = gpu.layer_norm(x, w, b, eps=1e-6, save="x")
    assert torch.equal(mean, x[:, 0].float()) and bool(((rstd - 1e3).abs() <= 1e3 * 2.0 ** -22).all())
    assert torch.equal(y, b.to(dtype).expand_as(y))
    if C % 16:
        return
    codes, s = gpu.quantize_layer_norm(x, w, b, eps=1e-6)
    want, ws = gpu.quantize_int8(b[None])
    assert torch.equal(codes, want.expand_as(codes)) and torch.equal(s, ws.expand_as(s))


@pytest.mark.parametrize("C", [64, 240, 248, 1360, 5120, 16384])
def test_rows_beside_large_ones(gpu, C):
    """Large equal values, an infinity and deviations without squares in binary32 among ordinary rows, whose bits stay."""
    announce(f"layer_norm beside large rows {C}")
    x = torch.randn(101, C, device="cuda")
    clean = gpu.layer_norm(x, save="x")
    x[::10], x[5::20], x[7::20, C // 2] = 3e38, torch.randn(C, device="cuda") * 1e30, float("inf")
    got = gpu.layer_norm(x, save="x")
    plain = torch.ones(101, dtype=torch.bool, device="cuda")
    plain[::10] = plain[5::20] = plain[7::20] = False
    assert all(torch.equal(a[plain], b[plain]) for a, b in zip(got, clean))
    assert not got[0][::10].any() and bool((got[1][::10] == x[0, 0]).all()) and got[0][7::20].isnan().all()
    y = x.clone()
    assert torch.equal(gpu.layer_norm(y, out=y).nan_to_num(1e9), got[0].nan_to_num(1e9))
    if C % 16:
        return
    codes, s = gpu.quantize_layer_norm(x)
    assert s[5::20].isnan().all() and s[7::20].isnan().all() and not s[::10].any() and s[plain].isfinite().all()


@pytest.mark.parametrize("C", WIDTHS)
def test_range_of_the_deviations(gpu, C):
    """Without eps a power of two comes out of y exactly, from deviations of 2^-60 up to where the sum of their squares
    nears 2^128: the bits of deviations around 1."""
    announce(f"layer_norm range of deviations {C}")
    g = torch.Generator("cuda").manual_seed(C)
    x = torch.randn(65, C, device="cuda", generator=g).clamp(-4, 4)
    # at least 2^-5 off the mean on the whole, at most 4: sums of squares below 2^4 C
    y, mean, rstd = gpu.layer_norm(x, eps=0.0, save="x")
    top = int(62 - torch.tensor(float(C)).log2().ceil().item() / 2)
    for e in (-55, -30, 30, top - 4, top - 3):
        y2, mean2, rstd2 = gpu.layer_norm(x * 2.0 ** e, eps=0.0, save="x")
        assert torch.equal(y2, y) and torch.equal(mean2, mean * 2.0 ** e) and torch.equal(rstd2, rstd * 2.0 ** -e), e


@pytest.mark.parametrize("C", [64, 248, 1360, 5120, 16384])
def test_outside_the_range(gpu, C):
    """Squares that overflow, or vanish without eps: y is b, infinite or NaN, and the quantized form's scale NaN."""
    announce(f"layer_norm outside the range {C}")
    x = torch.randn(3, C, device="cuda")
    x[0] *= 2.0 ** 70
    x[1] *= 2.0 ** -85
    y = gpu.layer_norm(x, eps=0.0)
    assert not (y[0].isfinite() & (y[0] != 0)).any() and not (y[1].isfinite() & (y[1] != 0)).any() and y[2].isfinite().all()
    if C % 16:
        return
    codes, s = gpu.quantize_layer_norm(x, eps=0.0)
    assert s[:2].isnan().all() and not codes[:2].any() and s[2].isfinite()
