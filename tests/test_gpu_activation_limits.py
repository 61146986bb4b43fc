"""The activation's gradient on scales of any size: the slope's limits, 0 and 1, beyond its way to them."""

import pytest
import torch

from helpers import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_slope_of_any_scale(gpu, act, dtype):
    """Beyond |v| = 110 the distance from a limit is under 111 exp(-110), less than 2^-151."""
    announce(f"activation_backward scales of any size {act} {dtype}")
    codes = torch.tensor([-128, -127, -100, -2, -1, 0, 1, 2, 3, 64, 100, 126, 127, 5, -5, 0], dtype=torch.int8, device="cuda")
    scales = torch.tensor([110.0, 127.99, 128.0, 128.01, 500.0, 1e4, 1e6, 1e8, 1e10, 1e11, 1e13, 1e19, 1e25, 1e30, 2e36], device="cuda")
    dy = torch.linspace(-3, 3, 16, device="cuda").to(dtype).repeat(len(scales), 1)
    for sign in (1.0, -1.0):
        du = gpu.activation_backward(dy, codes.repeat(len(scales), 1), scales * sign, act)
        v = codes.float() * sign
        want = dy.float() * torch.where(v > 0, 1.0, torch.where(v < 0, 0.0, 0.5))
        assert bool(((du.float() - want).abs() <= 2.0 ** -22 * dy.float().abs() + (want.abs() * 2.0 ** -8 if dtype == BF16 else 0)).all())


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_scales_that_are_not_finite(gpu, act):
    """A NaN, as a checkpoint's row with a NaN has it, or an infinity: the whole row is NaN, and no other."""
    announce(f"activation_backward scales not finite {act}")
    codes = torch.randint(-127, 128, (6, 48), device="cuda").to(torch.int8)
    codes[:, 7] = 0
    scales = torch.tensor([1e-2, float("nan"), 3e-2, float("inf"), -float("inf"), 2e-2], device="cuda")
    du = gpu.activation_backward(torch.ones(6, 48, device="cuda"), codes, scales, act)
    assert du[[1, 3, 4]].isnan().all() and du[[0, 2, 5]].isfinite().all()
    assert torch.equal(du[[0, 2, 5]], gpu.activation_backward(torch.ones(3, 48, device="cuda"), codes[[0, 2, 5]], scales[[0, 2, 5]], act))


def test_rows_of_no_columns(gpu):
    """Their scales are 0, as quantize_int8's are, and not what the memory held."""
    announce("activation no columns")
    for dtype in (BF16, F32):
        u = torch.zeros(5, 0, dtype=dtype, device="cuda")
        for run, at in ((lambda: gpu.activation(u, save="int8"), (2,)), (lambda: gpu.quantize_activation(u, save="int8"), (1, 3)),
                        (lambda: gpu.quantize_activation(u), (1,)), (lambda: gpu.quantize_int8(u), (1,))):
            held = [torch.full((5,), 7.0, device="cuda") for _ in range(8)]
            del held
            out = run()
            assert all(out[k].shape == (5,) and not out[k].any() for k in at)
        y, codes, s = gpu.activation(u, save="int8")
        assert gpu.activation_backward(y, codes, s).shape == (5, 0)
