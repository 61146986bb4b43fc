"""Sums over many rows from codes, held as closely as those from the input, and an activation of more rows than a launch has
workgroups: each then takes rows in turn."""

import pytest
import torch

from helpers import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _fill(t, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    for r in range(0, t.shape[0], 65536):
        t[r:r + 65536] = torch.randn(min(65536, t.shape[0] - r), t.shape[1], device="cuda", generator=g)
    return t


@pytest.mark.parametrize("rows,cols,pad", [(540000, 4112, 0), (9000000, 128, 128), (150001, 1040, 13360)])
def test_sums_from_codes(gpu, rows, cols, pad):
    """At most rows / 256 + 64 additions in binary32, whose rounding errors (half a step of a partial sum below sum |d|)
    stay under 2^-12 of the sum of magnitudes."""
    announce(f"layer_norm_backward from codes {rows}x{cols} pad {pad}")
    x = _fill(torch.empty(rows, cols + pad, dtype=BF16, device="cuda"), 1)[:, :cols]
    w = torch.randn(cols, device="cuda")
    _, mean, rstd, xc, xs = gpu.layer_norm(x, w, None, save="int8")
    _, dw, db = gpu.layer_norm_backward(x, xc, mean, rstd, w, x_scales=xs)
    ew = torch.zeros(cols, dtype=torch.float64, device="cuda")
    eb, aw, ab = torch.zeros_like(ew), torch.zeros_like(ew), torch.zeros_like(ew)
    for r in range(0, rows, 65536):
        d, at = x[r:r + 65536].double(), slice(r, r + 65536)
        t = d * (((xc[at].float() * xs[at, None]).double() - mean[at, None].double()) * rstd[at, None].double())
        ew, eb, aw, ab = ew + t.sum(0), eb + d.sum(0), aw + t.abs().sum(0), ab + d.abs().sum(0)
    assert ((dw.double() - ew).abs() <= 2.0 ** -12 * aw).all() and ((db.double() - eb).abs() <= 2.0 ** -12 * ab).all()


@pytest.mark.parametrize("rows,cols", [(1100003, 2064), (1048600, 2560)])
def test_activation_of_many_rows(gpu, rows, cols):
    announce(f"activation {rows}x{cols}")
    u = _fill(torch.empty(rows, cols, dtype=BF16, device="cuda"), 3)
    y, uc, us = gpu.activation(u, "silu", save="int8")
    q, qs, uc2, us2 = gpu.quantize_activation(u, "silu", save="int8")
    assert torch.equal(uc, uc2) and torch.equal(us, us2)
    for at in (0, 2 ** 20 - 300, 2 ** 20, rows - 300):
        cut = slice(at, min(at + 300, rows))
        part = u[cut].contiguous()
        assert all(torch.equal(a, b) for a, b in zip((y[cut], uc[cut], us[cut]), gpu.activation(part, "silu", save="int8")))
        assert all(torch.equal(a, b) for a, b in zip((q[cut], qs[cut]), gpu.quantize_activation(part, "silu")))
