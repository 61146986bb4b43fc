"""Layer norm, activation and weight gradient on tensors past 2^32 bytes: the rows behind the border give the bits of the same
rows by themselves (no row depends on another), and sums over all rows those of their parts."""

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
def test_norm_and_activation(gpu, rows, cols, pad):
    announce(f"large norm and activation {rows}x{cols} pad {pad}")
    wide = _fill(torch.empty(rows, cols + pad, dtype=BF16, device="cuda"), 1)
    x = wide[:, :cols]
    assert wide.numel() * 2 > 2 ** 32
    w = torch.randn(cols, device="cuda")
    y, mean, rstd, xc, xs = gpu.layer_norm(x, w, None, save="int8")
    codes, s = gpu.quantize_layer_norm(x, w)
    dx, dw, db = gpu.layer_norm_backward(x, xc, mean, rstd, w, x_scales=xs)
    dx2, dw2, db2 = gpu.layer_norm_backward(x, x, mean, rstd, w)
    u, uc, us = gpu.activation(x, "silu", save="int8")
    q, qs = gpu.quantize_activation(x)
    du = gpu.activation_backward(x, uc, us, "silu")
    for at in (0, rows // 2 - 5, rows - 300):
        cut = slice(at, at + 300)
        part = x[cut].contiguous()
        want = gpu.layer_norm(part, w, None, save="int8")
        assert all(torch.equal(a, b) for a, b in zip((y[cut], mean[cut], rstd[cut], xc[cut], xs[cut]), want))
        assert all(torch.equal(a, b) for a, b in zip((codes[cut], s[cut]), gpu.quantize_layer_norm(part, w)))
        assert torch.equal(dx[cut], gpu.layer_norm_backward(part, want[3], want[1], want[2], w, x_scales=want[4])[0])
        assert torch.equal(dx2[cut], gpu.layer_norm_backward(part, part, want[1], want[2], w)[0])
        want = gpu.activation(part, "silu", save="int8")
        assert all(torch.equal(a, b) for a, b in zip((u[cut], uc[cut], us[cut]), want))
        assert all(torch.equal(a, b) for a, b in zip((q[cut], qs[cut]), gpu.quantize_activation(part)))
        assert torch.equal(du[cut], gpu.activation_backward(part, want[1], want[2], "silu"))
    # sums over all rows against those of slices, in binary64: at most rows / 256 + 64 additions in binary32, whose
    # rounding errors (half a step of a partial sum below sum |d|) stay under 2^-12 of the sum of magnitudes
    ew = torch.zeros(cols, dtype=torch.float64, device="cuda")
    eb, aw, ab = torch.zeros_like(ew), torch.zeros_like(ew), torch.zeros_like(ew)
    for r in range(0, rows, 65536):
        d = x[r:r + 65536].double()
        t = d * ((d - mean[r:r + 65536, None].double()) * rstd[r:r + 65536, None].double())
        ew, eb, aw, ab = ew + t.sum(0), eb + d.sum(0), aw + t.abs().sum(0), ab + d.abs().sum(0)
    assert ((dw2.double() - ew).abs() <= 2.0 ** -12 * aw).all() and ((db2.double() - eb).abs() <= 2.0 ** -12 * ab).all()
    assert torch.equal(db, db2) and ((dw.double() - ew).abs() <= 0.05 * aw).all()


@pytest.mark.parametrize("M,N,K,pad", [(2200000, 1000, 48, 0), (560000, 4096, 256, 0), (40000, 512, 272, 60000)])
def test_grad_weight(gpu, M, N, K, pad):
    announce(f"large grad_weight_int8 {M}x{N}x{K} pad {pad}")
    dy = torch.zeros(M, N + pad, dtype=BF16, device="cuda")[:, :N]
    g = torch.Generator("cuda").manual_seed(2)
    assert dy.stride(0) * M * 2 > 2 ** 32
    # integers, so that every sum is exact: one value a row, +-1, and codes of -2 .. 2 with scale 1
    col = torch.randint(0, N, (M,), device="cuda", generator=g)
    sign = torch.randint(0, 2, (M,), device="cuda", generator=g) * 2 - 1
    dy[torch.arange(M, device="cuda"), col] = sign.bfloat16()
    codes = torch.randint(-2, 3, (M, K), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
    want = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    want.index_add_(0, col, codes.double() * sign.double()[:, None])
    assert torch.equal(gpu.grad_weight_int8(dy, codes, torch.ones(M, device="cuda")).double(), want)


def test_grad_weight_largest_output(gpu):
    """An output past 2^32 bytes from a few tokens, into rows of a wider buffer."""
    announce("large grad_weight_int8 output")
    M, N, K = 5, 65536, 20000
    g = torch.Generator("cuda").manual_seed(3)
    dy = torch.randint(-3, 4, (M, N), device="cuda", generator=g).bfloat16()
    codes = torch.randint(-3, 4, (M, K), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
    out = gpu.grad_weight_int8(dy, codes, torch.ones(M, device="cuda"))
    assert out.numel() * 4 > 2 ** 32
    for r in (0, 30000, 65536 - 64):
        assert torch.equal(out[r:r + 64].double(), dy[:, r:r + 64].double().t() @ codes.double())
