"""Weight gradient of the 8-bit product on the GPU against the float64 oracle: within 1e-5 of the sum of
magnitudes (the bar of every product here: binary32 accumulation of exact products) plus half a step of the output."""

import numpy as np
import pytest
import torch

from oracle import training as tr
from helpers import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(M, N, K, seed, pad=0):
    g = torch.Generator("cuda").manual_seed(seed)
    dy = torch.randn(M, N + pad, device="cuda", generator=g).bfloat16()[:, :N]
    codes = torch.randint(-128, 128, (M, K + 2 * pad), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)[:, :K]
    return dy, codes, torch.rand(M, device="cuda", generator=g) * 0.05 + 1e-3


def _check(out, ref, size, extra=0.0):
    got = _np(out)
    tol = 1e-5 * size + HALF[out.dtype] * (np.abs(ref) * (1 + 2.0 ** -10) + 1e-5 * size) + extra
    assert got.shape == ref.shape and np.all(np.abs(got - ref) <= tol), np.nanmax(np.abs(got - ref) / tol)


# ragged tiles, a few tokens, windows cut short, splits of M, the large tile
SHAPES = [(1, 8, 16), (1, 520, 272), (3, 64, 48), (31, 128, 128), (33, 136, 144), (63, 8, 256), (64, 256, 16), (65, 264, 272), (127, 16, 528),
          (129, 128, 384), (500, 72, 80), (1001, 2056, 1360), (2049, 136, 112), (4099, 64, 64), (10000, 24, 32), (700, 2816, 2832),
          (192, 3016, 3008), (20000, 512, 256)]


@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matches_oracle(gpu, M, N, K, pad):
    announce(f"grad_weight_int8 {M}x{N}x{K} pad {pad}")
    dy, codes, s = _inputs(M, N, K, M + N + K, pad)
    ref, size = tr.grad_weight_int8(_np(dy), codes.cpu().numpy(), s.cpu().numpy())
    out = gpu.grad_weight_int8(dy, codes, s)
    assert out.dtype == F32 and out.is_contiguous()
    _check(out, ref, size)
    assert torch.equal(out, gpu.grad_weight_int8(dy, codes, s))
    half = gpu.grad_weight_int8(dy, codes, s, out_dtype=BF16)
    assert torch.equal(half, out.bfloat16())      # the same sum, rounded once
    # into a wider buffer, and added to what it holds; nothing else is written
    for dtype in (F32, BF16):
        for off in (0, 1):
            wide = torch.randn(N + 2, K + 8, device="cuda").to(dtype)
            view, before = wide[1:N + 1, off:K + off], wide.clone()
            assert gpu.grad_weight_int8(dy, codes, s, out=view, accumulate=True) is view
            have = _np(before[1:N + 1, off:K + off])
            # one more rounding, of the sum
            _check(view, ref + have, size, 2.0 ** -23 * (np.abs(have) + np.abs(ref)))
            gpu.grad_weight_int8(dy, codes, s, out=view)
            assert torch.equal(view, out.to(dtype))
            view.copy_(before[1:N + 1, off:K + off])
            assert torch.equal(wide, before)


def test_is_the_product_of_the_dequantized_codes(gpu):
    """Small integers: every sum exact, equal to the product of dequantize_int8's values."""
    announce("grad_weight_int8 integers")
    g = torch.Generator("cuda").manual_seed(2)
    for M, N, K in ((300, 272, 304), (5000, 40, 48)):
        dy = torch.randint(-8, 9, (M, N), device="cuda", generator=g).bfloat16()
        codes = torch.randint(-7, 8, (M, K), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
        s = torch.full((M,), 0.5, device="cuda")
        want = dy.double().t() @ gpu.dequantize_int8(codes, s).double()
        assert torch.equal(gpu.grad_weight_int8(dy, codes, s).double(), want)


def test_against_differences(gpu):
    """The loss sum(dy * (x W^T)) of the forward product in 8 bits is linear in the weights: its change along a
    direction of integers is the gradient's product with it."""
    announce("grad_weight_int8 differences")
    g = torch.Generator("cuda").manual_seed(3)
    M, N, K = 96, 40, 64
    dy = torch.randint(-4, 5, (M, N), device="cuda", generator=g).bfloat16()
    codes, s = gpu.quantize_int8(torch.randn(M, K, device="cuda", generator=g))
    s = torch.exp2(torch.round(torch.log2(s)))     # code * scale is then exact in bf16
    w = torch.randint(-60, 60, (N, K), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
    v = torch.randint(-2, 3, (N, K), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
    one = torch.ones(N, device="cuda")
    loss = lambda m: (gpu.gemm_w8a8(codes, s, m, one, out_dtype=F32).double() * dy.double()).sum()   # noqa: E731
    dw = gpu.grad_weight_int8(dy, codes, s).double()
    diff, want = (loss(w + v) - loss(w - v)) / 2, (dw * v.double()).sum()
    # both sides: sums of exact products; the loss's outputs have one rounding each
    assert abs(diff - want).item() <= 1e-5 * (dw.abs() * v.double().abs()).sum().item() + 1e-3


def test_bad_tokens(gpu):
    """A token whose scale is NaN spreads over its columns' gradients only where dy meets it: everywhere; a NaN in dy
    stays in its row of the gradient."""
    announce("grad_weight_int8 bad tokens")
    dy, codes, s = _inputs(100, 72, 80, 5)
    clean = gpu.grad_weight_int8(dy, codes, s)
    dy[7, 9] = float("nan")
    out = gpu.grad_weight_int8(dy, codes, s)
    rows = torch.arange(72, device="cuda") != 9
    assert out[9].isnan().all() and torch.equal(out[rows], clean[rows])
    dy[7, 9], s[3] = 0.0, float("nan")
    assert gpu.grad_weight_int8(dy, codes, s).isnan().all()


def test_rows_past_the_end_are_not_read(gpu):
    """Views of larger buffers whose other rows and columns hold NaN."""
    announce("grad_weight_int8 NaN around the views")
    M, N, K = 70, 136, 144
    dy, codes, s = _inputs(M, N, K, 6)
    wide = torch.full((M + 64, N + 128), float("nan"), device="cuda", dtype=BF16)
    wide[:M, :N] = dy
    scales = torch.full((M + 64,), float("nan"), device="cuda")
    scales[:M] = s
    assert torch.equal(gpu.grad_weight_int8(wide[:M, :N], codes, scales[:M]), gpu.grad_weight_int8(dy, codes, s))


def test_empty(gpu):
    e = lambda *s: torch.zeros(s, device="cuda")   # noqa: E731
    out = gpu.grad_weight_int8(e(0, 24).bfloat16(), e(0, 32).to(torch.int8), e(0))
    assert out.shape == (24, 32) and not out.any()
    have = torch.ones(24, 32, device="cuda")
    assert gpu.grad_weight_int8(e(0, 24).bfloat16(), e(0, 32).to(torch.int8), e(0), out=have, accumulate=True).eq(1).all()
    assert gpu.grad_weight_int8(e(5, 0).bfloat16(), e(5, 32).to(torch.int8), e(5)).shape == (0, 32)


@pytest.mark.parametrize("M,N,K", [(2300, 136, 400), (9001, 264, 144), (30001, 136, 16), (24000, 1288, 272), (70000, 8, 48)])
def test_many_parts_of_few_tiles(gpu, M, N, K):
    """Sums cut into more than 16 parts of M, which several threads of the joining kernel share."""
    announce(f"grad_weight_int8 parts {M}x{N}x{K}")
    assert gpu.lib.mxq_grad_weight_int8_workspace_bytes(M, N, K) > 16 * 128 * 128 * 4
    dy, codes, s = _inputs(M, N, K, M + K, 8)
    ref, size = tr.grad_weight_int8(_np(dy), codes.cpu().numpy(), s.cpu().numpy())
    out = gpu.grad_weight_int8(dy, codes, s)
    _check(out, ref, size)
    assert torch.equal(out, gpu.grad_weight_int8(dy, codes, s))
    assert torch.equal(gpu.grad_weight_int8(dy, codes, s, out_dtype=BF16), out.bfloat16())
    have = torch.randn(N, K + 8, device="cuda")
    wide = have.clone()
    gpu.grad_weight_int8(dy, codes, s, out=wide[:, 1:K + 1], accumulate=True)
    _check(wide[:, 1:K + 1], ref + _np(have[:, 1:K + 1]), size, 2.0 ** -23 * (np.abs(_np(have[:, 1:K + 1])) + np.abs(ref)))
    assert torch.equal(wide[:, 0], have[:, 0]) and torch.equal(wide[:, K + 1:], have[:, K + 1:])
