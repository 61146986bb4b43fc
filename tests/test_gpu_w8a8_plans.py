"""Every kernel of the 8-bit product (tile, split of K, cut last round, shifted form) against exact sums,
every output of it: the sums in float64 are exact integers, and the two scale products round once
each as the rule says, so that binary32 outputs without a bias are equal, bf16 ones too, and those with
a bias are within the roundings of one fused multiply-add and of the output type."""

import pytest
import torch

from helpers import announce
from w8a8_shapes import AT_LARGEST_PITCH, LARGEST_PITCH, PLANS

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _codes(rows, cols, g):
    return torch.randint(-128, 128, (rows, cols), device="cuda", generator=g, dtype=torch.int8)


def _operands(M, N, K):
    g = torch.Generator("cuda").manual_seed(M + 3 * N + 5 * K)
    return (_codes(M, K, g), torch.rand(M, device="cuda", generator=g) * 0.1 + 1e-3, _codes(N, K, g),
            torch.rand(N, device="cuda", generator=g) * 0.01 + 1e-4, torch.randn(N, device="cuda", generator=g))


def _check(gpu, a, sa, w, sw, b):
    acc = a.double() @ w.double().t().contiguous()           # |sums| < 2^31: exact
    t = acc.float() * sa[:, None]
    v = t * sw[None, :]
    vb = t.double() * sw.double()[None, :] + b.double()      # the product is exact, the sum rounded to 53 bits
    del acc, t
    for dtype in (F32, BF16):
        assert torch.equal(gpu.gemm_w8a8(a, sa, w, sw, out_dtype=dtype), v.to(dtype))
        got = gpu.gemm_w8a8(a, sa, w, sw, bias=b, out_dtype=dtype).double()
        # one rounding to binary32, for bf16 a second one of half a step (2^-8) of that value
        half = 2.0 ** -24 if dtype == F32 else 2.0 ** -24 + 2.0 ** -8 * (1 + 2.0 ** -24)
        assert bool(((got - vb).abs() <= half * vb.abs() * (1 + 2.0 ** -50) + 2.0 ** -134).all())


@pytest.mark.parametrize("M,N,K,tile,parts,tail,off", PLANS)
def test_every_kernel(gpu, M, N, K, tile, parts, tail, off):
    announce(f"gemm_w8a8 {M}x{N}x{K}: {tile} in {parts} parts, last round {tail}, off the lines {off}")
    _check(gpu, *_operands(M, N, K))


@pytest.mark.parametrize("M,N,K,tile,parts,tail,off", AT_LARGEST_PITCH)
def test_largest_tiles_with_the_largest_row_pitch(gpu, M, N, K, tile, parts, tail, off):
    """Both operands as rows 8 MB apart of one buffer of 30 GB."""
    announce(f"gemm_w8a8 {M}x{N}x{K}: {tile}, rows {LARGEST_PITCH} bytes apart")
    a, sa, w, sw, b = _operands(M, N, K)
    buf = torch.empty(max(M, N) * LARGEST_PITCH, dtype=torch.int8, device="cuda")
    av, wv = buf.as_strided((M, K), (LARGEST_PITCH, 1), 0), buf.as_strided((N, K), (LARGEST_PITCH, 1), 4096)
    av.copy_(a)
    wv.copy_(w)
    for dtype in (F32, BF16):
        assert torch.equal(gpu.gemm_w8a8(av, sa, wv, sw, bias=b, out_dtype=dtype), gpu.gemm_w8a8(a, sa, w, sw, bias=b, out_dtype=dtype))
    _check(gpu, av, sa, wv, sw, b)
