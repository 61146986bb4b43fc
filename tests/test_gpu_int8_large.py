"""The 8-bit operators on tensors whose offsets pass 32 bits: a block of rows repeated many
times gives the block's results, repeated."""

import pytest
import torch

from helpers import announce

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _repeat(block, times):
    return block.expand(times, *block.shape).reshape(times * block.shape[0], *block.shape[1:])


def _repeats(out, block):
    return bool((out.view(-1, *block.shape) == block).all())


def test_quantizer_and_dequantizer(gpu):
    announce("quantize_int8 / dequantize_int8, 2.9e9 elements")
    block = torch.randn(1000, 7232, device="cuda").to(BF16)
    x = _repeat(block, 400)
    assert x.numel() > 2 ** 31 and x.numel() * 2 > 2 ** 32
    q, s = gpu.quantize_int8(x)
    rq, rs = gpu.quantize_int8(block)
    assert _repeats(q, rq) and _repeats(s, rs)
    del x
    assert _repeats(gpu.dequantize_int8(q, s), gpu.dequantize_int8(rq, rs))


@pytest.mark.parametrize("heads", [(40, 40), (0, 80)])
def test_head_norm(gpu, heads):
    announce(f"qk_norm_rope, 3e9 elements, heads {heads}")
    T, n, D = 1000, 300, 128
    block = torch.randn(T, 80 * D, device="cuda").to(BF16)
    ang = torch.rand(T, D // 2, device="cuda") * 6
    args = (torch.rand(D, device="cuda"), torch.rand(D, device="cuda"), ang.cos(), ang.sin())

    def views(t):
        h = t.view(-1, 80, D)
        return h[:, :heads[0]], h[:, heads[0]:]

    x = _repeat(block, n)
    assert x.numel() > 2 ** 31
    pos = torch.arange(T * n, device="cuda") % T
    for style in ("interleaved", "halves"):
        for fn in (gpu.qk_norm_rope, gpu.quantize_qk_norm_rope):
            for o, r in zip(fn(*views(x), *args, positions=pos, style=style), fn(*views(block), *args, style=style)):
                if r.numel():
                    assert _repeats(o, r)


@pytest.mark.parametrize("M,N,K,times,dtype", [(700, 16011, 64, 100, F32), (700, 16384, 96, 200, BF16), (2, 40000, 16, 4, BF16)])
def test_product(gpu, M, N, K, times, dtype):
    announce(f"gemm_w8a8 {M * times}x{N}x{K} {dtype}")
    a = torch.randint(-128, 128, (M, K), device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), device="cuda", dtype=torch.int8)
    sa, sw, b = torch.rand(M, device="cuda"), torch.rand(N, device="cuda"), torch.randn(N, device="cuda")
    ref = gpu.gemm_w8a8(a, sa, w, sw, bias=b, out_dtype=dtype)
    assert _repeats(gpu.gemm_w8a8(_repeat(a, times), _repeat(sa, times), w, sw, bias=b, out_dtype=dtype), ref)


@pytest.mark.parametrize("M,N", [(5, 700), (40, 70), (300, 300), (1300, 1100)])
def test_product_with_the_largest_row_pitch(gpu, M, N):
    """Rows 2^23 - 16 bytes apart: the last ones of a tile start close to 2^31 bytes from its first."""
    announce(f"gemm_w8a8 {M}x{N}, rows 8 MB apart")
    K, pitch = 208, 2 ** 23 - 16
    rows = max(M, N)
    buf = torch.empty(rows * pitch, dtype=torch.int8, device="cuda")
    a, w = buf.as_strided((M, K), (pitch, 1), 0), buf.as_strided((N, K), (pitch, 1), 4096)
    a.copy_(torch.randint(-128, 128, (M, K), device="cuda", dtype=torch.int8))
    w.copy_(torch.randint(-128, 128, (N, K), device="cuda", dtype=torch.int8))
    sa, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    for dtype in (BF16, F32):
        assert torch.equal(gpu.gemm_w8a8(a, sa, w, sw, out_dtype=dtype),
                           gpu.gemm_w8a8(a.contiguous(), sa, w.contiguous(), sw, out_dtype=dtype))
