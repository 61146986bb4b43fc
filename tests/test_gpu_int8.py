"""The 8-bit operators on the GPU against the oracle: the row quantizer and its
dequantization bit for bit, the product against exact sums (each output within its roundings)."""

import numpy as np
import pytest
import torch

import oracle
from helpers import announce, bf16_bits_to_f32, to_np_bf16_bits

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _x(rows, cols, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))
    return x.to(dtype)


def _np(t):
    return t.detach().float().cpu().numpy()


def _codes(rows, cols, seed, lo=-128):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, 128, (rows, cols), generator=g, dtype=torch.int8)


def _wide(t, pad, fill):
    """t as a view of a buffer `pad` columns wider whose other bytes hold `fill`."""
    w = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    w[:, :t.shape[1]] = t.cuda()
    return w[:, :t.shape[1]], w


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (5, 512), (4, 528), (7, 1024), (2, 1040), (9, 2048), (3, 2064),
                                       (2, 5120), (3, 8192), (2, 8208), (3, 13824), (2, 16384), (2, 16400), (2, 65536),
                                       (2, 65552), (1, 131056), (1030, 64)])
def test_quantize_is_bit_exact(gpu, rows, cols, dtype):
    announce(f"quantize_int8 {rows}x{cols} {dtype}")
    x = _x(rows, cols, dtype, rows * 7 + cols, 3.0)
    q, s = gpu.quantize_int8(x.cuda())
    rq, rs = oracle.quantize_int8(_np(x))
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)


def test_quantize_strided_in_and_out_leaves_the_rest(gpu):
    announce("quantize_int8 strided")
    for dtype in (BF16, F32):
        x = _x(33, 336, dtype, 5)
        xv, _ = _wide(x, 16, 1e30)
        cv, cw = _wide(torch.zeros(33, 336, dtype=torch.int8), 48, 77)
        sw = torch.full((40,), -5.0, device="cuda")
        gpu.quantize_int8(xv, codes=cv, scales=sw[3:36])
        rq, rs = oracle.quantize_int8(_np(x))
        np.testing.assert_array_equal(cv.cpu().numpy(), rq)
        np.testing.assert_array_equal(sw[3:36].cpu().numpy(), rs)
        assert (cw[:, 336:] == 77).all() and (sw[:3] == -5).all() and (sw[36:] == -5).all()


@pytest.mark.parametrize("cols", [16, 1040, 13824, 65552])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_degenerate_rows(gpu, cols, dtype):
    announce(f"quantize_int8 degenerate rows {cols} {dtype}")
    x = _x(12, cols, dtype, 11)
    x[0] = 0
    x[1, cols - 1] = float("inf")
    x[2, 0] = float("-inf")
    x[3, cols // 2] = float("nan")
    x[4] = 0
    x[4, 5] = 2.0 ** -118
    x[5] = 0
    x[5, 5] = 2.0 ** -119
    x[6] = torch.finfo(dtype).max
    x[7] = -0.0
    x[8, :] = 1.0
    x[9] = torch.finfo(dtype).tiny
    x[10] *= 2.0 ** 100
    q, s = gpu.quantize_int8(x.cuda())
    rq, rs = oracle.quantize_int8(_np(x))
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)


def test_quantize_every_tie_and_neighbour(gpu):
    """Values on and next to the border between two codes, for several maxima."""
    announce("quantize_int8 ties")
    rows = []
    for amax in (127.0, 254.0, 1.0, 0.7, 3.3e-5, 6.02e23):
        s = np.float32(np.float64(np.float32(amax)) / 127.0)
        k = (np.arange(-127, 127) + 0.5) * np.float64(s)
        v = k.astype(np.float32)
        v = np.concatenate([v, np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(-np.inf))])
        v = v[np.abs(v) <= np.float32(amax)]
        row = np.zeros(784, np.float32)
        row[:v.size] = v
        row[-1] = amax
        rows.append(row)
    x = np.stack(rows)
    q, s = gpu.quantize_int8(torch.from_numpy(x).cuda())
    rq, rs = oracle.quantize_int8(x)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)


def test_quantize_every_finite_bf16(gpu):
    announce("quantize_int8 every finite bf16")
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    vals = bf16_bits_to_f32(bits)
    vals = np.sort(vals[np.isfinite(vals)])
    vals = vals[: vals.size // 64 * 64].reshape(-1, 64).copy()
    x = torch.from_numpy(vals).to(BF16)
    q, s = gpu.quantize_int8(x.cuda())
    rq, rs = oracle.quantize_int8(vals)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("rows,cols,pad", [(1, 8, 0), (3, 128, 0), (77, 96, 8), (129, 1360, 16), (5, 13824, 0)])
def test_dequantize_is_bit_exact(gpu, rows, cols, pad):
    announce(f"dequantize_int8 {rows}x{cols}")
    q = _codes(rows, cols, 3)
    s = torch.exp(4 * torch.randn(rows, generator=torch.Generator().manual_seed(4)))
    s[0] = 0.0
    qv, _ = _wide(q, pad, 99)
    out = torch.full((rows, cols + pad), -3.0, dtype=BF16, device="cuda")
    gpu.dequantize_int8(qv, s.cuda(), out=out[:, :cols])
    ref = torch.from_numpy(oracle.dequantize_int8(q.numpy(), s.numpy())).to(BF16)
    np.testing.assert_array_equal(to_np_bf16_bits(out[:, :cols]), to_np_bf16_bits(ref))
    assert (out[:, cols:] == -3).all()
    assert torch.equal(gpu.dequantize_int8(q.cuda(), s.cuda()).cpu(), ref)


# ------------------------------------------------------------------ product
def _check(out, v, biased):
    """Within the output type's half step of the rule's value.  Without a bias the binary32
    value is the rule's own; with one the oracle leaves the last sum in float64, which the
    kernel rounds to binary32 once (2^-24) before the output type."""
    got = out.double().cpu().numpy()
    if out.dtype == F32:
        if not biased:
            np.testing.assert_array_equal(got, v)
        else:
            assert np.all(np.abs(got - v) <= 2.0 ** -24 * np.abs(v) + 2.0 ** -149)
    else:
        tol = 2.0 ** -8 * np.abs(v) * (1 + 2.0 ** -15) + 2.0 ** -24 * np.abs(v) + 2.0 ** -134
        assert np.all(np.abs(got - v) <= tol)
        if not biased:
            ref = torch.from_numpy(v.astype(np.float32)).to(BF16)
            np.testing.assert_array_equal(to_np_bf16_bits(out), to_np_bf16_bits(ref))


def _operands(M, N, K, seed):
    a, w = _codes(M, K, seed), _codes(N, K, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    sa, sw = torch.rand(M, generator=g) * 0.1 + 1e-3, torch.rand(N, generator=g) * 0.01 + 1e-4
    return a, sa, w, sw, torch.randn(N, generator=g)


SHAPES = [(1, 1, 16), (1, 5120, 1360), (2, 3, 131056), (1, 17, 4096), (3, 16, 64), (8, 100, 144), (15, 33, 128),
          (16, 256, 2048), (17, 255, 272), (31, 64, 112), (32, 48, 4112), (33, 1000, 240), (48, 640, 1024), (63, 129, 80),
          (64, 512, 13824), (65, 257, 384), (100, 320, 96), (127, 130, 528), (128, 128, 256), (129, 1, 1040),
          (200, 640, 640), (255, 300, 48), (256, 256, 512), (257, 511, 1360), (300, 2051, 160), (513, 769, 2064),
          (1001, 2051, 1360), (2048, 96, 320), (1, 13824, 5120), (5, 40000, 32),
          # every tile, and splits of K with a ragged last part
          (9, 5120, 96), (30, 13824, 160), (48, 5120, 13824), (60, 515, 13808), (60, 7000, 304), (130, 5120, 1040), (250, 13824, 272),
          (256, 5120, 8192), (500, 5120, 400), (500, 770, 16000), (700, 13824, 144), (1300, 5120, 272), (2100, 5000, 160),
          (64, 256, 131056),
          # a last round of the largest tile cut into halves and quarters, ragged at both edges
          (4100, 4500, 48), (3900, 4700, 1040), (4400, 5000, 400), (4099, 4501, 160),
          # a short K: the largest tile, and the one with two workgroups on a CU, with every output alignment
          (3600, 3584, 128), (2100, 2048, 512), (2100, 2056, 400), (2100, 2052, 64), (2100, 2050, 272), (1500, 1504, 240), (1500, 1502, 240),
          (3000, 3000, 208)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_contiguous(gpu, M, N, K):
    announce(f"gemm_w8a8 {M}x{N}x{K}")
    a, sa, w, sw, b = _operands(M, N, K, M + N + K)
    dev = [t.cuda() for t in (a, sa, w, sw)]
    v, _ = oracle.gemm_w8a8(a.numpy(), sa.numpy(), w.numpy(), sw.numpy())
    vb, _ = oracle.gemm_w8a8(a.numpy(), sa.numpy(), w.numpy(), sw.numpy(), b.numpy())
    for dt in (F32, BF16):
        _check(gpu.gemm_w8a8(*dev, out_dtype=dt), v, False)
        _check(gpu.gemm_w8a8(*dev, bias=b.cuda(), out_dtype=dt), vb, True)


@pytest.mark.parametrize("M,N,K,pa,pw,po", [(1, 200, 160, 16, 32, 0), (9, 64, 1360, 32, 16, 8), (40, 77, 208, 48, 0, 3),
                                            (70, 300, 16, 16, 16, 4), (130, 260, 400, 112, 96, 1), (300, 512, 144, 16, 48, 8),
                                            (520, 256, 1072, 64, 16, 16)])
def test_product_strided_and_padded(gpu, M, N, K, pa, pw, po):
    """Rows inside wider buffers whose other bytes are not zeros; strided and shared scales."""
    announce(f"gemm_w8a8 strided {M}x{N}x{K}")
    a, sa, w, sw, b = _operands(M, N, K, 3 * M + N + K)
    av, _ = _wide(a, pa, 91)
    wv, _ = _wide(w, pw, -107)
    sa2 = torch.full((M, 3), 7.0, device="cuda")
    sa2[:, 1] = sa.cuda()
    for dt in (F32, BF16):
        out = torch.full((M + 2, N + po), -3.0, dtype=dt, device="cuda")
        gpu.gemm_w8a8(av, sa2[:, 1], wv, sw.cuda(), bias=b.cuda(), out=out[1:-1, :N])
        v, _ = oracle.gemm_w8a8(a.numpy(), sa.numpy(), w.numpy(), sw.numpy(), b.numpy())
        _check(out[1:-1, :N], v, True)
        assert (out[0] == -3).all() and (out[-1] == -3).all() and (out[:, N:] == -3).all()
        # one scale for all tokens, one for all channels
        one = gpu.gemm_w8a8(av, sa[:1].cuda().expand(M), wv, sw[:1].cuda().expand(N), out_dtype=dt)
        v1, _ = oracle.gemm_w8a8(a.numpy(), sa[:1].repeat(M).numpy(), w.numpy(), sw[:1].repeat(N).numpy())
        _check(one, v1, False)


@pytest.mark.parametrize("at_a,pad_a,at_w,pad_w", [(0, 0, 0, 0), (16, 0, 112, 0), (0, -1, 48, 16), (96, 32, 0, -1), (80, -1, 64, -1)])
@pytest.mark.parametrize("M,N,K", [(5, 100, 1168), (20, 300, 2064), (60, 515, 4112), (130, 700, 1296), (300, 2000, 1360), (700, 2000, 1552),
                                   (1001, 2051, 1360), (1100, 4100, 2064), (4100, 4500, 1072), (2048, 5000, 1056)])
def test_product_rows_off_the_cache_lines(gpu, M, N, K, at_a, pad_a, at_w, pad_w):
    """Operands from byte at_* of a cache line, rows K + pad_* bytes apart (-1: to the next line); the
    bytes around them are not zeros."""
    announce(f"gemm_w8a8 {M}x{N}x{K} from {at_a} +{pad_a} and {at_w} +{pad_w}")
    a, sa, w, sw, b = _operands(M, N, K, M + 2 * N + K)

    def place(t, at, pad):
        pitch = (K + 127) // 128 * 128 if pad < 0 else K + pad
        buf = torch.full((256 + t.shape[0] * pitch,), 85, dtype=torch.int8, device="cuda")
        start = -buf.data_ptr() % 128 + at
        v = buf.as_strided(t.shape, (pitch, 1), start)
        v.copy_(t)
        assert v.data_ptr() % 128 == at
        return v

    av, wv = place(a, at_a, pad_a), place(w, at_w, pad_w)
    v, _ = oracle.gemm_w8a8(a.numpy(), sa.numpy(), w.numpy(), sw.numpy(), b.numpy())
    for dt in (F32, BF16):
        _check(gpu.gemm_w8a8(av, sa.cuda(), wv, sw.cuda(), bias=b.cuda(), out_dtype=dt), v, True)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_product_largest_sums(gpu, M):
    """Every product at its largest: the sum reaches 2^31 - 2^18 and -(2^31 - ...)."""
    announce(f"gemm_w8a8 largest sums M={M}")
    K = 131056
    a = torch.full((M, K), -128, dtype=torch.int8)
    w = torch.full((5, K), -128, dtype=torch.int8)
    w[1] = 127
    w[2, ::2] = 127
    one_m, one_n = torch.ones(M), torch.ones(5)
    v, _ = oracle.gemm_w8a8(a.numpy(), one_m.numpy(), w.numpy(), one_n.numpy())
    assert v.max() == 128 * 128 * K and v.max() < 2 ** 31
    _check(gpu.gemm_w8a8(a.cuda(), one_m.cuda(), w.cuda(), one_n.cuda(), out_dtype=F32), v, False)


def test_product_degenerate_sizes(gpu):
    announce("gemm_w8a8 degenerate sizes")
    for M, N, K in ((0, 8, 32), (8, 0, 32), (0, 0, 0)):
        a, sa, w, sw, b = (t.cuda() for t in _operands(M, N, K, 1))
        assert gpu.gemm_w8a8(a, sa, w, sw, bias=b).shape == (M, N)
        assert gpu.gemm_w8a8_fused(torch.zeros(M, K, device="cuda"), w, sw).shape == (M, N)
    for M in (1, 40, 300):
        a, sa, w, sw, b = (t.cuda() for t in _operands(M, 70, 0, 1))
        for dt in (F32, BF16):
            assert not gpu.gemm_w8a8(a, sa, w, sw, out_dtype=dt).any()
            assert torch.equal(gpu.gemm_w8a8(a, sa, w, sw, bias=b, out_dtype=dt), b.to(dt).expand(M, 70))
            x = torch.zeros(M, 0, device="cuda")
            assert torch.equal(gpu.gemm_w8a8_fused(x, w, sw, bias=b, out_dtype=dt), b.to(dt).expand(M, 70))
    torch.cuda.synchronize()
    q, s = gpu.quantize_int8(torch.zeros(3, 0, device="cuda"))
    assert q.shape == (3, 0) and not s.any()
    q, s = gpu.quantize_int8(torch.zeros(0, 32, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0,)
    assert gpu.dequantize_int8(q, s).shape == (0, 32)


def test_product_scales_that_are_nan_or_zero_stay_in_their_row(gpu):
    announce("gemm_w8a8 NaN scales")
    a, sa, w, sw, b = _operands(70, 40, 256, 9)
    sa[3], sa[5], sw[7] = float("nan"), 0.0, float("nan")
    for M in (6, 70):
        out = gpu.gemm_w8a8(a[:M].cuda(), sa[:M].cuda(), w.cuda(), sw.cuda(), bias=b.cuda(), out_dtype=F32).cpu()
        nan = torch.zeros(M, 40, dtype=torch.bool)
        nan[3], nan[:, 7] = True, True
        assert torch.equal(out.isnan(), nan)
        keep = torch.arange(40) != 7
        assert torch.equal(out[5][keep], b[keep])


# ------------------------------------------------------------------ fused
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 64, 16), (1, 5120, 13824), (1, 13825, 5120), (2, 40, 1360), (3, 300, 2048),
                                   (4, 1000, 8192), (5, 129, 2064), (8, 77, 4112), (16, 512, 1024), (17, 96, 528),
                                   (64, 256, 640), (100, 333, 1040), (300, 512, 784), (2, 33, 65552), (1, 9, 131056),
                                   # the largest and the next K of the one-launch form, for 1, 2, 3 and 8 tokens
                                   (1, 100, 15744), (1, 100, 15760), (2, 64, 7808), (2, 64, 7824), (3, 31, 5248), (3, 31, 5264), (8, 70, 1920),
                                   (8, 70, 1936), (7, 50, 112), (6, 1000, 16), (8, 33, 144)])
def test_fused_equals_the_two_calls(gpu, M, N, K, dtype):
    announce(f"gemm_w8a8_fused {M}x{N}x{K} {dtype}")
    x = _x(M, K, dtype, M + N + K, 2.0)
    if M > 2:
        x[1] = 0
        x[2, 3] = float("inf")
    xv, _ = _wide(x, 16, 1e30)
    _, _, w, sw, b = _operands(1, N, K, 5)
    w, sw, b = w.cuda(), sw.cuda(), b.cuda()
    for dt in (BF16, F32):
        for bias in (None, b):
            two = gpu.gemm_w8a8(*gpu.quantize_int8(xv), w, sw, bias=bias, out_dtype=dt)
            one = gpu.gemm_w8a8_fused(xv, w, sw, bias=bias, out_dtype=dt)
            bits = torch.int16 if dt == BF16 else torch.int32
            # NaN rows compare as bits
            assert torch.equal(one.view(bits), two.view(bits))


# ------------------------------------------------------------------ together
def test_block_path_together(gpu):
    """The QKV projection in 8 bits, the norm and rotation of its heads to 8-bit codes, and
    the score product of a head on strided views, against the oracle's chain on the same codes."""
    announce("8-bit block path")
    T, H, D, K = 200, 3, 64, 320
    x = _x(T, K, BF16, 1, 1.0)
    wt = _x(3 * H * D, K, BF16, 2, 0.2)
    xq, xs = gpu.quantize_int8(x.cuda())
    wq, ws = gpu.quantize_int8(wt.cuda())
    qkv = gpu.gemm_w8a8(xq, xs, wq, ws)
    v, _ = oracle.gemm_w8a8(*oracle.quantize_int8(_np(x)), *oracle.quantize_int8(_np(wt)))
    _check(qkv, v, False)
    q, k = qkv[:, :H * D].view(T, H, D), qkv[:, H * D:2 * H * D].view(T, H, D)
    ang = torch.arange(T)[:, None] * torch.rand(D // 2, generator=torch.Generator().manual_seed(3))
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    wn = torch.rand(D, generator=torch.Generator().manual_seed(4)).cuda()
    qc, qs, kc, ks = gpu.quantize_qk_norm_rope(q, k, wn, wn, cos, sin)
    for h in range(H):
        s = gpu.gemm_w8a8(qc[:, h], qs[:, h], kc[:, h], ks[:, h], out_dtype=F32)
        v, _ = oracle.gemm_w8a8(qc[:, h].cpu().numpy(), qs[:, h].cpu().numpy(), kc[:, h].cpu().numpy(), ks[:, h].cpu().numpy())
        _check(s, v, False)
        # against the unquantized heads: each code is off by at most half a step plus the
        # kernel's binary32 roundings (127 * 2^-18 of a step), for both factors
        qf, _ = oracle.qk_norm_rope(_np(q), wn.cpu().numpy(), cos.cpu().numpy(), sin.cpu().numpy())
        kf, _ = oracle.qk_norm_rope(_np(k), wn.cpu().numpy(), cos.cpu().numpy(), sin.cpu().numpy())
        eq = (0.5 + 2.0 ** -11) * qs[:, h].cpu().double().numpy()[:, None]
        ek = (0.5 + 2.0 ** -11) * ks[:, h].cpu().double().numpy()[:, None]
        bound = eq * np.abs(kf[:, h]).sum(-1)[None, :] + np.abs(qf[:, h]).sum(-1)[:, None] * ek.T + D * eq * ek.T
        exact = qf[:, h] @ kf[:, h].T
        assert np.all(np.abs(s.double().cpu().numpy() - exact) <= bound * (1 + 1e-6))
