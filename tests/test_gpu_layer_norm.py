"""Layer norm (to the input's type and to 8-bit codes) and its gradient on the GPU against the float64 oracle.

Tolerances, in steps of 2^-24, before the half step of the output type:
* forward: a sum of C terms passes at most 32 additions in a thread, 6 in a wave and 8 across waves, so the
  mean that is taken off is within 48 mean|d| <= 48 / rstd, and 1 / rstd within (48 + 3) / 2 + 4 of itself (the root
  halves, rsqrt has 2 of 2^-23 at most); x - m0, d - e, the two products and the sum with b add 5:
  |y - ref| <= (48 + 5 + 30 |xh|) |w| + |y| < 64 |w| (1 + |xh|) + |y|, i.e. 2^-18 of the oracle's size.
* backward, for the given statistics: the row's two sums pass at most 16 + 6 + 4 additions of terms with 3
  roundings; xh, g, the last sums and products add 8 to their terms: below 64, 2^-18 of the size.
* dw, db: at most rows / 256 + 2 rows in a thread, then parts / 64 + 2 + 16 in the joining: 2^-17 of the sum of
  magnitudes for the sizes here (fewer than 128 additions)."""

import numpy as np
import pytest
import torch

import oracle
from oracle import training as tr
from helpers import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _rows(g, T, C, dtype, pad=0, scale=1.0, shift=0.0):
    wide = torch.randn(T, C + pad, generator=g) * scale + shift
    return wide.to(dtype).cuda()[:, :C]


def _near(out, ref, size, steps=2.0 ** -18):
    got = _np(out)
    tol = steps * size + HALF[out.dtype] * np.abs(ref) * (1 + 2.0 ** -10) + 2.0 ** -134
    assert got.shape == ref.shape and np.all(np.abs(got - ref) <= tol), np.nanmax(np.abs(got - ref) / tol)


def _stats_near(mean, rstd, x, ref_mean, ref_rstd):
    sigma = np.asarray(x).std(axis=-1)
    assert np.all(np.abs(_np(mean) - ref_mean) <= 2.0 ** -18 * sigma + 2.0 ** -23 * np.abs(ref_mean) + 2.0 ** -134)
    assert np.all(np.abs(_np(rstd) - ref_rstd) <= 2.0 ** -18 * ref_rstd)


# every route: a wave a row with 1, 2 and 4 units a thread, 4 and 8 waves; odd rows
SHAPES = [(1, 8), (1, 5120), (3, 64), (5, 504), (7, 512), (2, 520), (9, 1016), (6, 1360), (5, 2048), (4, 2056), (3, 4096), (5, 4112),
          (2, 6144), (3, 6152), (1, 8192), (2, 8200), (3, 13824), (1, 16384), (130, 96), (1001, 1360), (513, 5120), (2050, 264)]


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,C", SHAPES)
def test_forward_matches_oracle(gpu, T, C, dtype, wdtype):
    announce(f"layer_norm {T}x{C} {dtype} w {wdtype}")
    g = torch.Generator().manual_seed(T * 7 + C)
    x = _rows(g, T, C, dtype, pad=16 if C % 16 == 0 else 8, scale=2.0, shift=0.7)
    w, b = (1 + 0.3 * torch.randn(C, generator=g)).to(wdtype).cuda(), torch.randn(C, generator=g).to(wdtype).cuda()
    for ww, bb in ((w, b), (None, None), (w, None), (None, b)):
        ref, m, r, size = tr.layer_norm(_np(x), _np(ww), _np(bb), 1e-5)
        y, mean, rstd = gpu.layer_norm(x, ww, bb, eps=1e-5, save="x")
        _near(y, ref, size)
        _stats_near(mean, rstd, _np(x), m, r)
        assert torch.equal(y, gpu.layer_norm(x, ww, bb, eps=1e-5))
    if C % 16:
        return
    y8, mean8, rstd8, xc, xs = gpu.layer_norm(x, w, b, eps=1e-5, save="int8")
    y, mean, rstd = gpu.layer_norm(x, w, b, eps=1e-5, save="x")
    qc, qs = gpu.quantize_int8(x)
    assert torch.equal(y8, y) and torch.equal(mean8, mean) and torch.equal(rstd8, rstd)
    assert torch.equal(xc, qc) and torch.equal(xs, qs)
    # to codes: every value within half a step of its code, the step within its roundings
    ref, _, _, size = tr.layer_norm(_np(x), _np(w), _np(b), 1e-5)
    codes, s, m2, r2, xc, xs = gpu.quantize_layer_norm(x, w, b, eps=1e-5, save="int8")
    assert torch.equal(m2, mean) and torch.equal(r2, rstd) and torch.equal(xc, qc) and torch.equal(xs, qs)
    tol = 2.0 ** -18 * size + 2.0 ** -24 * np.abs(ref)
    step, sv = np.abs(ref).max(-1) / 127, _np(s)
    assert np.all(np.abs(sv - step) <= tol.max(-1) / 127 + 2.0 ** -24 * step)
    # the code's product and sum, and s against 1 / inv: three roundings of up to 127 steps
    assert np.all(np.abs(_np(codes) * sv[:, None] - ref) <= (0.5 + 127 * 2.0 ** -22) * sv[:, None] + tol)
    assert np.abs(_np(codes)).max() == 127
    again = gpu.quantize_layer_norm(x, w, b, eps=1e-5)
    assert len(again) == 2 and torch.equal(again[0], codes) and torch.equal(again[1], s)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_means_and_equal_rows(gpu, dtype):
    """A mean far from zero costs nothing beyond the input's own digits; a row of equal values is b."""
    announce(f"layer_norm far means {dtype}")
    g = torch.Generator().manual_seed(3)
    C = 1040
    x = _rows(g, 6, C, dtype)
    x[1] = (torch.randn(C, generator=g) + 1000).to(dtype).cuda()
    x[2] = (torch.randn(C, generator=g) * 1e-3 - 300).to(dtype).cuda()
    x[3], x[4], x[5] = 12345.0, 0.0, x[0] * 2.0 ** 40
    b = torch.randn(C, generator=g).cuda()
    ref, m, r, size = tr.layer_norm(_np(x), None, _np(b))
    y, mean, rstd = gpu.layer_norm(x, None, b, save="x")
    _near(y, ref, size)
    _stats_near(mean, rstd, _np(x), m, r)
    assert torch.equal(y[3], b.to(dtype)) and torch.equal(y[4], b.to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C", [96, 1360, 5120, 16384])
def test_bad_rows_stay_alone(gpu, dtype, C):
    announce(f"layer_norm non-finite rows {C} {dtype}")
    g = torch.Generator().manual_seed(4)
    x = _rows(g, 9, C, dtype)
    clean, ccodes, cscales = gpu.layer_norm(x), *gpu.quantize_layer_norm(x)
    x[1, 3], x[4, C - 1], x[6, C // 2] = float("inf"), float("nan"), -float("inf")
    y, mean, rstd, xc, xs = gpu.layer_norm(x, save="int8")
    codes, scales = gpu.quantize_layer_norm(x)
    for t in range(9):
        if t in (1, 4, 6):
            assert y[t].isnan().all() and rstd[t].isnan() and scales[t].isnan() and not codes[t].any() and xs[t].isnan()
        else:
            assert torch.equal(y[t], clean[t]) and torch.equal(codes[t], ccodes[t]) and scales[t] == cscales[t]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_in_place_and_neighbours(gpu, dtype):
    """Outputs over the inputs and inside wider buffers; nothing beside the rows is written."""
    announce(f"layer_norm in place {dtype}")
    g = torch.Generator().manual_seed(5)
    for T, C in ((37, 96), (5, 5120), (3, 13824)):
        wide = torch.randn(T + 2, C + 32, generator=g).to(dtype).cuda()
        x = wide[1:T + 1, 16:C + 16]
        before, ref = wide.clone(), gpu.layer_norm(x.contiguous())
        assert gpu.layer_norm(x, out=x) is x and torch.equal(x, ref)
        wide[1:T + 1, 16:C + 16] = before[1:T + 1, 16:C + 16]
        assert torch.equal(wide, before)
        dy = torch.randn(T + 2, C + 32, generator=g).to(dtype).cuda()
        inner, kept = dy[1:T + 1, 16:C + 16], dy.clone()
        _, mean, rstd = gpu.layer_norm(x, save="x")
        w = torch.randn(C, generator=g).cuda()
        dx, dw, db = gpu.layer_norm_backward(inner.contiguous(), x, mean, rstd, w)
        o, dw2, db2 = gpu.layer_norm_backward(inner, x, mean, rstd, w, out=inner)
        assert o is inner and torch.equal(inner, dx) and torch.equal(dw, dw2) and torch.equal(db, db2)
        dy[1:T + 1, 16:C + 16] = kept[1:T + 1, 16:C + 16]
        assert torch.equal(dy, kept)


BACK = [(1, 8), (1, 5120), (2, 64), (3, 504), (5, 512), (77, 1360), (9, 2064), (63, 5120), (1023, 264), (1024, 272), (1025, 1040), (3, 8192),
        (4, 8208), (2, 13824), (5, 16384), (1031, 8208), (4099, 528)]


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,C", BACK)
def test_backward_matches_oracle(gpu, T, C, dtype, wdtype):
    announce(f"layer_norm_backward {T}x{C} {dtype} w {wdtype}")
    g = torch.Generator().manual_seed(T * 11 + C)
    x, dy = _rows(g, T, C, dtype, 16 if C % 16 == 0 else 8, 2.0, 0.5), _rows(g, T, C, dtype, 32 if C % 16 == 0 else 24)
    w = (1 + 0.3 * torch.randn(C, generator=g)).to(wdtype).cuda()
    _, mean, rstd = gpu.layer_norm(x, w, save="x")
    sources = [(x, None, _np(x))]
    if C % 16 == 0:
        codes, s = gpu.quantize_int8(x)
        sources.append((codes, s, oracle.dequantize_int8(codes.cpu().numpy(), s.cpu().numpy())))
    for src, s, values in sources:
        dx, dw, db, size, size_w, size_b = tr.layer_norm_backward(_np(dy), values, _np(mean), _np(rstd), _np(w))
        got = gpu.layer_norm_backward(dy, src, mean, rstd, w, x_scales=s)
        _near(got[0], dx, size)
        _near(got[1], dw, size_w, 2.0 ** -17)
        _near(got[2], db, size_b, 2.0 ** -17)
        assert all(torch.equal(a, b) for a, b in zip(got, gpu.layer_norm_backward(dy, src, mean, rstd, w, x_scales=s)))
        dx, _, _, size, _, _ = tr.layer_norm_backward(_np(dy), values, _np(mean), _np(rstd))
        plain = gpu.layer_norm_backward(dy, src, mean, rstd, x_scales=s)
        assert plain[1] is None and plain[2] is None
        _near(plain[0], dx, size)


def test_backward_against_differences(gpu):
    """The gradient of sum(y * dy) along a direction against central differences of the kernel's own forward
    pass in binary32: rounding of y (2^-20 of at most 16 each, 4096 terms, random signs) over 2 h, and h^2 terms."""
    announce("layer_norm_backward differences")
    g = torch.Generator().manual_seed(8)
    T, C, h = 8, 512, 2.0 ** -7
    x, dy, v = (torch.randn(T, C, generator=g).cuda() for _ in range(3))
    w, b = (1 + 0.3 * torch.randn(C, generator=g)).cuda(), torch.randn(C, generator=g).cuda()
    _, mean, rstd = gpu.layer_norm(x, w, b, save="x")
    dx, dw, db = gpu.layer_norm_backward(dy, x, mean, rstd, w)
    f = lambda *a: (gpu.layer_norm(*a).double() * dy.double()).sum().item()   # noqa: E731
    scale = (dx.abs() * v.abs()).sum().item()
    assert abs((f(x + h * v, w, b) - f(x - h * v, w, b)) / (2 * h) - (dx.double() * v.double()).sum().item()) < 1e-3 * scale
    u = v[0]
    assert abs((f(x, w + h * u, b) - f(x, w - h * u, b)) / (2 * h) - (dw * u).sum().item()) < 1e-4 * (dw * u).abs().sum().item()
    assert abs((f(x, w, b + h * u) - f(x, w, b - h * u)) / (2 * h) - (db * u).sum().item()) < 1e-4 * (db * u).abs().sum().item()


def test_backward_of_bad_rows(gpu):
    """A row with a NaN gives NaN in its own dx and in the sums over rows, and nowhere else."""
    announce("layer_norm_backward bad rows")
    g = torch.Generator().manual_seed(9)
    x, dy, w = _rows(g, 7, 528, BF16), _rows(g, 7, 528, BF16), torch.ones(528, device="cuda")
    _, mean, rstd = gpu.layer_norm(x, save="x")
    clean = gpu.layer_norm_backward(dy, x, mean, rstd, w)
    dy[3, 100] = float("nan")
    got = gpu.layer_norm_backward(dy, x, mean, rstd, w)
    rows = [0, 1, 2, 4, 5, 6]
    assert got[0][3].isnan().all() and torch.equal(got[0][rows], clean[0][rows])
    cols = torch.arange(528, device="cuda") != 100
    assert got[2][100].isnan() and torch.equal(got[2][cols], clean[2][cols]) and torch.equal(got[1][cols], clean[1][cols])


def test_empty(gpu):
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    y, mean, rstd, c, s = gpu.layer_norm(x, save="int8")
    assert y.shape == (0, 64) and mean.numel() == 0 and c.shape == (0, 64)
    dx, dw, db = gpu.layer_norm_backward(x, x, mean, rstd, torch.ones(64, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any() and not db.any() and dw.shape == (64,)


@pytest.mark.parametrize("T,C", [(5, 96), (3, 1040), (7, 4112), (2, 9008), (1100, 272)])
def test_sums_and_weights_apart(gpu, T, C):
    """Through the C ABI: weights without their sums, and sums without weights (weights of 1)."""
    announce(f"layer_norm_backward apart {T}x{C}")
    g = torch.Generator().manual_seed(T)
    x, dy, w = _rows(g, T, C, F32), _rows(g, T, C, F32), torch.randn(C, generator=g).cuda()
    _, mean, rstd = gpu.layer_norm(x, save="x")
    ptr = lambda t: None if t is None else t.data_ptr()   # noqa: E731
    nbytes = gpu.lib.mxq_layer_norm_backward_workspace_bytes(T, C)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")

    def call(w, dw, db):
        dx = torch.empty_like(x)
        st = gpu.lib.mxq_layer_norm_backward(ptr(dy), 0, T, C, C, ptr(x), C, None, ptr(mean), ptr(rstd), ptr(w), 0, ptr(dx), C, ptr(dw), ptr(db),
                                             ptr(ws), nbytes, torch.cuda.current_stream().cuda_stream)
        assert st == 0, gpu.lib.mxq_last_error()
        return dx

    full, dw, db = gpu.layer_norm_backward(dy, x, mean, rstd, w)
    assert torch.equal(call(w, None, None), full)
    ones, sw, sb = torch.ones(C, device="cuda"), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    plain = call(None, sw, sb)
    assert torch.equal(plain, gpu.layer_norm_backward(dy, x, mean, rstd, ones)[0]) and torch.equal(sw, dw) and torch.equal(sb, db)
    assert torch.equal(plain, gpu.layer_norm_backward(dy, x, mean, rstd)[0])


@pytest.mark.parametrize("C", [64, 512, 1360, 5120, 13824])
def test_rows_without_finite_statistics(gpu, C):
    """Squares past binary32, and equal values without eps: NaN scales and codes of 0 in the quantized form, other
    rows as they are alone."""
    announce(f"layer_norm statistics {C}")
    g = torch.Generator().manual_seed(C)
    x = _rows(g, 6, C, F32)
    clean, cs = gpu.quantize_layer_norm(x, eps=0.0)
    x[1], x[4] = x[1] * 1e30, 3.0
    codes, s = gpu.quantize_layer_norm(x, eps=0.0)
    y = gpu.layer_norm(x, eps=0.0)
    assert y[4].isnan().all() and s[[1, 4]].isnan().all() and not codes[[1, 4]].any()
    keep = [0, 2, 3, 5]
    assert torch.equal(codes[keep], clean[keep]) and torch.equal(s[keep], cs[keep])


def test_weights_that_are_not_numbers(gpu):
    """A NaN or an infinity in a weight or bias reaches its column of every row: the rows' scales are NaN."""
    announce("layer_norm bad weights")
    for C in (64, 528, 1040, 5120, 13824):
        x = torch.randn(3, C, device="cuda")
        for bad in (float("nan"), float("inf")):
            for which in (0, 1):
                v = [torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")]
                v[which][C - 3] = bad
                codes, s = gpu.quantize_layer_norm(x, *v)
                y = gpu.layer_norm(x, *v)
                cols = torch.arange(C, device="cuda") != C - 3
                assert s.isnan().all() and not codes.any() and not y[:, C - 3].isfinite().any() and y[:, cols].isfinite().all()
