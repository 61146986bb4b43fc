"""The layer norm's gradient where a workgroup takes two rows at once, over many waves: binary32 rows of any width up to 8192
columns and bf16 rows of 6152 to 8192, from 1024 rows on, an odd one last.  Against the float64 oracle, with the bounds of
test_gpu_layer_norm."""

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
    return t.detach().double().cpu().numpy()


def _near(out, ref, size, steps):
    got = _np(out)
    tol = steps * size + HALF[out.dtype] * np.abs(ref) * (1 + 2.0 ** -10) + 2.0 ** -134
    assert got.shape == ref.shape and np.all(np.abs(got - ref) <= tol), np.nanmax(np.abs(got - ref) / tol)


@pytest.mark.parametrize("T,C,dtype", [(1025, 528, F32), (1025, 2064, F32), (1031, 5120, F32), (1027, 8184, F32), (1025, 8192, F32),
                                       (1025, 6152, BF16), (1029, 6160, BF16), (1024, 8192, BF16), (1025, 8192, BF16)])
def test_two_rows_at_once(gpu, T, C, dtype):
    announce(f"layer_norm_backward pairs {T}x{C} {dtype}")
    g = torch.Generator().manual_seed(T + C)
    wide = lambda pad, s, m: (torch.randn(T, C + pad, generator=g) * s + m).to(dtype).cuda()[:, :C]   # noqa: E731
    x, dy, w = wide(16, 2.0, 0.5), wide(32, 1.0, 0.0), (1 + 0.3 * torch.randn(C, generator=g)).cuda()
    _, mean, rstd = gpu.layer_norm(x, w, save="x")
    sources = [(x, None, _np(x))]
    if C % 16 == 0:
        codes, s = gpu.quantize_int8(x)
        sources.append((codes, s, oracle.dequantize_int8(codes.cpu().numpy(), s.cpu().numpy())))
    for src, s, values in sources:
        dx, dw, db, size, size_w, size_b = tr.layer_norm_backward(_np(dy), values, _np(mean), _np(rstd), _np(w))
        got = gpu.layer_norm_backward(dy, src, mean, rstd, w, x_scales=s)
        _near(got[0], dx, size, 2.0 ** -18)
        _near(got[1], dw, size_w, 2.0 ** -17)
        _near(got[2], db, size_b, 2.0 ** -17)
        assert all(torch.equal(a, b) for a, b in zip(got, gpu.layer_norm_backward(dy, src, mean, rstd, w, x_scales=s)))
        dx, _, _, size, _, _ = tr.layer_norm_backward(_np(dy), values, _np(mean), _np(rstd))
        _near(gpu.layer_norm_backward(dy, src, mean, rstd, x_scales=s)[0], dx, size, 2.0 ** -18)


def test_pairs_stay_apart(gpu):
    """A NaN in one row of a pair, and in the last row alone, reaches no other row; in place as beside."""
    announce("layer_norm_backward pairs with NaN")
    T, C = 1025, 2064
    x, dy, w = torch.randn(T, C, device="cuda"), torch.randn(T, C, device="cuda"), torch.randn(C, device="cuda")
    _, mean, rstd = gpu.layer_norm(x, w, save="x")
    clean = gpu.layer_norm_backward(dy, x, mean, rstd, w)[0]
    bad = [0, 7, 500, 1024]
    dy[bad, 9] = float("nan")
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[bad] = False
    dx = gpu.layer_norm_backward(dy, x, mean, rstd, w)[0]
    assert dx[bad].isnan().all() and torch.equal(dx[rows], clean[rows])
    assert torch.equal(gpu.layer_norm_backward(dy, x, mean, rstd, w, out=dy)[0].nan_to_num(7.0), dx.nan_to_num(7.0))
