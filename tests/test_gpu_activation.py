"""The feed-forward activation, its 8-bit checkpoint and its gradient on the GPU against the float64 oracle.

Tolerances, in steps of 2^-24, before the half step of the output type.  z (in powers of two) has three
roundings and two rounded constants, which exp turns into 6 |z| of its value, exp and 1 / (1 + e) 2 each, and the
sum and products 1 each: |y - ref| <= (6 |z| + 16) |y|, and where exp(-z) overflows (z below -88) y may be 0:
2^-100 |u|.  The slope's two terms take that twice: (12 |z| + 32) of the sum of their magnitudes."""

import numpy as np
import pytest
import torch

import oracle
from oracle import training as tr
from helpers import announce, bf16_from_bits

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
ACTS = ["gelu_tanh", "silu"]


def _np(t):
    return t.detach().double().cpu().numpy()


def _forward_tol(u, act):
    ref, z = tr.activation(u, act)
    return ref, 2.0 ** -24 * (6 * z + 16) * np.abs(ref) + 2.0 ** -100 * np.abs(u)


def _check(out, ref, tol):
    got = _np(out)
    tol = tol + HALF[out.dtype] * np.abs(ref) * (1 + 2.0 ** -10) + 2.0 ** -134
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.all((np.abs(got - ref) <= tol) | (got == ref) | np.isnan(ref))


def _check_slope(gpu, dy, codes, s, act):
    v = oracle.dequantize_int8(codes.cpu().numpy(), s.cpu().numpy())
    slope, z, size = tr.activation_slope(v, act)
    d = _np(dy)
    _check(gpu.activation_backward(dy, codes, s, act), d * slope, 2.0 ** -24 * (12 * z + 32) * size * np.abs(d))


SHAPES = [(1, 16), (1, 13824), (3, 512), (5, 528), (9, 1024), (7, 1360), (6, 2048), (4, 2064), (3, 4096), (5, 4112), (2, 8192), (3, 8208),
          (2, 16384), (1, 16400), (2, 65536), (130, 96), (777, 1936), (515, 5120)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,C", SHAPES)
def test_matches_oracle(gpu, T, C, dtype, act):
    announce(f"activation {act} {T}x{C} {dtype}")
    g = torch.Generator().manual_seed(T * 3 + C)
    u = (torch.randn(T, C + 16, generator=g) * 2).to(dtype).cuda()[:, :C]
    u[0, :8] = torch.tensor([0.0, -0.0, 30.0, -30.0, 1e-30, -1e-30, 300.0, -9.0]).to(dtype)
    ref, tol = _forward_tol(_np(u), act)
    y = gpu.activation(u, act)
    _check(y, ref, tol)
    y2, codes, s = gpu.activation(u, act, save="int8")
    assert torch.equal(y, y2)
    rc, rs = tr.activation_checkpoint(u.float().cpu().numpy(), act)
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs)
    # to codes
    q, qs, c2, s2 = gpu.quantize_activation(u, act, save="int8")
    assert torch.equal(c2, codes) and torch.equal(s2, s)
    step, sv = np.abs(ref).max(-1) / 127, _np(qs)
    assert np.all(np.abs(sv - step) <= tol.max(-1) / 127 + 2.0 ** -24 * step)
    assert np.all(np.abs(_np(q) * sv[:, None] - ref) <= (0.5 + 127 * 2.0 ** -22) * sv[:, None] + tol)
    again = gpu.quantize_activation(u, act)
    assert len(again) == 2 and torch.equal(again[0], q) and torch.equal(again[1], qs)
    # backward
    dy = torch.randn(T, C + 32, generator=g).to(dtype).cuda()[:, :C]
    _check_slope(gpu, dy, codes, s, act)


@pytest.mark.parametrize("act", ACTS)
def test_every_bf16(gpu, act):
    """Every bf16 pattern, the non-finite ones in rows of their own, against the oracle and torch's rules of infinities."""
    announce(f"activation {act} every bf16")
    bits = np.arange(65536, dtype=np.uint16).reshape(256, 256)     # row: sign and the high exponent bits
    u = bf16_from_bits(bits)
    y, codes, s = gpu.activation(u, act, save="int8")
    x = _np(u)
    fin = np.isfinite(x)
    ref, tol = _forward_tol(np.where(fin, x, 0.0), act)
    got = _np(y)
    ok = np.abs(got - ref) <= tol + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -10) + 2.0 ** -134
    assert np.all(ok | ~fin)
    assert np.all(np.isnan(got[np.isnan(x)])) and np.all(got[x == np.inf] == np.inf) and np.all(np.isnan(got[x == -np.inf]))
    rc, rs = tr.activation_checkpoint(u.float().cpu().numpy(), act)
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(s.cpu().numpy(), rs, equal_nan=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C", [96, 1360, 13824])
def test_bad_rows_stay_alone(gpu, dtype, C, act):
    announce(f"activation {act} non-finite rows {C} {dtype}")
    g = torch.Generator().manual_seed(4)
    u = torch.randn(9, C, generator=g).to(dtype).cuda()
    clean = gpu.quantize_activation(u, act, save="int8")
    u[1, 3], u[4, C - 1], u[6, C // 2] = float("inf"), float("nan"), -float("inf")
    q, qs, c, s = gpu.quantize_activation(u, act, save="int8")
    y = gpu.activation(u, act)
    for t in range(9):
        if t in (1, 4, 6):
            assert qs[t].isnan() and not q[t].any() and y[t].isnan().sum() == (t != 1)
        else:
            assert all(torch.equal(a[t], b[t]) for a, b in zip((q, qs, c, s), clean))
    L = tr.LIMITS[act]
    assert s[4].isnan() and not c[4].any()
    for t, code in ((1, 127), (6, -127)):    # an infinity saturates
        assert s[t].item() == np.float32(L / 127) and c[t, {1: 3, 6: C // 2}[t]].item() == code
    du = gpu.activation_backward(torch.ones(9, C, dtype=dtype, device="cuda"), c, s, act)
    assert du[4].isnan().all() and not du[[0, 1, 2, 3, 5, 6, 7, 8]].isnan().any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_in_place_and_neighbours(gpu, dtype):
    announce(f"activation in place {dtype}")
    g = torch.Generator().manual_seed(5)
    for T, C in ((37, 96), (5, 1360), (3, 13824)):
        wide = torch.randn(T + 2, C + 32, generator=g).to(dtype).cuda()
        u, before = wide[1:T + 1, 16:C + 16], wide.clone()
        ref, codes, s = gpu.activation(u.contiguous(), save="int8")
        o, c2, s2 = gpu.activation(u, save="int8", out=u)
        assert o is u and torch.equal(u, ref) and torch.equal(c2, codes) and torch.equal(s2, s)
        du = gpu.activation_backward(u.contiguous(), codes, s)
        assert gpu.activation_backward(u, codes, s, out=u) is u and torch.equal(u, du)
        wide[1:T + 1, 16:C + 16] = before[1:T + 1, 16:C + 16]
        assert torch.equal(wide, before)


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(gpu, act):
    """At the points that a checkpoint stands for, the slope against central differences of the kernel's own
    forward pass in binary32: 2^-20 of at most 4 over 2 h, and h^2 / 6 times a third derivative below 2."""
    announce(f"activation differences {act}")
    L, h = tr.LIMITS[act], 2.0 ** -6
    codes = torch.arange(-127, 129, device="cuda").clamp(max=127).to(torch.int8).view(1, 256)
    s = torch.full((1,), L / 127, device="cuda")
    v = codes.float() * s
    slope = gpu.activation_backward(torch.ones(1, 256, device="cuda"), codes, s, act)
    diff = (gpu.activation(v + h, act).double() - gpu.activation(v - h, act).double()) / (2 * h)
    assert (diff - slope.double()).abs().max().item() < 2.0 ** -18 / (2 * h) * 2 + 2 * h * h / 6


def test_codes_of_all_values(gpu):
    """-128 is a code like any other to the backward pass."""
    announce("activation_backward every code")
    codes = torch.arange(-128, 128, dtype=torch.int16, device="cuda").to(torch.int8).view(1, 256).repeat(3, 1)
    s = torch.tensor([4.0 / 127, 0.0, 1e-3], device="cuda")
    for act in ACTS:
        for dtype in (BF16, F32):
            _check_slope(gpu, torch.full((3, 256), 1.5, dtype=dtype, device="cuda"), codes, s, act)


def test_empty(gpu):
    u = torch.zeros(0, 64, dtype=BF16, device="cuda")
    y, c, s = gpu.activation(u, save="int8")
    assert y.shape == c.shape == (0, 64) and s.shape == (0,) and gpu.activation_backward(y, c, s).shape == (0, 64)
    z = torch.zeros(3, 0, dtype=BF16, device="cuda")
    assert gpu.activation(z).shape == (3, 0)


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_slope_far_beyond_the_checkpoint(gpu, act):
    """Scales that no checkpoint has: the derivative goes to its limits, 0 and 1, and never to NaN."""
    announce(f"activation_backward far values {act}")
    codes = torch.tensor([-128, -127, -100, 0, 100, 126, 127, 127] * 2, dtype=torch.int8, device="cuda").repeat(5, 1)
    scales = torch.tensor([0.5, 1.0, 16.0, 100.0, 1e4], device="cuda")
    slope = gpu.activation_backward(torch.ones(5, 16, device="cuda"), codes, scales, act)
    v = codes.float() * scales[:, None]
    assert torch.equal(v < 0, codes < 0) and bool((v.abs()[codes != 0] >= 50).all())
    # beyond 50 the distance from a limit is under 51 exp(-50), less than a step of binary32
    want = torch.where(v > 0, 1.0, torch.where(v < 0, 0.0, 0.5))
    assert bool(((slope - want).abs() <= 2.0 ** -23).all())


@pytest.mark.parametrize("C", [72, 264, 1032, 1048, 2056, 4104, 9224])
def test_large_rows_past_the_caches(gpu, C):
    """Inputs over 256 MB are stored past the caches, in runs of 4 lanes where a row has them: the bits of small ones."""
    announce(f"large binary32 rows of {C}")
    T = (300 << 20) // (4 * C) + 3
    x = torch.randn(T, C, device="cuda")
    w = torch.rand(C, device="cuda") + 0.5
    for run in (lambda t: gpu.activation(t, "silu"), lambda t: gpu.layer_norm(t, w)):
        whole = run(x)
        for r in range(0, T, T // 3):
            part = slice(r, min(r + T // 3, T))
            assert torch.equal(whole[part], run(x[part]))
    y = x.clone()
    assert torch.equal(gpu.activation(y, "silu", out=y), gpu.activation(x, "silu")) and y.shape == x.shape
