"""Norm and rotation of query and key heads on the GPU against the float64 oracle.

Tolerance: the kernel's sum of squares has at most 15 roundings of non-negative terms, which
the square root halves; the reciprocal root, x r, (x r) w, the two products and the sum of
the rotation add at most 7 more, and the tables are exact inputs: 15 / 2 + 7 < 16 steps of
2^-24, i.e. 2^-20 relative to |a c| + |b s|; then half a step of the output type."""

import numpy as np
import pytest
import torch

import oracle
from helpers import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _inputs(T, Hq, Hk, D, R, P, dtype, wdtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, (Hq + 2 * Hk) * D, generator=g) * scale).to(dtype).cuda()
    q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).to(wdtype).cuda() for _ in range(2))
    cos = sin = pos = None
    if R:
        ang = torch.rand(P, R // 2, generator=g, dtype=torch.float64) * 50
        cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()
        pos = torch.randint(0, P, (T,), generator=g).cuda()
    return qkv, q, k, wq, wk, cos, sin, pos


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _oracle(x, w, cos, sin, pos, eps, style):
    return oracle.qk_norm_rope(_np(x), _np(w), _np(cos), _np(sin), None if pos is None else pos.cpu().numpy(), eps, style)


def _check(out, ref, size):
    got = _np(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    tol = 2.0 ** -20 * size + HALF[out.dtype] * np.abs(ref) * (1 + 2.0 ** -12) + 2.0 ** -134
    assert np.all((np.abs(got - ref) <= tol) | np.isnan(ref))


CASES = [  # T, Hq, Hk, D, R
    (1, 1, 1, 8, 8), (1, 32, 8, 128, 128), (2, 3, 1, 64, 64), (3, 5, 5, 72, 40), (7, 4, 2, 96, 64), (5, 24, 24, 128, 128),
    (9, 2, 2, 256, 128), (4, 3, 2, 264, 264), (3, 2, 1, 512, 512), (33, 12, 3, 80, 40), (130, 40, 40, 128, 128),
    (511, 2, 2, 64, 32), (512, 3, 2, 128, 64), (700, 5, 1, 80, 80), (515, 9, 7, 256, 256), (600, 2, 3, 512, 8), (513, 1, 0, 16, 16),
    (513, 0, 4, 40, 24), (6, 0, 3, 128, 128), (6, 2, 0, 128, 0), (600, 17, 4, 64, 0), (520, 33, 33, 120, 56)]


@pytest.mark.parametrize("style", ["interleaved", "halves"])
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,Hq,Hk,D,R", CASES)
def test_matches_oracle(gpu, T, Hq, Hk, D, R, dtype, wdtype, style):
    announce(f"qk_norm_rope T={T} {Hq}+{Hk}x{D} R={R} {dtype} w {wdtype} {style}")
    qkv, q, k, wq, wk, cos, sin, pos = _inputs(T, Hq, Hk, D, R, 37, dtype, wdtype, T + D)
    before = qkv.clone()
    oq, ok = gpu.qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, eps=1e-5, style=style)
    assert torch.equal(qkv, before)
    _check(oq, *_oracle(q, wq, cos, sin, pos, 1e-5, style))
    _check(ok, *_oracle(k, wk, cos, sin, pos, 1e-5, style))
    # quantized: every value within half a step of its code, the step within its roundings
    qc, qs, kc, ks = gpu.quantize_qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, eps=1e-5, style=style)
    for c, s, x, w in ((qc, qs, q, wq), (kc, ks, k, wk)):
        ref, size = _oracle(x, w, cos, sin, pos, 1e-5, style)
        if ref.size == 0:
            assert c.numel() == 0
            continue
        step = np.abs(ref).max(-1) / 127
        off = 2.0 ** -20 * size.max(-1) / 127 + 2.0 ** -24 * step
        assert np.all(np.abs(_np(s) - step) <= off)
        # x inv: 127 steps times (2^-20 |size| / amax + two roundings), size <= sqrt(2) amax of the pair's
        # length, itself at most sqrt(2) amax: below 127 * 2^-18
        err = np.abs(_np(c) * _np(s)[..., None] - ref)
        assert np.all(err <= (0.5 + 127 * 2.0 ** -18) * _np(s)[..., None] + 2.0 ** -20 * size)
        assert np.abs(_np(c)).max() == 127


def test_in_place_and_strided_heads(gpu):
    """Outputs over the inputs; heads that are not next to each other ([T, H, 3, D] packing);
    what lies between them stays."""
    announce("qk_norm_rope in place")
    T, H, D = 530, 3, 96
    for dtype in (BF16, F32):
        for style in ("interleaved", "halves"):
            g = torch.Generator().manual_seed(2)
            packed = torch.randn(T, H, 3, D, generator=g).to(dtype).cuda()
            before = packed.clone()
            q, k = packed[:, :, 0], packed[:, :, 1]
            ang = torch.rand(T, D // 2, generator=g) * 9
            cos, sin = ang.cos().cuda(), ang.sin().cuda()
            rq, rk = gpu.qk_norm_rope(q, k, None, None, cos, sin, style=style)
            _check(rq, *_oracle(q, None, cos, sin, None, 1e-6, style))
            oq, ok = gpu.qk_norm_rope(q, k, None, None, cos, sin, style=style, out_q=q, out_k=k)
            assert torch.equal(oq, rq) and torch.equal(ok, rk) and torch.equal(packed[:, :, 2], before[:, :, 2])


def test_no_rotation_is_the_norm_alone(gpu):
    announce("qk_norm_rope without tables")
    _, q, k, wq, wk, _, _, _ = _inputs(12, 4, 2, 128, 0, 1, BF16, BF16, 7)
    oq, ok = gpu.qk_norm_rope(q, k, wq, wk, None, None)
    _check(oq, *_oracle(q, wq, None, None, None, 1e-6, "halves"))
    _check(ok, *_oracle(k, wk, None, None, None, 1e-6, "halves"))


@pytest.mark.parametrize("T", [4, 600])
def test_positions_outside_the_table_give_nan(gpu, T):
    announce(f"qk_norm_rope bad positions T={T}")
    _, q, k, wq, wk, cos, sin, pos = _inputs(T, 2, 2, 96, 64, 10, BF16, BF16, 3)
    pos[1], pos[2], pos[3] = -1, 10, 2 ** 62
    good = pos.clone()
    good[1:4] = 0
    for style in ("interleaved", "halves"):
        oq, ok = gpu.qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, style=style)
        _check(oq, *_oracle(q, wq, cos, sin, pos, 1e-6, style))
        assert oq[1:4, :, :64].isnan().all() and not oq[1:4, :, 64:].isnan().any() and not ok[4:].isnan().any()
        rq, rk = gpu.qk_norm_rope(q, k, wq, wk, cos, sin, positions=good, style=style)
        assert torch.equal(oq[4:], rq[4:]) and torch.equal(ok[0], rk[0])
        qc, qs, kc, ks = gpu.quantize_qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, style=style)
        assert qs[1:4].isnan().all() and not qc[1:4].any() and not qs[4:].isnan().any() and not ks[0].isnan().any()


def test_degenerate_heads(gpu):
    """Zero heads give zeros (eps > 0); an infinity or NaN stays in its head; large and small values."""
    announce("qk_norm_rope degenerate heads")
    _, q, k, wq, wk, cos, sin, pos = _inputs(8, 3, 3, 128, 128, 20, F32, F32, 5)
    q = q.clone()
    q[0, 1] = 0
    q[1, 0, 5] = float("inf")
    q[2, 2, 7] = float("nan")
    q[3] *= 1e15
    q[4] *= 1e-15
    with np.errstate(all="ignore"):
        ref, size = _oracle(q, wq, cos, sin, pos, 1e-6, "halves")
    oq, _ = gpu.qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, style="halves")
    assert (oq[0, 1] == 0).all()
    keep = torch.ones(8, 3, dtype=torch.bool)
    keep[1, 0] = keep[2, 2] = False
    _check(oq.cpu()[keep], ref[keep.numpy()], size[keep.numpy()])
    qc, qs, _, _ = gpu.quantize_qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, style="halves")
    assert qs[0, 1] == 0 and not qc[0, 1].any() and qs[1, 0].isnan() and not qc[1, 0].any() and qs[2, 2].isnan()
    assert int(qs.isnan().sum()) == 2


def test_results_do_not_depend_on_the_batch(gpu):
    """A token gives the same bits alone, among a few and among many (other variants of the
    kernel), in every layout; and the same twice."""
    announce("qk_norm_rope batch invariance")
    T = 3000
    for dtype, D, R, Hq, Hk in ((BF16, 128, 128, 40, 40), (F32, 96, 64, 12, 3), (BF16, 256, 256, 8, 8), (BF16, 64, 64, 24, 24)):
        for style in ("interleaved", "halves"):
            _, q, k, wq, wk, cos, sin, pos = _inputs(T, Hq, Hk, D, R, 100, dtype, dtype, 9)
            kw = dict(eps=1e-6, style=style)
            full = gpu.qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, **kw)
            full8 = gpu.quantize_qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, **kw)
            for _ in range(3):
                again = gpu.qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, **kw)
                assert all(torch.equal(a, b) for a, b in zip(again, full))
            for lo, hi in ((0, 1), (17, 18), (100, 400), (1000, 1600)):
                part = gpu.qk_norm_rope(q[lo:hi], k[lo:hi], wq, wk, cos, sin, positions=pos[lo:hi], **kw)
                part8 = gpu.quantize_qk_norm_rope(q[lo:hi], k[lo:hi], wq, wk, cos, sin, positions=pos[lo:hi], **kw)
                assert all(torch.equal(a, b[lo:hi]) for a, b in zip(part, full))
                assert all(torch.equal(a, b[lo:hi]) for a, b in zip(part8, full8))


@pytest.mark.parametrize("Hq,Hk,D,R", [(1, 1, 128, 128), (2, 1, 80, 40), (4, 4, 128, 64), (7, 1, 104, 104), (8, 8, 64, 64), (3, 0, 32, 32),
                                       (0, 2, 256, 256), (3, 1, 256, 128), (1, 1, 512, 512), (1, 1, 8, 8), (16, 0, 48, 0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_heads_of_many_tokens(gpu, Hq, Hk, D, R, dtype):
    """Waves that take pairs of tokens and heads against the oracle, and against parts of the batch
    that are too small for them; positions outside the table; in place."""
    announce(f"qk_norm_rope {Hq}+{Hk} heads x {D}, rotated {R}, {dtype}")
    T = 1501
    for style in ("interleaved", "halves"):
        qkv, q, k, wq, wk, cos, sin, pos = _inputs(T, Hq, Hk, D, R, 100, dtype, dtype, D + Hq)
        if R:
            pos[5], pos[700], pos[T - 1] = -1, 100, 2 ** 40
        kw = dict(eps=1e-6, style=style)
        full = gpu.qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, **kw)
        full8 = gpu.quantize_qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, **kw)
        good = torch.ones(T, dtype=torch.bool)
        if R:
            good[[5, 700, T - 1]] = False
        safe = pos.cpu().masked_fill(~good, 0) if R else None
        cut = lambda lo: pos[lo:lo + 400] if R else None
        for o, x, w in ((full[0], q, wq), (full[1], k, wk)):
            if x.shape[1]:
                ref, size = _oracle(x, w, cos, sin, safe, 1e-6, style)
                _check(o.cpu()[good], ref[good.numpy()], size[good.numpy()])
                assert bool(o[~good][..., :R].isnan().all())
        bits = lambda t: t.view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])
        for lo in range(0, T, 400):
            part = gpu.qk_norm_rope(q[lo:lo + 400], k[lo:lo + 400], wq, wk, cos, sin, positions=cut(lo), **kw)
            part8 = gpu.quantize_qk_norm_rope(q[lo:lo + 400], k[lo:lo + 400], wq, wk, cos, sin, positions=cut(lo), **kw)
            for a, b in zip((*part, *part8), (*full, *full8)):
                assert torch.equal(bits(a), bits(b[lo:lo + 400]))
        before = qkv.clone()
        gpu.qk_norm_rope(q, k, wq, wk, cos, sin, positions=pos, out_q=q, out_k=k, **kw)
        assert torch.equal(bits(q), bits(full[0])) and torch.equal(bits(k), bits(full[1]))
        assert torch.equal(qkv[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])


def test_one_head_with_any_head_pitch(gpu):
    """A single head has no head pitch: a huge one through the C ABI changes nothing and
    writes nothing else."""
    announce("qk_norm_rope one head, huge head pitch")
    x = torch.randn(5, 1, 64, device="cuda")
    ref, _ = gpu.qk_norm_rope(x, x[:, :0], None, None, None, None)
    out = torch.full((7, 64), -3.0, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    for hs in (0, 1 << 29, 1 << 31):
        out.fill_(-3.0)
        assert gpu.lib.mxq_qk_norm_rope(x.data_ptr(), 1, 64, hs, None, 0, 0, 0, 0, 5, 64, None, None, 0, 1e-6, None, None, 0, 0,
                                        0, None, 0, out[1:].data_ptr(), 64, max(hs, 64), None, 0, 0, st) == 0
        assert torch.equal(out[1:6], ref[:, 0]) and (out[0] == -3).all() and (out[6] == -3).all()


def test_shared_and_many_heads(gpu):
    """Inputs whose heads are one and the same (head pitch 0), and more heads than a grid row
    has workgroups for."""
    announce("qk_norm_rope shared heads")
    for T in (3, 600):
        x = torch.randn(T, 1, 128, device="cuda").to(BF16)
        one, _ = gpu.qk_norm_rope(x, x[:, :0], None, None, None, None)
        many, _ = gpu.qk_norm_rope(x.expand(T, 9, 128), x[:, :0], None, None, None, None)
        assert torch.equal(many, one.expand(T, 9, 128))
    x = torch.randn(2, 40000, 512, device="cuda").to(BF16)
    q, k = gpu.qk_norm_rope(x, x, None, None, None, None)
    assert torch.equal(q, k)
    _check(q[:, ::1777], *_oracle(x[:, ::1777], None, None, None, None, 1e-6, "halves"))


def test_empty(gpu):
    announce("qk_norm_rope empty")
    e = torch.empty(0, 3, 64, device="cuda")
    oq, ok = gpu.qk_norm_rope(e, e, None, None, None, None)
    assert oq.shape == ok.shape == (0, 3, 64)
    e = torch.empty(5, 0, 64, device="cuda")
    qc, qs, kc, ks = gpu.quantize_qk_norm_rope(e, e, None, None, None, None)
    assert qc.shape == (5, 0, 64) and ks.shape == (5, 0)
