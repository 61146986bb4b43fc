"""Refusals of the 8-bit operators, decided before anything is launched (no GPU needed):
through the C ABI with pointers that are never dereferenced, and through the binding's
checks of tensors."""

import ctypes

import pytest
import torch

import mxfp4_microscaled_quantization_amd as mxq

P = ctypes.c_void_p
OK16 = P(0x10000)
ODD8 = P(0x10008)    # 8-byte but not 16-byte aligned
ODD2 = P(0x10002)
BIG, NEG = 2 ** 63 - 1, -2 ** 63


def _quant(x=OK16, dt=1, rows=4, cols=64, ld=64, codes=OK16, ldc=64, scales=OK16):
    return mxq.lib.mxq_quantize_int8(x, dt, rows, cols, ld, codes, ldc, scales, None)


def _dequant(codes=OK16, ldc=64, scales=OK16, rows=4, cols=64, y=OK16, ldy=64):
    return mxq.lib.mxq_dequantize_int8(codes, ldc, scales, rows, cols, y, ldy, None)


def _gemm(a=OK16, lda=64, sa=OK16, ia=1, w=OK16, ldw=64, sw=OK16, iw=1, bias=None, M=8, N=8, K=64, out=OK16, dt=1, ldo=8,
          ws=None, nbytes=0):
    return mxq.lib.mxq_gemm_w8a8(a, lda, sa, ia, w, ldw, sw, iw, bias, M, N, K, out, dt, ldo, ws, nbytes, None)


def _fused(a=OK16, dt=1, lda=64, w=OK16, ldw=64, sw=OK16, iw=1, bias=None, M=8, N=8, K=64, out=OK16, odt=1, ldo=8,
           ws=OK16, nbytes=1 << 20):
    return mxq.lib.mxq_gemm_w8a8_fused(a, dt, lda, w, ldw, sw, iw, bias, M, N, K, out, odt, ldo, ws, nbytes, None)


def _qk(q=OK16, hq=2, ldq=256, hsq=64, k=OK16, hk=1, ldk=256, hsk=64, dt=1, T=4, D=64, wq=None, wk=None, wdt=1, eps=1e-6,
        cos=OK16, sin=OK16, ldt=32, rows=4, rot=64, pos=None, style=0, oq=OK16, loq=128, hoq=64, ok=OK16, lok=64, hok=64):
    return mxq.lib.mxq_qk_norm_rope(q, hq, ldq, hsq, k, hk, ldk, hsk, dt, T, D, wq, wk, wdt, ctypes.c_float(eps), cos, sin,
                                    ldt, rows, rot, pos, style, oq, loq, hoq, ok, lok, hok, None)


def _qk8(q=OK16, hq=2, T=4, D=64, cq=OK16, lcq=128, hcq=64, sq=OK16, lsq=2, ck=OK16, lck=64, hck=64, sk=OK16, lsk=1, **kw):
    a = dict(dt=1, style=0) | kw
    return mxq.lib.mxq_quantize_qk_norm_rope(q, hq, 256, 64, OK16, 1, 256, 64, a["dt"], T, D, None, None, 1,
                                             ctypes.c_float(1e-6), OK16, OK16, 32, 4, 64, None, a["style"], cq, lcq, hcq,
                                             sq, lsq, ck, lck, hck, sk, lsk, None)


INVALID = [
    (_quant, dict(cols=72), "multiple of 16"), (_quant, dict(rows=-1), "negative"), (_quant, dict(ld=48), "ld_x"),
    (_quant, dict(ld=68), "aligned"), (_quant, dict(x=ODD8), "aligned"), (_quant, dict(x=None), "NULL"),
    (_quant, dict(codes=None), "NULL"), (_quant, dict(codes=ODD8), "multiples of 16"), (_quant, dict(ldc=48), "ld_codes"),
    (_quant, dict(ldc=72), "multiples of 16"), (_quant, dict(scales=None), "scales"), (_quant, dict(scales=ODD2), "scales"),
    (_quant, dict(rows=BIG), "2^31"), (_quant, dict(ldc=BIG), "2^32"), (_quant, dict(cols=0, scales=None), "scales"),
    (_dequant, dict(cols=60), "multiple of 8"), (_dequant, dict(rows=NEG), "not negative"), (_dequant, dict(ldc=48), "pitch"),
    (_dequant, dict(ldy=48), "pitch"), (_dequant, dict(codes=None), "NULL"), (_dequant, dict(scales=None), "NULL"),
    (_dequant, dict(y=None), "NULL"), (_dequant, dict(codes=P(0x10004)), "multiples of 8"), (_dequant, dict(y=ODD8), "16-byte"),
    (_dequant, dict(ldy=68), "16-byte"), (_dequant, dict(scales=ODD2), "4-byte"), (_dequant, dict(rows=BIG, ldc=64), "2^31"),
    (_dequant, dict(rows=2 ** 31 - 1, cols=64), "too large"),
    (_gemm, dict(K=56), "multiple of 16"), (_gemm, dict(K=1 << 17, lda=1 << 17, ldw=1 << 17), "2^17"),
    (_gemm, dict(M=-1), "negative"), (_gemm, dict(N=BIG), "too large"), (_gemm, dict(lda=48), "ld_a"),
    (_gemm, dict(lda=1 << 23), "ld_a"), (_gemm, dict(lda=72), "ld_a"), (_gemm, dict(a=ODD8), "multiples of 16"),
    (_gemm, dict(a=None), "a is NULL"), (_gemm, dict(sa=None), "a_scales"), (_gemm, dict(sa=ODD2), "a_scales"),
    (_gemm, dict(ia=-1), "inc_as"), (_gemm, dict(iw=-1), "inc_ws"), (_gemm, dict(iw=BIG), "inc_ws"),
    (_gemm, dict(ldw=48), "ld_w"), (_gemm, dict(ldw=1 << 23), "ld_w"), (_gemm, dict(ldw=72), "ld_w"),
    (_gemm, dict(w=ODD8), "multiples of 16"), (_gemm, dict(w=None), "w is NULL"), (_gemm, dict(sw=None), "w_scales"),
    (_gemm, dict(bias=ODD2), "bias"), (_gemm, dict(out=None), "out is NULL"), (_gemm, dict(out=P(0x10001)), "2-byte"),
    (_gemm, dict(out=ODD2, dt=0), "4-byte"), (_gemm, dict(ldo=7), "ld_out"), (_gemm, dict(ldo=BIG), "ld_out"),
    (_gemm, dict(M=2 ** 30, N=2 ** 20, ldo=2 ** 20), "too large"),
    (_gemm, dict(M=1, N=2 ** 28 + 1, ldo=2 ** 29), "too large"), (_fused, dict(M=8, N=2 ** 29, ldo=2 ** 29), "too large"),
    (_gemm, dict(ws=ODD8, nbytes=1 << 30), "workspace"),
    (_gemm, dict(M=48, N=5120, K=13824, lda=13824, ldw=13824, ldo=5120, ws=OK16, nbytes=16), "workspace"),
    (_fused, dict(K=56, lda=56), "multiple of 16"), (_fused, dict(lda=48), "ld_x"), (_fused, dict(lda=68), "aligned"),
    (_fused, dict(a=ODD8), "aligned"), (_fused, dict(a=None), "NULL"), (_fused, dict(w=None), "w is NULL"),
    (_fused, dict(M=64, ws=None), "workspace"), (_fused, dict(M=64, ws=ODD8), "workspace"),
    (_fused, dict(M=64, nbytes=64 * 64), "workspace"), (_fused, dict(out=None), "out is NULL"),
    (_qk, dict(D=60), "head_dim"), (_qk, dict(D=0), "head_dim"), (_qk, dict(D=520), "head_dim"), (_qk, dict(rot=72), "rot_dim"),
    (_qk, dict(rot=12), "rot_dim"), (_qk, dict(rot=-8), "rot_dim"), (_qk, dict(T=-1), "tokens"), (_qk, dict(T=BIG), "tokens"),
    (_qk, dict(hq=-1), "heads_q"), (_qk, dict(hk=65537), "heads_k"), (_qk, dict(q=None), "q or its output"),
    (_qk, dict(ok=None), "k or its output"), (_qk, dict(q=ODD8), "16-byte"), (_qk, dict(ldq=252), "16-byte"),
    (_qk, dict(hsk=68), "16-byte"), (_qk, dict(ldk=-8), "pitches"), (_qk, dict(hsq=BIG), "pitches"), (_qk, dict(oq=ODD8), "16-byte"),
    (_qk, dict(hq=3, hsq=2 ** 30), "span"), (_qk, dict(hq=3, hoq=2 ** 30, loq=2 ** 31), "span"),
    (_qk, dict(loq=32), "below head_dim"), (_qk, dict(hoq=32), "below head_dim"), (_qk, dict(wq=ODD2), "w_q"),
    (_qk, dict(wk=ODD8, wdt=0), "w_k"), (_qk, dict(eps=-1.0), "eps"), (_qk, dict(eps=float("nan")), "eps"),
    (_qk, dict(eps=float("inf")), "eps"), (_qk, dict(cos=None), "cos and sin"), (_qk, dict(sin=ODD8), "cos and sin"),
    (_qk, dict(ldt=28), "ld_table"), (_qk, dict(ldt=34), "ld_table"), (_qk, dict(rows=3), "table_rows"),
    (_qk, dict(rows=-1, pos=OK16), "table_rows"), (_qk, dict(pos=P(0x10004)), "positions"),
    (_qk8, dict(cq=P(0x10004)), "8-byte"), (_qk8, dict(lcq=132), "8-byte"), (_qk8, dict(sq=None), "scales_q"),
    (_qk8, dict(sk=ODD2), "scales_k"), (_qk8, dict(lsq=1), "scales_q"), (_qk8, dict(ck=None), "k or its output"),
    (_qk8, dict(hck=32, lck=32), "below head_dim"),
]


@pytest.mark.parametrize("fn,kw,needle", INVALID)
def test_invalid_arguments_are_rejected(fn, kw, needle):
    assert fn(**kw) == mxq.MXQ_ERR_INVALID_ARG
    assert needle in mxq.lib.mxq_last_error().decode(), mxq.lib.mxq_last_error()


@pytest.mark.parametrize("fn,kw,needle", [
    (_quant, dict(dt=7), "dtype"), (_gemm, dict(dt=7), "dtype"), (_fused, dict(dt=7), "dtype"), (_fused, dict(odt=7), "dtype"),
    (_qk, dict(dt=2), "dtype"), (_qk, dict(wdt=2), "dtype"), (_qk, dict(style=2), "style"), (_qk8, dict(style=5), "style")])
def test_unknown_values_are_unsupported(fn, kw, needle):
    assert fn(**kw) == mxq.MXQ_ERR_UNSUPPORTED and needle in mxq.lib.mxq_last_error().decode()


def test_empty_problems_are_noops():
    assert _quant(x=None, codes=None, scales=None, rows=0) == 0
    assert _dequant(codes=None, scales=None, y=None, rows=0) == 0
    for kw in (dict(M=0), dict(N=0, ldo=0)):
        assert _gemm(a=None, w=None, sa=None, sw=None, out=None, **kw) == 0
        assert _fused(w=None, sw=None, out=None, ws=None, nbytes=0, **kw) == 0
    assert _qk(q=None, k=None, oq=None, ok=None, T=0) == 0
    assert _qk(q=None, k=None, oq=None, ok=None, hq=0, hk=0, cos=None) == 0
    assert mxq.lib.mxq_last_error() == b""


def test_workspace_covers_codes_and_scales():
    for M, N, K in ((300, 64, 128), (4096, 5120, 13824)):
        assert mxq.w8a8_fused_workspace_bytes(M, N, K) >= M * K + 4 * M
    for M, N, K in ((0, 8, 64), (8, 0, 64), (8, 8, 40), (-1, 8, 64), (8, 8, 1 << 17), (8, 8, -16)):
        assert mxq.w8a8_fused_workspace_bytes(M, N, K) == 0 and mxq.w8a8_workspace_bytes(M, N, K) == 0
    # up to 8 tokens whose codes fit the LDS: one launch, no workspace
    for M, N, K in ((1, 64, 15744), (8, 64, 1920), (3, 5120, 5248)):
        assert mxq.w8a8_fused_workspace_bytes(M, N, K) == 0
    for M, N, K in ((1, 64, 15760), (8, 64, 1936), (9, 64, 128)):
        assert mxq.w8a8_fused_workspace_bytes(M, N, K) >= M * K + 4 * M
    assert mxq.w8a8_workspace_bytes(48, 5120, 13824) > 0 and mxq.w8a8_workspace_bytes(4096, 5120, 13824) == 0
    assert mxq.w8a8_fused_workspace_bytes(48, 5120, 13824) >= 48 * 13828 + mxq.w8a8_workspace_bytes(48, 5120, 13824)


# ------------------------------------------------------------------ binding
C8 = lambda *s: torch.zeros(s, dtype=torch.int8)   # noqa: E731


@pytest.mark.parametrize("call", [
    lambda: mxq.quantize_int8(torch.zeros(4, 64, dtype=torch.bfloat16)),
    lambda: mxq.dequantize_int8(C8(4, 64), torch.zeros(4)),
    lambda: mxq.gemm_w8a8(C8(4, 64), torch.zeros(4), C8(8, 64), torch.zeros(8)),
    lambda: mxq.gemm_w8a8_fused(torch.zeros(4, 64), C8(8, 64), torch.zeros(8)),
    lambda: mxq.qk_norm_rope(torch.zeros(4, 2, 64), torch.zeros(4, 1, 64), None, None, None, None),
    lambda: mxq.quantize_qk_norm_rope(torch.zeros(4, 2, 64), torch.zeros(4, 1, 64), None, None, None, None),
])
def test_host_tensors_are_rejected(call):
    with pytest.raises(ValueError, match="GPU tensor"):
        call()


def _fake(monkeypatch):
    """Meta tensors stand in for GPU tensors in the checks; nothing past them may run."""
    monkeypatch.setattr(mxq, "_dev", lambda t, name, device=None: t)
    monkeypatch.setattr(mxq, "_call", lambda *a: pytest.fail("reached the library"))


def _m(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


I8 = torch.int8


@pytest.mark.parametrize("call,needle", [
    (lambda: mxq.quantize_int8(_m(4, 64, dtype=torch.float16)), "x must be"),
    (lambda: mxq.quantize_int8(_m(4)), "2-D"),
    (lambda: mxq.quantize_int8(_m(64, 4).t()), "contiguous rows"),
    (lambda: mxq.quantize_int8(_m(4, 64), codes=_m(4, 64)), "codes must be"),
    (lambda: mxq.quantize_int8(_m(4, 64), codes=_m(4, 32, dtype=I8)), "shape"),
    (lambda: mxq.quantize_int8(_m(4, 64), scales=_m(3)), "scales must have shape"),
    (lambda: mxq.quantize_int8(_m(4, 64), scales=_m(8)[::2]), "contiguous"),
    (lambda: mxq.dequantize_int8(_m(4, 64, dtype=I8), _m(4), out=_m(4, 64)), "out must be"),
    (lambda: mxq.gemm_w8a8(_m(4, 64), _m(4), _m(8, 64, dtype=I8), _m(8)), "a_codes must be"),
    (lambda: mxq.gemm_w8a8(_m(4, 64, dtype=I8), _m(4), _m(8, 32, dtype=I8), _m(8)), "columns"),
    (lambda: mxq.gemm_w8a8(_m(4, 64, dtype=I8), _m(5), _m(8, 64, dtype=I8), _m(8)), "a_scales must have shape"),
    (lambda: mxq.gemm_w8a8(_m(4, 64, dtype=I8), _m(4, dtype=torch.float64), _m(8, 64, dtype=I8), _m(8)), "a_scales must be"),
    (lambda: mxq.gemm_w8a8(_m(4, 64, dtype=I8), _m(4), _m(8, 64, dtype=I8), _m(8), bias=_m(7)), "bias"),
    (lambda: mxq.gemm_w8a8(_m(4, 64, dtype=I8), _m(4), _m(8, 64, dtype=I8), _m(8), out_dtype=torch.float16), "out_dtype"),
    (lambda: mxq.gemm_w8a8(_m(4, 64, dtype=I8), _m(4), _m(8, 64, dtype=I8), _m(8), out=_m(4, 9)), "out must have shape"),
    (lambda: mxq.gemm_w8a8_fused(_m(4, 64, dtype=I8), _m(8, 64, dtype=I8), _m(8)), "a must be"),
    (lambda: mxq.qk_norm_rope(_m(4, 64), _m(4, 1, 64), None, None, None, None), "3-D"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(5, 1, 64), None, None, None, None), "k must have shape"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64, dtype=torch.bfloat16), None, None, None, None), "k must be"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64), _m(32), None, None, None), "q_weight"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64), _m(64, dtype=torch.float16), None, None, None), "q_weight"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64), _m(64), _m(64, dtype=torch.bfloat16), None, None), "one dtype"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64), None, None, _m(4, 32), None), "together"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64), None, None, _m(4, 32), _m(4, 16)), "sin must have shape"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64), None, None, _m(4, 32), _m(4, 64)[:, :32]), "row pitch"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64), None, None, _m(4, 32), _m(4, 32), positions=_m(4)), "positions"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64), None, None, _m(4, 32), _m(4, 32), style="pairs"), "style"),
    (lambda: mxq.qk_norm_rope(_m(4, 2, 64), _m(4, 1, 64), None, None, None, None, out_q=_m(4, 2, 32)), "out_q"),
    (lambda: mxq.qk_norm_rope(_m(4, 64, 2).transpose(1, 2), _m(4, 1, 64), None, None, None, None), "contiguous heads"),
])
def test_binding_refuses_wrong_tensors(monkeypatch, call, needle):
    _fake(monkeypatch)
    with pytest.raises(ValueError, match=needle):
        call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device failure path")
def test_launch_without_gpu_reports_hip_error():
    for fn in (_quant, _dequant, _gemm, _fused, _qk, _qk8):
        assert fn() == mxq.MXQ_ERR_HIP and b"HIP error" in mxq.lib.mxq_last_error()
