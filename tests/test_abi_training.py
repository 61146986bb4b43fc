"""Refusals of the layer norm, activation and weight gradient entry points, decided before anything is launched
(no GPU needed): through the C ABI with pointers that are never dereferenced, and through the binding's
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
F = ctypes.c_float
L = mxq.lib


def _norm(x=OK16, dt=1, T=4, C=64, ld=64, w=OK16, b=OK16, wdt=1, eps=1e-6, y=OK16, ldy=64, mean=OK16, rstd=OK16, xc=None,
          ldxc=0, xs=None):
    return L.mxq_layer_norm(x, dt, T, C, ld, w, b, wdt, F(eps), y, ldy, mean, rstd, xc, ldxc, xs, None)


def _norm8(x=OK16, dt=1, T=4, C=64, ld=64, w=OK16, b=OK16, wdt=1, eps=1e-6, c=OK16, ldc=64, s=OK16, mean=None, rstd=None, xc=None,
           ldxc=0, xs=None):
    return L.mxq_quantize_layer_norm(x, dt, T, C, ld, w, b, wdt, F(eps), c, ldc, s, mean, rstd, xc, ldxc, xs, None)


def _back(dy=OK16, dt=1, T=4, C=64, ld=64, x=OK16, ldx=64, xs=None, mean=OK16, rstd=OK16, w=OK16, wdt=1, dx=OK16, lddx=64, dw=OK16,
          db=OK16, ws=OK16, nbytes=1 << 20):
    return L.mxq_layer_norm_backward(dy, dt, T, C, ld, x, ldx, xs, mean, rstd, w, wdt, dx, lddx, dw, db, ws, nbytes, None)


def _act(u=OK16, dt=1, T=4, C=64, ld=64, act=0, y=OK16, ldy=64, uc=None, lduc=0, us=None):
    return L.mxq_activation(u, dt, T, C, ld, act, y, ldy, uc, lduc, us, None)


def _act8(u=OK16, dt=1, T=4, C=64, ld=64, act=0, c=OK16, ldc=64, s=OK16, uc=None, lduc=0, us=None):
    return L.mxq_quantize_activation(u, dt, T, C, ld, act, c, ldc, s, uc, lduc, us, None)


def _act_back(dy=OK16, dt=1, T=4, C=64, ld=64, uc=OK16, lduc=64, us=OK16, act=0, du=OK16, lddu=64):
    return L.mxq_activation_backward(dy, dt, T, C, ld, uc, lduc, us, act, du, lddu, None)


def _grad(dy=OK16, ldy=64, c=OK16, ldc=32, s=OK16, M=4, N=64, K=32, out=OK16, dt=0, ldo=32, acc=0, ws=OK16, nbytes=1 << 30):
    return L.mxq_grad_weight_int8(dy, ldy, c, ldc, s, M, N, K, out, dt, ldo, acc, ws, nbytes, None)


KEEP = dict(xc=OK16, ldxc=64, xs=OK16)
CKPT = dict(uc=OK16, lduc=64, us=OK16)
BIGGER = dict(M=3584, N=5120, K=5120, ldy=5120, ldc=5120, ldo=5120)   # with a workspace
INVALID = [
    (_norm, dict(C=60, ld=64), "multiple of 8"), (_norm, dict(C=72, ld=72, ldy=72, xc=OK16, ldxc=80, xs=OK16), "multiple of 16"),
    (_norm, dict(C=0), "cols"), (_norm, dict(C=16392, ld=16392, ldy=16392), "cols"), (_norm, dict(T=-1), "negative"),
    (_norm, dict(T=BIG), "2^31"), (_norm, dict(ld=56), "ld_x"), (_norm, dict(ld=68), "aligned"), (_norm, dict(x=ODD8), "aligned"),
    (_norm, dict(x=None), "NULL"), (_norm, dict(y=None), "y is NULL"), (_norm, dict(y=ODD8), "y base"), (_norm, dict(ldy=56), "ld of y"),
    (_norm, dict(ldy=68), "y base"), (_norm, dict(ldy=BIG), "2^32"), (_norm, dict(w=ODD8), "w and b"), (_norm, dict(b=ODD2), "w and b"),
    (_norm, dict(eps=-1e-6), "eps"), (_norm, dict(eps=float("nan")), "eps"), (_norm, dict(eps=float("inf")), "eps"),
    (_norm, dict(mean=None), "together"), (_norm, dict(rstd=None), "together"), (_norm, dict(mean=ODD2), "mean"),
    (_norm, dict(rstd=ODD2), "rstd"), (_norm, KEEP | dict(xc=ODD8), "x_codes"), (_norm, KEEP | dict(ldxc=72), "x_codes"),
    (_norm, KEEP | dict(ldxc=48), "ld of x_codes"), (_norm, KEEP | dict(xs=None), "x_scales"), (_norm, KEEP | dict(xs=ODD2), "x_scales"),
    (_norm, dict(T=2 ** 31 - 1, C=16384, ld=16384, ldy=16384), "too large"),
    (_norm8, dict(C=72, ld=72, ldc=80), "multiple of 16"), (_norm8, dict(c=None), "codes is NULL"), (_norm8, dict(c=ODD8), "codes base"),
    (_norm8, dict(ldc=72), "codes base"), (_norm8, dict(ldc=48), "ld of codes"), (_norm8, dict(s=None), "scales"),
    (_norm8, dict(s=ODD2), "scales"), (_norm8, dict(mean=OK16), "together"), (_norm8, KEEP | dict(xs=None), "x_scales"),
    (_back, dict(C=60), "multiple of 8"), (_back, dict(C=72, ld=72, ldx=80, lddx=72, xs=OK16), "multiple of 16"),
    (_back, dict(C=16392, ld=16392, ldx=16392, lddx=16392), "cols"), (_back, dict(T=NEG), "negative"), (_back, dict(dy=None), "NULL"),
    (_back, dict(dy=ODD8), "aligned"), (_back, dict(ld=60), "ld_x"), (_back, dict(x=None), "x is NULL"), (_back, dict(x=ODD8), "x base"),
    (_back, dict(ldx=56), "ld of x"), (_back, dict(ldx=72, xs=OK16), "x base"), (_back, dict(xs=ODD2), "x_scales"),
    (_back, dict(dx=None), "dx is NULL"), (_back, dict(dx=ODD8), "dx base"), (_back, dict(lddx=68), "dx base"),
    (_back, dict(mean=None), "mean"), (_back, dict(rstd=None), "rstd"), (_back, dict(mean=ODD2), "mean"), (_back, dict(w=ODD8), "w and b"),
    (_back, dict(dw=None), "together"), (_back, dict(db=None), "together"), (_back, dict(dw=ODD8), "dw and db"),
    (_back, dict(db=ODD2), "dw and db"), (_back, dict(T=4096, ws=None), "workspace"), (_back, dict(T=4096, ws=ODD8), "workspace"),
    (_back, dict(T=4096, nbytes=100), "workspace"),
    (_act, dict(C=60), "multiple of 8"), (_act, CKPT | dict(C=72, ld=72, ldy=72, lduc=80), "multiple of 16"),
    (_act, dict(C=65544, ld=65544, ldy=65544), "at most"), (_act, dict(T=-1), "negative"), (_act, dict(u=None), "NULL"),
    (_act, dict(u=ODD8), "aligned"), (_act, dict(ld=56), "ld_x"), (_act, dict(y=None), "y is NULL"), (_act, dict(ldy=60), "ld of y"),
    (_act, dict(ldy=68), "y base"), (_act, CKPT | dict(uc=ODD8), "u_codes"), (_act, CKPT | dict(lduc=48), "u_codes"),
    (_act, CKPT | dict(us=None), "u_scales"), (_act8, dict(C=72, ld=72, ldc=80), "multiple of 16"), (_act8, dict(c=None), "codes is NULL"),
    (_act8, dict(ldc=72), "codes base"), (_act8, dict(s=None), "scales"), (_act8, CKPT | dict(us=ODD2), "u_scales"),
    (_act_back, dict(C=72, ld=72, lduc=80, lddu=72), "multiple of 16"), (_act_back, dict(dy=None), "NULL"), (_act_back, dict(uc=None), "u_codes"),
    (_act_back, dict(uc=ODD8), "u_codes"), (_act_back, dict(lduc=72), "u_codes"), (_act_back, dict(lduc=48), "u_codes"),
    (_act_back, dict(us=None), "u_scales"), (_act_back, dict(du=None), "du is NULL"), (_act_back, dict(lddu=68), "du base"),
    (_act_back, dict(T=BIG), "2^31"), (_act_back, dict(lddu=BIG), "2^32"),
    (_grad, dict(N=60), "N (60)"), (_grad, dict(K=24), "K (24)"), (_grad, dict(M=-1), "negative"), (_grad, dict(M=BIG), "too large"),
    (_grad, dict(N=2 ** 23, ldy=2 ** 23 - 8), "too large"), (_grad, dict(K=2 ** 23, ldc=2 ** 23, ldo=2 ** 23), "too large"),
    (_grad, dict(N=2 ** 20, K=2 ** 20), "too large"), (_grad, dict(ldy=2 ** 23), "ld of dy"), (_grad, dict(ldy=56), "ld of dy"),
    (_grad, dict(ldy=68), "dy base"), (_grad, dict(dy=ODD8), "dy base"), (_grad, dict(dy=None), "dy is NULL"), (_grad, dict(c=None), "codes is NULL"),
    (_grad, dict(c=ODD8), "codes base"), (_grad, dict(ldc=40), "codes base"), (_grad, dict(ldc=16), "ld of codes"), (_grad, dict(ldc=2 ** 23), "ld of codes"), (_grad, dict(s=None), "scales"),
    (_grad, dict(s=ODD2), "scales"), (_grad, dict(out=None), "out is NULL"), (_grad, dict(out=ODD2), "out base"), (_grad, dict(ldo=31), "ld of out"),
    (_grad, dict(ldo=BIG), "2^32"), (_grad, BIGGER | dict(ws=None), "workspace"), (_grad, BIGGER | dict(ws=ODD8), "workspace"), (_grad, BIGGER | dict(nbytes=16), "workspace"),
]


@pytest.mark.parametrize("fn,kw,needle", INVALID)
def test_invalid_arguments_are_rejected(fn, kw, needle):
    assert fn(**kw) == mxq.MXQ_ERR_INVALID_ARG
    assert needle in L.mxq_last_error().decode(), L.mxq_last_error()


@pytest.mark.parametrize("fn,kw,needle", [
    (_norm, dict(dt=7), "dtype"), (_norm, dict(wdt=3), "dtype"), (_norm8, dict(dt=2), "dtype"), (_back, dict(dt=2), "dtype"),
    (_back, dict(wdt=2), "dtype"), (_act, dict(dt=2), "dtype"), (_act, dict(act=2), "activation"), (_act8, dict(act=-1), "activation"),
    (_act_back, dict(act=9), "activation"), (_act_back, dict(dt=5), "dtype"), (_grad, dict(dt=2), "dtype")])
def test_unknown_values_are_unsupported(fn, kw, needle):
    assert fn(**kw) == mxq.MXQ_ERR_UNSUPPORTED and needle in L.mxq_last_error().decode()


def test_empty_problems_are_noops():
    assert _norm(x=None, y=None, mean=None, rstd=None, T=0) == 0
    assert _norm8(x=None, c=None, s=None, T=0) == 0
    assert _back(dy=None, x=None, dx=None, mean=None, rstd=None, dw=None, db=None, ws=None, nbytes=0, T=0) == 0
    assert _act(u=None, y=None, T=0) == 0 and _act8(u=None, c=None, s=None, T=0) == 0
    assert _act_back(dy=None, uc=None, us=None, du=None, T=0) == 0
    assert _grad(dy=None, ldy=0, out=None, N=0, ws=None, nbytes=0) == 0
    assert _grad(c=None, ldc=0, out=None, ldo=0, K=0, ws=None, nbytes=0) == 0
    assert _grad(dy=None, c=None, s=None, M=0, acc=1, ws=None, nbytes=0) == 0
    assert L.mxq_last_error() == b""


def test_workspace_sizes():
    back, grad = L.mxq_layer_norm_backward_workspace_bytes, L.mxq_grad_weight_int8_workspace_bytes
    for T, C in ((0, 64), (-1, 64), (4, 60), (4, 0), (4, 16392), (2 ** 31, 64)):
        assert back(T, C) == 0
    assert back(1, 5120) == 0 and back(75600, 5120) > 0 and back(75600, 5120) < 75600 * 5120
    for M, N, K in ((-1, 8, 16), (4, 0, 16), (4, 8, 0), (4, 12, 16), (4, 8, 24), (2 ** 31, 8, 16), (4, 2 ** 23, 16)):
        assert grad(M, N, K) == 0
    assert grad(0, 8, 16) == 0 and grad(64, 64, 64) == 0
    assert grad(3584, 5120, 5120) >= 3584 * 5120 * 2


# ------------------------------------------------------------------ binding
I8, B16 = torch.int8, torch.bfloat16


@pytest.mark.parametrize("call", [
    lambda: mxq.layer_norm(torch.zeros(4, 64)), lambda: mxq.quantize_layer_norm(torch.zeros(4, 64)),
    lambda: mxq.layer_norm_backward(torch.zeros(4, 64), torch.zeros(4, 64), torch.zeros(4), torch.zeros(4)),
    lambda: mxq.activation(torch.zeros(4, 64)), lambda: mxq.quantize_activation(torch.zeros(4, 64)),
    lambda: mxq.activation_backward(torch.zeros(4, 64), torch.zeros(4, 64, dtype=I8), torch.zeros(4)),
    lambda: mxq.grad_weight_int8(torch.zeros(4, 64, dtype=B16), torch.zeros(4, 64, dtype=I8), torch.zeros(4)),
])
def test_host_tensors_are_rejected(call):
    with pytest.raises(ValueError, match="GPU tensor"):
        call()


def _m(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call,needle", [
    (lambda: mxq.layer_norm(_m(4, 64, dtype=torch.float16)), "x must be"),
    (lambda: mxq.layer_norm(_m(64)), "2-D"),
    (lambda: mxq.layer_norm(_m(64, 4).t()), "contiguous rows"),
    (lambda: mxq.layer_norm(_m(4, 64), _m(32)), "weight"),
    (lambda: mxq.layer_norm(_m(4, 64), _m(128)[::2]), "weight"),
    (lambda: mxq.layer_norm(_m(4, 64), None, _m(64, dtype=torch.float64)), "bias"),
    (lambda: mxq.layer_norm(_m(4, 64), _m(64), _m(64, dtype=B16)), "one dtype"),
    (lambda: mxq.layer_norm(_m(4, 64), save="bf16"), "save"),
    (lambda: mxq.layer_norm(_m(4, 64), out=_m(4, 32)), "out must have shape"),
    (lambda: mxq.layer_norm(_m(4, 64), out=_m(4, 64, dtype=B16)), "out must be"),
    (lambda: mxq.quantize_layer_norm(_m(4, 64), save="codes"), "save"),
    (lambda: mxq.layer_norm_backward(_m(4, 64), _m(4, 64, dtype=B16), _m(4), _m(4)), "x must be"),
    (lambda: mxq.layer_norm_backward(_m(4, 64), _m(4, 64, dtype=I8), _m(4), _m(4)), "x must be"),
    (lambda: mxq.layer_norm_backward(_m(4, 64), _m(4, 64), _m(4), _m(4), x_scales=_m(4)), "x must be"),
    (lambda: mxq.layer_norm_backward(_m(4, 64), _m(4, 64, dtype=I8), _m(4), _m(4), x_scales=_m(5)), "x_scales"),
    (lambda: mxq.layer_norm_backward(_m(4, 64), _m(5, 64), _m(4), _m(4)), "x must have shape"),
    (lambda: mxq.layer_norm_backward(_m(4, 64), _m(4, 64), _m(4, 1), _m(4)), "mean"),
    (lambda: mxq.layer_norm_backward(_m(4, 64), _m(4, 64), _m(4), _m(8)[::2]), "rstd"),
    (lambda: mxq.layer_norm_backward(_m(4, 64), _m(4, 64), _m(4), _m(4), _m(63)), "weight"),
    (lambda: mxq.layer_norm_backward(_m(4, 64), _m(4, 64), _m(4), _m(4), out=_m(4, 64, dtype=B16)), "out must be"),
    (lambda: mxq.activation(_m(4, 64), "relu"), "act must be"),
    (lambda: mxq.activation(_m(4, 64), save="x"), "save"),
    (lambda: mxq.activation(_m(4, 64), out=_m(5, 64)), "out must have shape"),
    (lambda: mxq.quantize_activation(_m(4, 64, dtype=I8)), "u must be"),
    (lambda: mxq.quantize_activation(_m(4, 64), "gelu"), "act must be"),
    (lambda: mxq.activation_backward(_m(4, 64), _m(4, 64), _m(4)), "u_codes"),
    (lambda: mxq.activation_backward(_m(4, 64), _m(4, 32, dtype=I8), _m(4)), "u_codes"),
    (lambda: mxq.activation_backward(_m(4, 64), _m(4, 64, dtype=I8), _m(4, dtype=torch.float64)), "u_scales"),
    (lambda: mxq.activation_backward(_m(4, 64), _m(4, 64, dtype=I8), _m(4), act="tanh"), "act must be"),
    (lambda: mxq.grad_weight_int8(_m(4, 64), _m(4, 32, dtype=I8), _m(4)), "dy must be"),
    (lambda: mxq.grad_weight_int8(_m(4, 64, dtype=B16), _m(4, 32), _m(4)), "codes must be"),
    (lambda: mxq.grad_weight_int8(_m(4, 64, dtype=B16), _m(5, 32, dtype=I8), _m(4)), "rows"),
    (lambda: mxq.grad_weight_int8(_m(4, 64, dtype=B16), _m(4, 32, dtype=I8), _m(5)), "scales"),
    (lambda: mxq.grad_weight_int8(_m(4, 64, dtype=B16), _m(4, 32, dtype=I8), _m(4), out_dtype=torch.float16), "out_dtype"),
    (lambda: mxq.grad_weight_int8(_m(4, 64, dtype=B16), _m(4, 32, dtype=I8), _m(4), accumulate=True), "accumulate"),
    (lambda: mxq.grad_weight_int8(_m(4, 64, dtype=B16), _m(4, 32, dtype=I8), _m(4), out=_m(32, 64)), "out must have shape"),
])
def test_binding_refuses_wrong_tensors(monkeypatch, call, needle):
    """Meta tensors stand in for GPU tensors in the checks; nothing past them may run."""
    monkeypatch.setattr(mxq, "_dev", lambda t, name, device=None: t)
    monkeypatch.setattr(mxq, "_call", lambda *a: pytest.fail("reached the library"))
    with pytest.raises(ValueError, match=needle):
        call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device failure path")
def test_launch_without_gpu_reports_hip_error():
    for fn in (_norm, _norm8, _back, _act, _act8, _act_back, _grad):
        assert fn() == mxq.MXQ_ERR_HIP and b"HIP error" in L.mxq_last_error()
