"""Python binding of libmxq (OCP MXFP4 quantization + W4A4 / W4A8 GEMMs for MI355X).

The functions here only marshal arguments: they check every tensor's device, dtype and
shape (inputs and caller-supplied output or scratch buffers, ``check_buffer``), allocate
outputs with torch (device memory) and call the C ABI declared in
``include/mxq.h`` on torch's current HIP stream.  Every step of the computation runs in
the library's gfx950 kernels.  Importing fails loudly if ``libmxq.so`` has not been
built (``python mxfp4_microscaled_quantization_amd/build.py``); there is no fallback.

Function names mirror the C entry points without the ``mxq_`` prefix:
``quantize``, ``quantize_fp8``, ``absmax``, ``gemm_w4a4``, ``gemm_w4a4_fused``, ``gemm_w4a8``, ``gemm_bf16``,
``sqnr``, ``dequantize``, ``dequantize_fp8``, ``fp8_static_scales``, ``quantize_int8``, ``dequantize_int8``, ``gemm_w8a8``,
``gemm_w8a8_fused``, ``qk_norm_rope``, ``quantize_qk_norm_rope``, ``layer_norm``, ``quantize_layer_norm``,
``layer_norm_backward``, ``activation``, ``quantize_activation``, ``activation_backward``, ``grad_weight_int8``.  ``lib`` exposes the raw ctypes functions.
"""

import ctypes
import os

import torch

__all__ = [
    "lib", "MxqError", "quantize", "quantize_into", "quantize_hadamard", "SCALE_RULES", "quantize_fp8", "absmax", "fp8_static_scales",
    "gemm_w4a4", "gemm_w4a4_fused", "gemm_w4a8", "gemm_bf16", "sqnr", "sqnr_noalloc", "sqnr_workspace_bytes", "dequantize", "dequantize_fp8",
    "quantize_int8", "dequantize_int8", "gemm_w8a8", "gemm_w8a8_fused", "w8a8_workspace_bytes",
    "w8a8_fused_workspace_bytes",
    "qk_norm_rope", "quantize_qk_norm_rope", "ROPE_STYLES", "layer_norm", "quantize_layer_norm", "layer_norm_backward",
    "activation", "quantize_activation", "activation_backward", "ACTIVATIONS", "grad_weight_int8", "mfma_ceiling", "MFMA_FLOP", "check_buffer",
    "LIB_PATH", "ABI_SYMBOLS", "ABI_VERSION",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxq.so")

#: MXQ_ABI_VERSION of include/mxq.h that the signatures below describe
ABI_VERSION = 2

MXQ_OK, MXQ_ERR_INVALID_ARG, MXQ_ERR_UNSUPPORTED, MXQ_ERR_HIP = 0, 1, 2, 3
MXQ_F32, MXQ_BF16 = 0, 1

_i64, _ptr, _f32, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t

# q and k (pointer, heads, pitches), dt, tokens, head_dim, weights, w_dt, eps, tables, rot_dim, positions, style
_QK_ARGS = [_ptr, _i64, _i64, _i64, _ptr, _i64, _i64, _i64, ctypes.c_int, _i64, _i64, _ptr, _ptr, ctypes.c_int, _f32,
            _ptr, _ptr, _i64, _i64, _i64, _ptr, ctypes.c_int]

#: every exported symbol with (restype, argtypes) -- the C ABI of include/mxq.h
_NORM_ARGS = [_ptr, ctypes.c_int, _i64, _i64, _i64, _ptr, _ptr, ctypes.c_int, _f32]
_NORM_SAVED = [_ptr, _ptr, _ptr, _i64, _ptr]

ABI_SYMBOLS = {
    "mxq_quantize": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, _ptr, _i64, _ptr, _i64, _ptr]),
    "mxq_quantize_rule": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, _ptr, _i64, _ptr, _i64, ctypes.c_int,
                                         _ptr]),
    "mxq_quantize_hadamard": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _ptr,
                                             _i64, _ptr, _i64, _ptr]),
    "mxq_quantize_fp8": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, _f32, _ptr, _i64, _ptr]),
    "mxq_absmax": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, _ptr, _ptr]),
    "mxq_gemm_w4a4": (ctypes.c_int, [_ptr, _ptr, _ptr, _ptr, _i64, _i64, _i64, _ptr, _i64, _ptr]),
    "mxq_gemm_w4a4_fused": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _ptr, _ptr, _i64, _i64, _i64, ctypes.c_int, _ptr,
                                           _i64, _ptr, _sz, _ptr]),
    "mxq_gemm_w4a4_fused_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mxq_gemm_w4a8": (ctypes.c_int, [_ptr, _f32, _ptr, _ptr, _i64, _i64, _i64, _ptr, _i64, _ptr]),
    "mxq_gemm_bf16": (ctypes.c_int, [_ptr, _ptr, _i64, _i64, _i64, _ptr, _i64, _ptr]),
    "mxq_sqnr_workspace_bytes": (_sz, [_i64]),
    "mxq_sqnr": (ctypes.c_int, [_ptr, _ptr, _i64, _i64, _i64, _i64, _ptr, _sz, _ptr, _ptr]),
    "mxq_sqnr_noalloc": (ctypes.c_int, [_ptr, _ptr, _i64, _i64, _i64, _i64, _ptr, _ptr]),
    "mxq_dequantize": (ctypes.c_int, [_ptr, _i64, _ptr, _i64, _i64, _i64, _ptr, _i64, _ptr]),
    "mxq_dequantize_fp8": (ctypes.c_int, [_ptr, _i64, _f32, _i64, _i64, _ptr, _i64, _ptr]),
    "mxq_fp8_static_scales": (ctypes.c_int, [_f32, ctypes.POINTER(_f32), ctypes.POINTER(_f32)]),
    "mxq_mfma_ceiling": (ctypes.c_int, [ctypes.c_int, _ptr, _ptr, _ptr, _ptr, _i64, _i64, _i64, _i64, _i64, _ptr,
                                        _ptr]),
    "mxq_quantize_int8": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, _ptr, _i64, _ptr, _ptr]),
    "mxq_dequantize_int8": (ctypes.c_int, [_ptr, _i64, _ptr, _i64, _i64, _ptr, _i64, _ptr]),
    "mxq_gemm_w8a8": (ctypes.c_int, [_ptr, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _i64, _i64, _ptr,
                                     ctypes.c_int, _i64, _ptr, _sz, _ptr]),
    "mxq_gemm_w8a8_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mxq_gemm_w8a8_fused": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _i64, _i64,
                                           _ptr, ctypes.c_int, _i64, _ptr, _sz, _ptr]),
    "mxq_gemm_w8a8_fused_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mxq_qk_norm_rope": (ctypes.c_int, _QK_ARGS + [_ptr, _i64, _i64, _ptr, _i64, _i64, _ptr]),
    "mxq_quantize_qk_norm_rope": (ctypes.c_int, _QK_ARGS + [_ptr, _i64, _i64, _ptr, _i64] * 2 + [_ptr]),
    "mxq_layer_norm": (ctypes.c_int, _NORM_ARGS + [_ptr, _i64] + _NORM_SAVED + [_ptr]),
    "mxq_quantize_layer_norm": (ctypes.c_int, _NORM_ARGS + [_ptr, _i64, _ptr] + _NORM_SAVED + [_ptr]),
    "mxq_layer_norm_backward_workspace_bytes": (_sz, [_i64, _i64]),
    "mxq_layer_norm_backward": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, _ptr, _i64, _ptr, _ptr, _ptr, _ptr,
                                               ctypes.c_int, _ptr, _i64, _ptr, _ptr, _ptr, _sz, _ptr]),
    "mxq_activation": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, ctypes.c_int, _ptr, _i64, _ptr, _i64, _ptr,
                                      _ptr]),
    "mxq_quantize_activation": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, ctypes.c_int, _ptr, _i64, _ptr, _ptr,
                                               _i64, _ptr, _ptr]),
    "mxq_activation_backward": (ctypes.c_int, [_ptr, ctypes.c_int, _i64, _i64, _i64, _ptr, _i64, _ptr, ctypes.c_int, _ptr,
                                               _i64, _ptr]),
    "mxq_grad_weight_int8": (ctypes.c_int, [_ptr, _i64, _ptr, _i64, _ptr, _i64, _i64, _i64, _ptr, ctypes.c_int, _i64,
                                            ctypes.c_int, _ptr, _sz, _ptr]),
    "mxq_grad_weight_int8_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mxq_last_error": (ctypes.c_char_p, []),
    "mxq_abi_version": (ctypes.c_int, []),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libmxq.so not found at {LIB_PATH}; build it with "
            "`python mxfp4_microscaled_quantization_amd/build.py` (hipcc, gfx950)")
    handle = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in ABI_SYMBOLS.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    found = handle.mxq_abi_version()
    if found != ABI_VERSION:
        raise ImportError(f"{LIB_PATH} reports ABI version {found}, this binding expects {ABI_VERSION}: "
                          "rebuild it with `python mxfp4_microscaled_quantization_amd/build.py`")
    return handle


lib = _load()


class MxqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[mxq status {status}] {message}")
        self.status = status


def _check(status: int):
    if status != MXQ_OK:
        raise MxqError(status, lib.mxq_last_error().decode(errors="replace"))


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(t, name: str, device=None):
    """``t`` must be a GPU tensor (on ``device`` when given)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _rowmajor(t: torch.Tensor, name: str):
    """2-D tensor with unit column stride; returns its row pitch in elements."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))


def check_buffer(t, name: str, dtype, shape=None, device=None, contiguous=False, min_numel=None, is_gpu=None):
    """Validate a tensor the caller hands to the library (input or output buffer).

    Checks, in order, raising ValueError before anything reaches the C ABI: a tensor;
    on a GPU (``is_gpu``, default the ``is_cuda`` test) and on ``device`` when given;
    ``dtype``; ``shape`` (a tuple, for a 2-D buffer with contiguous rows) or
    ``min_numel`` (for a flat contiguous buffer); fully contiguous when ``contiguous``.
    Returns the row pitch in elements for 2-D buffers, else None.  A pure function of
    tensor metadata, so it is unit-tested on CPU / meta tensors (``is_gpu`` lets a test
    stand those in for device tensors).
    """
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    gpu = t.is_cuda if is_gpu is None else is_gpu(t)
    if not gpu:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if min_numel is not None:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.numel() < min_numel:
            raise ValueError(f"{name} needs at least {min_numel} elements (got {t.numel()})")
        return None
    if shape is not None:
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
        return _rowmajor(t, name)
    return None


def _dtype_code(t: torch.Tensor):
    if t.dtype == torch.bfloat16:
        return MXQ_BF16
    if t.dtype == torch.float32:
        return MXQ_F32
    raise ValueError("input must be bfloat16 or float32")


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


SCALE_RULES = {"ocp": 0, "uos": 1}


def _rule_code(rule: str) -> int:
    if rule not in SCALE_RULES:
        raise ValueError(f"scale rule must be one of {sorted(SCALE_RULES)}")
    return SCALE_RULES[rule]


def _input(x, name="x"):
    """A bf16 / binary32 2-D GPU input with contiguous rows: (row pitch, dtype code)."""
    _dev(x, name)
    code = _dtype_code(x)
    return _rowmajor(x, name), code


def _mx_outputs(x, R, K, codes, scales):
    if codes is None:
        codes = torch.empty((R, K // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((R, K // 32), dtype=torch.uint8, device=x.device)
    ldc = check_buffer(codes, "codes", torch.uint8, (R, K // 2), x.device)
    lds = check_buffer(scales, "scales", torch.uint8, (R, K // 32), x.device)
    return codes, ldc, scales, lds


def quantize(x: torch.Tensor, rule: str = "ocp"):
    """MXFP4-quantize rows of ``x`` (bf16 or fp32, [R, K], K % 32 == 0).

    ``rule``: "ocp" (X = 2^(floor(log2 amax) - 2)) or "uos" (smallest power of two with
    amax <= 7.25 X).  Returns (codes uint8 [R, K/2], scales uint8 [R, K/32]).
    """
    ld, dt = _input(x)
    R, K = x.shape
    codes, ldc, scales, lds = _mx_outputs(x, R, K, None, None)
    _check(lib.mxq_quantize_rule(_p(x), dt, R, K, ld, _p(codes), ldc, _p(scales), lds, _rule_code(rule), _stream()))
    return codes, scales


def quantize_into(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, rule: str = "ocp"):
    """MXFP4-quantize into caller-provided outputs: codes uint8 [R, K/2] and scales uint8
    [R, K/32] on x's device (rows may be strided views)."""
    ld, dt = _input(x)
    R, K = x.shape
    codes, ldc, scales, lds = _mx_outputs(x, R, K, codes, scales)
    _check(lib.mxq_quantize_rule(_p(x), dt, R, K, ld, _p(codes), ldc, _p(scales), lds, _rule_code(rule), _stream()))


def quantize_hadamard(x: torch.Tensor, block_n: int = 64, rule: str = "ocp"):
    """Rotate runs of ``block_n`` (16, 64, 256) elements of each row by H / sqrt(block_n)
    (Sylvester Hadamard, binary32 butterfly), then MXFP4-quantize.  Returns (codes, scales)."""
    ld, dt = _input(x)
    R, K = x.shape
    codes, ldc, scales, lds = _mx_outputs(x, R, K, None, None)
    _check(lib.mxq_quantize_hadamard(_p(x), dt, R, K, ld, int(block_n), _rule_code(rule), _p(codes), ldc,
                                     _p(scales), lds, _stream()))
    return codes, scales


def fp8_static_scales(amax: float):
    """(s_a, inv_s) for a per-tensor absolute maximum, formed by the library
    (mxq_fp8_static_scales): fl32(amax / 448) and fl32(448 / amax)."""
    s_a, inv_s = _f32(), _f32()
    _check(lib.mxq_fp8_static_scales(float(amax), ctypes.byref(s_a), ctypes.byref(inv_s)))
    return float(s_a.value), float(inv_s.value)


def quantize_fp8(x: torch.Tensor, inv_scale: float, out=None) -> torch.Tensor:
    """Static FP8 E4M3: q = E4M3(fl32(x * inv_scale)), saturating; returns uint8 [R, K]."""
    ld, dt = _input(x)
    R, K = x.shape
    q = torch.empty((R, K), dtype=torch.uint8, device=x.device) if out is None else out
    ldq = check_buffer(q, "out", torch.uint8, (R, K), x.device)
    _check(lib.mxq_quantize_fp8(_p(x), dt, R, K, ld, float(inv_scale), _p(q), ldq, _stream()))
    return q


def absmax(x: torch.Tensor) -> torch.Tensor:
    """max |x| as a 1-element float32 GPU tensor."""
    ld, dt = _input(x)
    R, K = x.shape
    out = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib.mxq_absmax(_p(x), dt, R, K, ld, _p(out), _stream()))
    return out


def _out(M, N, device, out):
    if out is None:
        return torch.empty((M, N), dtype=torch.bfloat16, device=device), N
    return out, check_buffer(out, "out", torch.bfloat16, (M, N), device)


def _contig(t, name, dtype, device=None, shape=None):
    check_buffer(t, name, dtype, device=device, contiguous=True)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    return t


def _2d(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return t


def _mx_weights(w_codes, w_scales, K, device):
    _2d(w_codes, "w_codes")
    N = w_codes.shape[0]
    _contig(w_codes, "w_codes", torch.uint8, device, (N, K // 2))
    _contig(w_scales, "w_scales", torch.uint8, device, (N, K // 32))
    return N


def gemm_w4a4(a_codes, a_scales, w_codes, w_scales, out=None):
    """W4A4: MXFP4 A [M, K] x MXFP4 W [N, K]^T -> bf16 [M, N]."""
    _2d(a_codes, "a_codes")
    _contig(a_codes, "a_codes", torch.uint8)
    dev = a_codes.device
    M, K = a_codes.shape[0], a_codes.shape[1] * 2
    _contig(a_scales, "a_scales", torch.uint8, dev, (M, K // 32))
    N = _mx_weights(w_codes, w_scales, K, dev)
    out, ld = _out(M, N, dev, out)
    _check(lib.mxq_gemm_w4a4(_p(a_codes), _p(a_scales), _p(w_codes), _p(w_scales), M, N, K, _p(out), ld, _stream()))
    return out


def fused_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes with which gemm_w4a4_fused takes the separate-quantization route
    (0 where the fused kernel is the faster)."""
    return int(lib.mxq_gemm_w4a4_fused_workspace_bytes(M, N, K))


def gemm_w4a4_fused(a, w_codes, w_scales, rule: str = "ocp", out=None, route: bool = True):
    """W4A4 with the activation quantization fused in: bf16 or fp32 A [M, K] (rows may be
    strided) x MXFP4 W [N, K]^T -> bf16 [M, N]; equal to gemm_w4a4(*quantize(a, rule), W).
    route=True lends the call a workspace, so shapes past the fused kernel's break-even
    quantize in a pass of their own; route=False always runs the fused kernel."""
    ld, dt = _input(a, "a")
    M, K = a.shape
    N = _mx_weights(w_codes, w_scales, K, a.device)
    out, ldo = _out(M, N, a.device, out)
    nbytes = fused_workspace_bytes(M, N, K) if route else 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=a.device) if nbytes else None
    _check(lib.mxq_gemm_w4a4_fused(_p(a), dt, ld, _p(w_codes), _p(w_scales), M, N, K, _rule_code(rule),
                                   _p(out), ldo, _p(ws) if ws is not None else None, nbytes, _stream()))
    return out


def gemm_w4a8(a_fp8, a_scale: float, w_codes, w_scales, out=None):
    """W4A8: FP8 E4M3 A [M, K] (dequant scale a_scale) x MXFP4 W [N, K]^T -> bf16 [M, N]."""
    _2d(a_fp8, "a_fp8")
    _contig(a_fp8, "a_fp8", torch.uint8)
    dev = a_fp8.device
    M, K = a_fp8.shape
    N = _mx_weights(w_codes, w_scales, K, dev)
    out, ld = _out(M, N, dev, out)
    _check(lib.mxq_gemm_w4a8(_p(a_fp8), float(a_scale), _p(w_codes), _p(w_scales), M, N, K, _p(out), ld, _stream()))
    return out


def gemm_bf16(a, w, out=None):
    """bf16 reference: A [M, K] x W [N, K]^T -> bf16 [M, N], fp32 accumulation."""
    _2d(a, "a")
    _2d(w, "w")
    _contig(a, "a", torch.bfloat16)
    M, K = a.shape
    N = w.shape[0]
    _contig(w, "w", torch.bfloat16, a.device, (N, K))
    out, ld = _out(M, N, a.device, out)
    _check(lib.mxq_gemm_bf16(_p(a), _p(w), M, N, K, _p(out), ld, _stream()))
    return out


#: MFMA instruction FLOP per mode, as mxq_mfma_ceiling runs them
MFMA_FLOP = {"w4a4": 2 * 32 * 32 * 64, "w4a8": 2 * 32 * 32 * 64, "bf16": 2 * 16 * 16 * 32}
_GEMM_MODES = {"w4a4": 0, "w4a8": 1, "bf16": 2}


def mfma_ceiling(mode: str, a, a_scales, w, w_scales, waves: int, iters: int, sink=None) -> int:
    """Enqueue the register-only MFMA loop of mxq_mfma_ceiling on the operand planes of a
    GEMM call (``mode`` "w4a4", "w4a8" or "bf16"; operands as for that GEMM, unused scales
    None) on the current stream; returns the FLOP it performs."""
    if mode not in _GEMM_MODES:
        raise ValueError(f"mode must be one of {sorted(_GEMM_MODES)}")
    _2d(a, "a")
    _2d(w, "w")
    if mode == "bf16":
        _contig(a, "a", torch.bfloat16)
        M, K = a.shape
        _contig(w, "w", torch.bfloat16, a.device, (w.shape[0], K))
    else:
        _contig(a, "a", torch.uint8)
        M = a.shape[0]
        K = a.shape[1] * (2 if mode == "w4a4" else 1)
        _mx_weights(w, w_scales, K, a.device)
        if mode == "w4a4":
            _contig(a_scales, "a_scales", torch.uint8, a.device, (M, K // 32))
    N = w.shape[0]
    if sink is None:
        sink = torch.empty(waves * 64, dtype=torch.float32, device=a.device)
    check_buffer(sink, "sink", torch.float32, device=a.device, min_numel=waves * 64)
    _check(lib.mxq_mfma_ceiling(_GEMM_MODES[mode], _p(a), _p(a_scales) if a_scales is not None else None, _p(w),
                                _p(w_scales) if w_scales is not None else None, M, N, K, waves, iters, _p(sink),
                                _stream()))
    return waves * iters * 16 * MFMA_FLOP[mode]


def sqnr_workspace_bytes(n: int) -> int:
    return int(lib.mxq_sqnr_workspace_bytes(n))


def sqnr(ref, test, workspace=None, out3=None) -> torch.Tensor:
    """Whole-output SQNR; returns a float64 GPU tensor [S, N, dB]."""
    _2d(ref, "ref")
    check_buffer(ref, "ref", torch.bfloat16)
    ldr = _rowmajor(ref, "ref")
    R, C = ref.shape
    ldt = check_buffer(test, "test", torch.bfloat16, (R, C), ref.device)
    nbytes = sqnr_workspace_bytes(R * C)
    if workspace is None:
        workspace = torch.empty(nbytes // 8, dtype=torch.float64, device=ref.device)
    check_buffer(workspace, "workspace", torch.float64, device=ref.device, min_numel=nbytes // 8)
    if out3 is None:
        out3 = torch.empty(3, dtype=torch.float64, device=ref.device)
    check_buffer(out3, "out3", torch.float64, device=ref.device, min_numel=3)
    _check(lib.mxq_sqnr(_p(ref), _p(test), R, C, ldr, ldt, _p(workspace),
                        workspace.numel() * workspace.element_size(), _p(out3), _stream()))
    return out3


def sqnr_noalloc(ref, test, out3) -> torch.Tensor:
    """Whole-output SQNR into ``out3`` (float64 [3] on ref's device) with the library's
    own per-GPU workspace (mxq_sqnr_noalloc), for callers that cannot allocate device
    memory.  Calls on one GPU must not overlap."""
    _2d(ref, "ref")
    check_buffer(ref, "ref", torch.bfloat16)
    ldr = _rowmajor(ref, "ref")
    R, C = ref.shape
    ldt = check_buffer(test, "test", torch.bfloat16, (R, C), ref.device)
    check_buffer(out3, "out3", torch.float64, device=ref.device, min_numel=3)
    _check(lib.mxq_sqnr_noalloc(_p(ref), _p(test), R, C, ldr, ldt, _p(out3), _stream()))
    return out3


def dequantize(codes, scales, K: int, out=None) -> torch.Tensor:
    """MXFP4 -> bf16 [R, K] (into ``out`` if given: bfloat16 [R, K], rows may be strided)."""
    _2d(codes, "codes")
    R = codes.shape[0]
    ldc = check_buffer(codes, "codes", torch.uint8, (R, K // 2))
    lds = check_buffer(scales, "scales", torch.uint8, (R, K // 32), codes.device)
    if out is None:
        out = torch.empty((R, K), dtype=torch.bfloat16, device=codes.device)
    ld = check_buffer(out, "out", torch.bfloat16, (R, K), codes.device)
    _check(lib.mxq_dequantize(_p(codes), ldc, _p(scales), lds, R, K, _p(out), ld, _stream()))
    return out


def dequantize_fp8(q, a_scale: float, out=None) -> torch.Tensor:
    """FP8 E4M3 [R, K] -> bf16 [R, K]: bf16(fl32(e4m3(q) * a_scale)) (into ``out`` if given)."""
    _2d(q, "q")
    R, K = q.shape
    ldq = check_buffer(q, "q", torch.uint8, (R, K))
    if out is None:
        out = torch.empty((R, K), dtype=torch.bfloat16, device=q.device)
    ld = check_buffer(out, "out", torch.bfloat16, (R, K), q.device)
    _check(lib.mxq_dequantize_fp8(_p(q), ldq, float(a_scale), R, K, _p(out), ld, _stream()))
    return out


# ---------------------------------------------------------------------------------
# 8-bit integers.  These entry points launch on the tensors' own device, whichever is current.

# the raw stream handle without building a Stream object (2 us of the 10 us of a small call); None without a GPU build
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# torch.cuda.current_device without its check that CUDA is initialized: the tensors are there
_current_device = getattr(torch._C, "_cuda_getDevice", None)
# allocations by explicit strides take 1.3 us, by shape alone 1.7
_empty = torch.empty_strided


def _there(t, name, device):
    """_dev, in fewer steps for a plain tensor on the device of one that _dev has seen."""
    if device is None or type(t) is not torch.Tensor or t.device != device:
        _dev(t, name, device)


def _call(fn, device, *args):
    """``fn(*args, stream)`` with torch's current stream of ``device``, checked."""
    index = device.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status != MXQ_OK:
        _check(status)


def _matrix(t, name, dtype, device=None, shape=None):
    """A 2-D GPU tensor of ``dtype`` (or one of several) with contiguous rows: its row pitch."""
    _there(t, name, device)
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    rows, cols = t.shape
    pitch, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return pitch if rows > 1 else cols


def _vector(t, name, n, device, dtype=torch.float32):
    """A 1-D GPU tensor of ``n`` elements: the distance between them (0 for an expanded one)."""
    _there(t, name, device)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape ({n},) (got {tuple(t.shape)})")
    return t.stride(0) if n > 1 else 1


def _flat(t, name, n, device, dtype=torch.float32):
    if _vector(t, name, n, device, dtype) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t


def _opt(t):
    return None if t is None else t.data_ptr()


_FLOATS = (torch.bfloat16, torch.float32)


def quantize_int8(x, codes=None, scales=None):
    """Symmetric 8-bit codes of the rows of ``x`` (bf16 or fp32 [R, K], K % 16 == 0) with one scale for each:
    s = fl32(amax / 127), q = RNE(fl32(x * fl32(127 / amax))).  For activations the rows are tokens, for weights
    output channels.  Returns (codes int8 [R, K], scales float32 [R]), the ones given where they are."""
    ld = _matrix(x, "x", _FLOATS)
    R, K = x.shape
    if codes is None:
        codes, ldc = _empty((R, K), (K, 1), dtype=torch.int8, device=x.device), K
    else:
        ldc = _matrix(codes, "codes", torch.int8, x.device, (R, K))
    if scales is None:
        scales = _empty((R,), (1,), dtype=torch.float32, device=x.device)
    else:
        _flat(scales, "scales", R, x.device)
    _call(lib.mxq_quantize_int8, x.device, x.data_ptr(), _dtype_code(x), R, K, ld, codes.data_ptr(), ldc,
          scales.data_ptr())
    return codes, scales


def dequantize_int8(codes, scales, out=None):
    """8-bit codes [R, K] and scales [R] -> bf16 [R, K]: bf16(fl32(code * scale)) (into ``out`` if given)."""
    ldc = _matrix(codes, "codes", torch.int8)
    R, K = codes.shape
    _flat(scales, "scales", R, codes.device)
    if out is None:
        out, ld = _empty((R, K), (K, 1), dtype=torch.bfloat16, device=codes.device), K
    else:
        ld = _matrix(out, "out", torch.bfloat16, codes.device, (R, K))
    _call(lib.mxq_dequantize_int8, codes.device, codes.data_ptr(), ldc, scales.data_ptr(), R, K, out.data_ptr(), ld)
    return out


def _w8_out(M, N, device, out, out_dtype):
    if out is None:
        if out_dtype not in _FLOATS:
            raise ValueError("out_dtype must be bfloat16 or float32")
        return _empty((M, N), (N, 1), dtype=out_dtype, device=device), N
    return out, _matrix(out, "out", _FLOATS, device, (M, N))


def gemm_w8a8(a_codes, a_scales, w_codes, w_scales, bias=None, out=None, out_dtype=torch.bfloat16):
    """8-bit A [M, K] x W [N, K]^T with a scale for each token and channel -> bf16 or fp32 [M, N]:
    (sum in int32) * a_scales[m] * w_scales[n] + bias[n].  Rows may be strided, scales too (or expanded from one
    value), ``bias`` is float32; ``out`` decides the output type where it is given.  Like every entry point here it
    records nothing for autograd."""
    lda = _matrix(a_codes, "a_codes", torch.int8)
    dev = a_codes.device
    M, K = a_codes.shape
    inc_a = _vector(a_scales, "a_scales", M, dev)
    ldw = _matrix(w_codes, "w_codes", torch.int8, dev)
    N = w_codes.shape[0]
    if w_codes.shape[1] != K:
        raise ValueError(f"w_codes must have {K} columns (got {w_codes.shape[1]})")
    inc_w = _vector(w_scales, "w_scales", N, dev)
    if bias is not None:
        _flat(bias, "bias", N, dev)
    out, ld = _w8_out(M, N, dev, out, out_dtype)
    nbytes = lib.mxq_gemm_w8a8_workspace_bytes(M, N, K)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _call(lib.mxq_gemm_w8a8, dev, a_codes.data_ptr(), lda, a_scales.data_ptr(), inc_a, w_codes.data_ptr(), ldw,
          w_scales.data_ptr(), inc_w, _opt(bias), M, N, K, out.data_ptr(), _dtype_code(out), ld, _opt(ws), nbytes)
    return out


def w8a8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes with which gemm_w8a8 splits K for a shape (0 where it does not)."""
    return int(lib.mxq_gemm_w8a8_workspace_bytes(M, N, K))


def w8a8_fused_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes of gemm_w8a8_fused for a shape."""
    return int(lib.mxq_gemm_w8a8_fused_workspace_bytes(M, N, K))


def gemm_w8a8_fused(a, w_codes, w_scales, bias=None, out=None, out_dtype=torch.bfloat16):
    """gemm_w8a8 of unquantized activations A [M, K] (bf16 or fp32, rows may be strided): equal, bit for bit, to
    gemm_w8a8(*quantize_int8(a), w_codes, w_scales, bias)."""
    lda = _matrix(a, "a", _FLOATS)
    dev = a.device
    M, K = a.shape
    ldw = _matrix(w_codes, "w_codes", torch.int8, dev)
    N = w_codes.shape[0]
    if w_codes.shape[1] != K:
        raise ValueError(f"w_codes must have {K} columns (got {w_codes.shape[1]})")
    inc_w = _vector(w_scales, "w_scales", N, dev)
    if bias is not None:
        _flat(bias, "bias", N, dev)
    out, ld = _w8_out(M, N, dev, out, out_dtype)
    nbytes = lib.mxq_gemm_w8a8_fused_workspace_bytes(M, N, K)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _call(lib.mxq_gemm_w8a8_fused, dev, a.data_ptr(), _dtype_code(a), lda, w_codes.data_ptr(), ldw,
          w_scales.data_ptr(), inc_w, _opt(bias), M, N, K, out.data_ptr(), _dtype_code(out), ld, _opt(ws), nbytes)
    return out


ROPE_STYLES = {"interleaved": 0, "halves": 1}


def _heads(t, name, dtype=None, device=None, shape=None):
    """A 3-D GPU tensor [tokens, heads, head_dim] with contiguous heads: (token pitch, head pitch)."""
    _there(t, name, device)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [tokens, heads, head_dim]")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    T, H, D = t.shape
    ld, hs, step = t.stride()
    if D > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous heads")
    if H <= 1:
        hs = D
    return (ld if T > 1 else H * hs), hs


def _qk_inputs(q, k, q_weight, k_weight, cos, sin, positions, eps, style):
    """Checks shared by the two forms: the C arguments up to the outputs."""
    ldq, hsq = _heads(q, "q")
    dev, (T, Hq, D) = q.device, q.shape
    dt = _dtype_code(q)
    ldk, hsk = _heads(k, "k", q.dtype, dev)
    Tk, Hk, Dk = k.shape
    if Tk != T or Dk != D:
        raise ValueError(f"k must have shape ({T}, heads, {D}) (got {tuple(k.shape)})")
    w_dt = None
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _there(w, name, dev)
            dtype = w.dtype
            if dtype not in _FLOATS:
                raise ValueError(f"{name} must be bfloat16 or float32")
            if w.shape != (D,) or w.stride(0) != 1:
                raise ValueError(f"{name} must be contiguous, of shape ({D},) (got {tuple(w.shape)})")
            if w_dt is not None and dtype != w_dt:
                raise ValueError("q_weight and k_weight must have one dtype")
            w_dt = dtype
    ldt = rows = rot = 0
    if cos is not None and sin is not None:
        ldt = _matrix(cos, "cos", torch.float32, dev)
        if _matrix(sin, "sin", torch.float32, dev, cos.shape) != ldt:
            raise ValueError("cos and sin must have one row pitch")
        rows, rot = cos.shape
    elif cos is not None or sin is not None:
        raise ValueError("cos and sin must be given together")
    if positions is not None:
        _flat(positions, "positions", T, dev, torch.int64)
    if style not in ROPE_STYLES:
        raise ValueError(f"style must be one of {sorted(ROPE_STYLES)}")
    return (q.data_ptr(), Hq, ldq, hsq, k.data_ptr(), Hk, ldk, hsk, dt, T, D, _opt(q_weight), _opt(k_weight),
            MXQ_BF16 if w_dt == torch.bfloat16 else MXQ_F32, eps, _opt(cos), _opt(sin), ldt, rows, 2 * rot,
            _opt(positions), ROPE_STYLES[style])


def _head_out(x, out, name):
    if out is None:
        T, H, D = x.shape
        return _empty((T, H, D), (H * D, D, 1), dtype=x.dtype, device=x.device), (H * D, D)
    return out, _heads(out, name, x.dtype, x.device, x.shape)


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions=None, eps=1e-6, style="interleaved", out_q=None,
                 out_k=None):
    """Root-mean-square norm of every query and key head by itself (not of a token's whole query or key), with the
    position rotation in the same pass.

    ``q`` [T, Hq, D] and ``k`` [T, Hk, D], bf16 or fp32, views of a QKV projection's output as they are (heads
    contiguous, D a multiple of 8 up to 512).  ``q_weight``, ``k_weight``: [D] or None.  ``cos``, ``sin``: float32
    [P, R / 2], R <= D the rotated width, or None for the norm alone.  ``positions``: int64 [T], rows of the tables
    (token t has row t if None); a position outside the tables gives NaN.  ``style``: the pairs that turn,
    "interleaved" (2i, 2i+1) or "halves" (i, i + R/2).  Returns (q, k) of the input's type; ``out_q=q`` and
    ``out_k=k`` work in place.  Like every entry point here it records nothing for autograd."""
    args = _qk_inputs(q, k, q_weight, k_weight, cos, sin, positions, eps, style)
    out_q, (ldq, hsq) = _head_out(q, out_q, "out_q")
    out_k, (ldk, hsk) = _head_out(k, out_k, "out_k")
    _call(lib.mxq_qk_norm_rope, q.device, *args, out_q.data_ptr(), ldq, hsq, out_k.data_ptr(), ldk, hsk)
    return out_q, out_k


def quantize_qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions=None, eps=1e-6, style="interleaved"):
    """qk_norm_rope, then the 8-bit rule of quantize_int8 for each token and head: (q codes int8 [T, Hq, D],
    q scales float32 [T, Hq], k codes, k scales).  With D % 16 == 0, ``gemm_w8a8(qc[:, h], qs[:, h], kc[:, h],
    ks[:, h])`` is the 8-bit score product of head h."""
    args = _qk_inputs(q, k, q_weight, k_weight, cos, sin, positions, eps, style)
    outs = []
    for x in (q, k):
        T, H, D = x.shape
        outs += [_empty((T, H, D), (H * D, D, 1), dtype=torch.int8, device=x.device),
                 _empty((T, H), (H, 1), dtype=torch.float32, device=x.device)]
    qc, qs, kc, ks = outs
    D, Hq, Hk = q.shape[2], q.shape[1], k.shape[1]
    _call(lib.mxq_quantize_qk_norm_rope, q.device, *args, qc.data_ptr(), Hq * D, D, qs.data_ptr(), Hq,
          kc.data_ptr(), Hk * D, D, ks.data_ptr(), Hk)
    return qc, qs, kc, ks


# ---------------------------------------------------------------------------------
# Layer norm, and activations kept in 8 bits for the backward pass.  Forward and backward are separate
# calls, and nothing is recorded for autograd here either.

_SAVES = (None, "x", "int8")


def _plane(t, name, dtype, rows, cols, device):
    """A given [rows, cols] output, or a new one: (tensor, row pitch)."""
    if t is None:
        return _empty((rows, cols), (cols, 1), dtype=dtype, device=device), cols
    return t, _matrix(t, name, dtype, device, (rows, cols))


def _row_values(rows, device):
    return _empty((rows,), (1,), dtype=torch.float32, device=device)


def _norm_vectors(weight, bias, cols, device):
    """The addresses of the weights and biases and their dtype code."""
    dt = None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _there(t, name, device)
            dtype = t.dtype
            if dtype not in _FLOATS:
                raise ValueError(f"{name} must be bfloat16 or float32")
            if t.shape != (cols,) or (cols > 1 and t.stride(0) != 1):
                raise ValueError(f"{name} must be contiguous, of shape ({cols},) (got {tuple(t.shape)})")
            if dt is not None and dtype != dt:
                raise ValueError("weight and bias must have one dtype")
            dt = dtype
    return _opt(weight), _opt(bias), MXQ_BF16 if dt == torch.bfloat16 else MXQ_F32


def _checkpoint(rows, cols, device):
    """New codes and scales: (tensors, C arguments)."""
    codes, scales = _empty((rows, cols), (cols, 1), dtype=torch.int8, device=device), _row_values(rows, device)
    if cols == 0:   # no address of codes, which asks for no checkpoint: the scales of nothing are 0
        scales.zero_()
    return (codes, scales), (codes.data_ptr(), cols, scales.data_ptr())


def _norm_inputs(x, weight, bias, eps, save):
    if save not in _SAVES:
        raise ValueError(f"save must be one of {_SAVES}")
    ld = _matrix(x, "x", _FLOATS)
    dev, (R, C) = x.device, x.shape
    args = (x.data_ptr(), _dtype_code(x), R, C, ld, *_norm_vectors(weight, bias, C, dev), eps)
    if save is None:
        return args, (), (None, None, None, 0, None)
    mean, rstd = _row_values(R, dev), _row_values(R, dev)
    kept, kept_args = _checkpoint(R, C, dev) if save == "int8" else ((), (None, 0, None))
    return args, (mean, rstd, *kept), (mean.data_ptr(), rstd.data_ptr(), *kept_args)


def layer_norm(x, weight=None, bias=None, eps=1e-6, save=None, out=None):
    """Layer norm of the rows of ``x`` [T, C] (bf16 or fp32; C a multiple of 8 up to 16384): ``y`` of x's type.

    ``weight``, ``bias``: [C], bf16 or fp32, either None.  ``save``: what the backward pass needs, from the same
    pass over x: "x" returns (y, mean, rstd), to be kept with x itself; "int8" (C a multiple of 16) returns
    (y, mean, rstd, x_codes, x_scales), the last two equal to quantize_int8(x): half the bytes or less, for a gradient whose
    normalized x is off by up to x_scales / 2 * rstd (much for a row with an outlier or a far mean).  ``out=x`` works in place."""
    args, saved, saved_args = _norm_inputs(x, weight, bias, eps, save)
    y, ld = _plane(out, "out", x.dtype, *x.shape, x.device)
    _call(lib.mxq_layer_norm, x.device, *args, y.data_ptr(), ld, *saved_args)
    return (y, *saved) if saved else y


def quantize_layer_norm(x, weight=None, bias=None, eps=1e-6, save=None):
    """layer_norm to 8-bit codes by the rule of quantize_int8, operands of gemm_w8a8: (codes int8 [T, C], scales
    float32 [T]), followed by what ``save`` asks for as in layer_norm.  C a multiple of 16."""
    args, saved, saved_args = _norm_inputs(x, weight, bias, eps, save)
    (codes, scales), _ = _checkpoint(*x.shape, x.device)
    _call(lib.mxq_quantize_layer_norm, x.device, *args, codes.data_ptr(), x.shape[1], scales.data_ptr(), *saved_args)
    return (codes, scales, *saved)


def layer_norm_backward(dy, x, mean, rstd, weight=None, x_scales=None, out=None, sums=None):
    """Gradient of layer_norm: (dx, dweight, dbias), the last two float32 [C], or None where they are not formed.

    ``dy`` [T, C], bf16 or fp32; ``x``: the forward input, of dy's type, or its int8 codes with ``x_scales``
    (save="int8").  ``mean``, ``rstd``: float32 [T] of the forward pass.  dx has dy's type; ``out=dy`` works in place.
    ``sums``: whether dweight and dbias are formed, by default where there is a ``weight``; True for a norm with a
    bias alone, False where the weights are not trained.  The sums over rows are formed in a fixed order."""
    ld = _matrix(dy, "dy", _FLOATS)
    dev, (R, C) = dy.device, dy.shape
    if x_scales is not None:
        _flat(x_scales, "x_scales", R, dev)
    ldx = _matrix(x, "x", dy.dtype if x_scales is None else torch.int8, dev, (R, C))
    _flat(mean, "mean", R, dev)
    _flat(rstd, "rstd", R, dev)
    w, _, w_dt = _norm_vectors(weight, None, C, dev)
    dx, ldo = _plane(out, "out", dy.dtype, R, C, dev)
    dw = db = ws = None
    nbytes = 0
    if weight is not None if sums is None else sums:
        dw, db = _row_values(C, dev), _row_values(C, dev)
        nbytes = lib.mxq_layer_norm_backward_workspace_bytes(R, C)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _call(lib.mxq_layer_norm_backward, dev, dy.data_ptr(), _dtype_code(dy), R, C, ld, x.data_ptr(), ldx, _opt(x_scales),
          mean.data_ptr(), rstd.data_ptr(), w, w_dt, dx.data_ptr(), ldo, _opt(dw), _opt(db), _opt(ws), nbytes)
    return dx, dw, db


ACTIVATIONS = {"gelu_tanh": 0, "silu": 1}


def _act_code(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def _act_inputs(u, act, save):
    if save not in (None, "int8"):
        raise ValueError("save must be None or 'int8'")
    ld = _matrix(u, "u", _FLOATS)
    R, C = u.shape
    kept, kept_args = _checkpoint(R, C, u.device) if save else ((), (None, 0, None))
    return (u.data_ptr(), _dtype_code(u), R, C, ld, _act_code(act)), kept, kept_args


def activation(u, act="gelu_tanh", save=None, out=None):
    """f(u) of a feed-forward layer, element by element ([T, C], bf16 or fp32, C a multiple of 8 up to 65536): ``y`` of u's
    type.  ``act``: "gelu_tanh" or "silu".  save="int8" (C a multiple of 16) returns (y, u_codes, u_scales), the 8-bit
    checkpoint that activation_backward takes, from the same pass.  ``out=u`` works in place."""
    args, kept, kept_args = _act_inputs(u, act, save)
    y, ld = _plane(out, "out", u.dtype, *u.shape, u.device)
    _call(lib.mxq_activation, u.device, *args, y.data_ptr(), ld, *kept_args)
    return (y, *kept) if kept else y


def quantize_activation(u, act="gelu_tanh", save=None):
    """activation to 8-bit codes by the rule of quantize_int8, operands of gemm_w8a8: (codes int8 [T, C], scales
    float32 [T]), followed by the checkpoint with save="int8".  C a multiple of 16."""
    args, kept, kept_args = _act_inputs(u, act, save)
    (codes, scales), _ = _checkpoint(*u.shape, u.device)
    _call(lib.mxq_quantize_activation, u.device, *args, codes.data_ptr(), u.shape[1], scales.data_ptr(), *kept_args)
    return (codes, scales, *kept)


def activation_backward(dy, u_codes, u_scales, act="gelu_tanh", out=None):
    """dy * f'(u) from the 8-bit checkpoint of the same ``act``: [T, C] of dy's type (``out=dy`` works in place)."""
    ld = _matrix(dy, "dy", _FLOATS)
    dev, (R, C) = dy.device, dy.shape
    ldc = _matrix(u_codes, "u_codes", torch.int8, dev, (R, C))
    _flat(u_scales, "u_scales", R, dev)
    du, ldo = _plane(out, "out", dy.dtype, R, C, dev)
    _call(lib.mxq_activation_backward, dev, dy.data_ptr(), _dtype_code(dy), R, C, ld, u_codes.data_ptr(), ldc,
          u_scales.data_ptr(), _act_code(act), du.data_ptr(), ldo)
    return du


def grad_weight_int8(dy, codes, scales, out=None, out_dtype=torch.float32, accumulate=False):
    """Weight gradient of gemm_w8a8 from the activations' codes: dy [M, N] (bf16)^T x dequantize_int8(codes [M, K],
    scales [M]) -> [N, K], float32 or bfloat16 (``out`` decides where it is given).  N a multiple of 8, K of 16; rows
    may be strided.  accumulate=True adds to ``out``.  The sum over M is formed in an order that the sizes alone decide."""
    ldy = _matrix(dy, "dy", torch.bfloat16)
    dev, (M, N) = dy.device, dy.shape
    ldc = _matrix(codes, "codes", torch.int8, dev)
    K = codes.shape[1]
    if codes.shape[0] != M:
        raise ValueError(f"codes must have {M} rows (got {codes.shape[0]})")
    _flat(scales, "scales", M, dev)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    out, ld = _w8_out(N, K, dev, out, out_dtype)
    nbytes = lib.mxq_grad_weight_int8_workspace_bytes(M, N, K)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _call(lib.mxq_grad_weight_int8, dev, dy.data_ptr(), ldy, codes.data_ptr(), ldc, scales.data_ptr(), M, N, K,
          out.data_ptr(), _dtype_code(out), ld, int(accumulate), _opt(ws), nbytes)
    return out
