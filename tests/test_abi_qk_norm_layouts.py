"""Output layouts of the head norm, decided before anything is launched (no GPU needed): two heads
on the same memory would be written by different waves, so such pitches are refused, and every
layout that keeps the heads apart passes the checks."""

import ctypes
import itertools

import pytest
import torch

import mxfp4_microscaled_quantization_amd as mxq

OK16 = ctypes.c_void_p(0x10000)   # never dereferenced
D = 64


def _norm(T, H, ld, hs):
    return mxq.lib.mxq_qk_norm_rope(OK16, H, H * D, D, None, 0, 0, 0, 1, T, D, None, None, 1, ctypes.c_float(1e-6), None, None, 0, 0,
                                    0, None, 0, OK16, ld, hs, None, 0, 0, None)


def _codes(T, H, ld, hs):
    return mxq.lib.mxq_quantize_qk_norm_rope(None, 0, 0, 0, OK16, H, H * D, D, 1, T, D, None, None, 1, ctypes.c_float(1e-6), None,
                                             None, 0, 0, 0, None, 0, None, 0, 0, None, 0, OK16, ld, hs, OK16, H, None)


def _overlap(T, H, ld, hs):
    """From the definition: the sorted starts of all heads, nearer than a head somewhere."""
    at = sorted(t * ld + h * hs for t in range(T) for h in range(H))
    return any(b - a < D for a, b in zip(at, at[1:]))


def _refused(status):
    return status == mxq.MXQ_ERR_INVALID_ARG and b"overlap" in mxq.lib.mxq_last_error()


@pytest.mark.parametrize("call", [_norm, _codes])
def test_two_heads_on_the_same_memory_are_refused(call):
    # token t's second head would be token t + 1's first
    assert _refused(call(4, 2, D, D))
    assert _refused(call(4, 2, D, D + 16)) and _refused(call(4, 3, 2 * D, D)) and _refused(call(600, 40, 39 * D, D))
    # the largest counts and pitches that do not pass the other limits
    assert _refused(call(2 ** 31 - 1, 65536, D, D)) and _refused(call(2 ** 31 - 1, 2, 2 ** 24, 2 ** 25))
    assert _refused(call(65536, 65536, 4097 * 64, D))


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would reach the launch with pointers to nothing")
@pytest.mark.parametrize("call", [_norm, _codes])
def test_every_layout_is_judged_as_its_places_are(call):
    """Against the places themselves, for all small counts and pitches: tokens outside, heads outside
    and layouts where the two are threaded through each other."""
    refused = 0
    for T, H, ld, hs in itertools.product(range(1, 6), range(1, 6), range(D, 6 * D + 1, 16), range(D, 6 * D + 1, 16)):
        status = call(T, H, ld, hs)
        if _overlap(T, H, ld, hs):
            assert _refused(status), (T, H, ld, hs)
            refused += 1
        else:
            assert status == mxq.MXQ_ERR_HIP, (T, H, ld, hs, mxq.lib.mxq_last_error())   # past the checks, no device
    assert refused > 100
