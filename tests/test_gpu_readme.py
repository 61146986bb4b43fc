"""The README's examples run as they stand, and the training example's gradients are those of the products that it ran."""

import os
import re

import pytest
import torch

from helpers import announce

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_examples(gpu):
    announce("README examples")
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert len(blocks) == 2
    env, calls = {}, []
    plain = gpu.gemm_bf16
    gpu.gemm_bf16 = lambda a, w, *r: calls.append((a, w, plain(a, w, *r))) or calls[-1][2]
    try:
        for b in blocks:
            exec(b, env)
    finally:
        gpu.gemm_bf16 = plain
    # the two input gradients: dy times the weights that the codes stand for, as dequantize_int8 gives them
    assert len(calls) == 2 and calls[0][0] is env["dz"] and calls[1][0] is env["du"]
    for (dy, _, got), c, s in zip(calls, (env["c2"], env["c1"]), (env["s2"], env["s1"])):
        w = (c.float() * s[:, None]).bfloat16().double()
        ref, size = dy.double() @ w, dy.double().abs() @ w.abs()
        # exact products summed in binary32 (the bar of every product here), rounded to bf16
        assert ((got.double() - ref).abs() <= 1e-5 * size + 2.0 ** -8 * (ref.abs() + 1e-5 * size)).all()
    for name, shape in (("dw1", (13824, 5120)), ("dw2", (5120, 13824)), ("dx", (4096, 5120)), ("dg", (5120,)), ("db", (5120,))):
        assert env[name].shape == shape and env[name].isfinite().all() and env[name].any()
