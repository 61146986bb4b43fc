"""Norm and rotation of few heads for many tokens (waves of (token, head) pairs) on tensors whose offsets pass
32 bits: a block of tokens repeated many times gives the block's results, repeated."""

import pytest
import torch

from helpers import announce

pytestmark = pytest.mark.gpu


def _repeats(out, block):
    return bool((out.view(-1, *block.shape) == block).all())


@pytest.mark.parametrize("dtype,heads", [(torch.bfloat16, (1, 1)), (torch.bfloat16, (3, 1)), (torch.float32, (1, 0))])
def test_pairs(gpu, dtype, heads):
    T, D, H = 1000, 128, sum(heads)
    n = 2 ** 32 // (T * H * D) + 200                       # more than 2^32 elements: offsets in bytes pass 2^33
    announce(f"qk_norm_rope {T * n} tokens x {heads} heads, {dtype}")
    block = torch.randn(T, H, D, device="cuda").to(dtype)
    ang = torch.rand(T, D // 2, device="cuda") * 6
    args = (torch.rand(D, device="cuda"), torch.rand(D, device="cuda"), ang.cos(), ang.sin())
    x = block.expand(n, T, H, D).reshape(n * T, H, D)
    assert x.numel() > 2 ** 32
    pos = torch.arange(T * n, device="cuda") % T
    for style in ("interleaved", "halves"):
        for fn in (gpu.qk_norm_rope, gpu.quantize_qk_norm_rope):
            small = fn(block[:, :heads[0]], block[:, heads[0]:], *args, style=style)
            for o, r in zip(fn(x[:, :heads[0]], x[:, heads[0]:], *args, positions=pos, style=style), small):
                if r.numel():
                    assert _repeats(o, r)
