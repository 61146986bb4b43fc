"""The weight gradient's routes: the largest tile on values widened ahead of it, and whole tiles beside tiles cut into parts of M
in one launch, of either tile.  The route of each shape is told by its workspace, so that another plan cannot pass
these by.  Against 64 bits on the GPU, with the bars of test_gpu_grad_weight."""

import pytest
import torch

from helpers import announce
from test_gpu_training_block import _Step, _same

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _inputs(M, N, K, seed, pad=0):
    """Operands inside wider buffers of NaN (dy, scales) and other codes."""
    g = torch.Generator("cuda").manual_seed(seed)
    dy = torch.full((M + 64, N + pad), float("nan"), device="cuda", dtype=BF16)
    dy[:M, :N] = torch.randn(M, N, device="cuda", generator=g).bfloat16()
    codes = torch.randint(-128, 128, (M + 64, K + 2 * pad), device="cuda", generator=g, dtype=torch.int16).to(torch.int8)
    s = torch.full((M + 64,), float("nan"), device="cuda")
    s[:M] = torch.rand(M, device="cuda", generator=g) * 0.05 + 1e-3
    return dy[:M, :N], codes[:M, :K], s[:M]


def _exact(dy, codes, s):
    x = (codes.float() * s[:, None]).bfloat16().double()
    d = dy.double().t().contiguous()
    return d @ x, d.abs() @ x.abs()


def _check(out, ref, size, extra=0.0):
    tol = 1e-5 * size + HALF[out.dtype] * (ref.abs() * (1 + 2.0 ** -10) + 1e-5 * size) + extra
    worst = ((out.double() - ref).abs() / tol).max().item()
    assert out.shape == ref.shape and worst <= 1.0, worst


def _route(gpu, M, N, K, tile, parts):
    """Whether the plan takes `tile`, with some ("cut": all tiles, "mixed": some) or no ("whole") tiles in parts of M."""
    nbytes = gpu.lib.mxq_grad_weight_int8_workspace_bytes(M, N, K)
    values = (2 * M * K + 255) // 256 * 256 if tile == 256 else 0
    tiles, slots = -(-N // tile) * -(-K // tile), 256 if tile == 256 else 512
    sums, rest = (nbytes - values) // (4 * tile * tile), tiles % slots
    assert nbytes >= values and (nbytes - values) % (4 * tile * tile) == 0
    if parts == "whole":
        return sums == 0
    return sums >= 2 * rest > 0 and sums % rest == 0 and (rest < tiles) == (parts == "mixed")


SHAPES = [(500, 3080, 4112, 256, "whole"), (1101, 4088, 4064, 256, "whole"), (4001, 2056, 2064, 256, "cut"), (2001, 4104, 4368, 256, "mixed"),
          (9001, 5128, 6160, 256, "mixed"), (1001, 2056, 4112, 128, "mixed"), (500, 72, 80, 128, "whole"), (2049, 136, 112, 128, "cut")]


@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("M,N,K,tile,parts", SHAPES)
def test_routes(gpu, M, N, K, tile, parts, pad):
    announce(f"grad_weight_int8 {M}x{N}x{K} tile {tile} {parts} pad {pad}")
    assert _route(gpu, M, N, K, tile, parts)
    dy, codes, s = _inputs(M, N, K, M + N + K, pad)
    ref, size = _exact(dy, codes, s)
    out = gpu.grad_weight_int8(dy, codes, s)
    _check(out, ref, size)
    assert torch.equal(out, gpu.grad_weight_int8(dy, codes, s))
    assert torch.equal(gpu.grad_weight_int8(dy, codes, s, out_dtype=BF16), out.bfloat16())
    # into a wider buffer, on a boundary and beside one, and added to what it holds; nothing else is written
    for dtype in (F32, BF16):
        for off in (0, 1):
            wide = torch.randn(N + 2, K + 8, device="cuda").to(dtype)
            view, before = wide[1:N + 1, off:K + off], wide.clone()
            have = before[1:N + 1, off:K + off].double()
            gpu.grad_weight_int8(dy, codes, s, out=view, accumulate=True)
            _check(view, ref + have, size, 2.0 ** -23 * (have.abs() + ref.abs()))
            gpu.grad_weight_int8(dy, codes, s, out=view)
            assert torch.equal(view, out.to(dtype))
            view.copy_(before[1:N + 1, off:K + off])
            assert torch.equal(wide, before)


def test_values_past_2_32(gpu):
    """Codes and widened values past 2^32 elements, whole and cut tiles of the largest size: exact sums of integers."""
    M, N, K = 220000, 2056, 20000
    announce(f"grad_weight_int8 {M}x{N}x{K}")
    assert M * K > 2 ** 32 and _route(gpu, M, N, K, 256, "mixed")
    g = torch.Generator("cuda").manual_seed(2)
    dy = torch.zeros(M, N, dtype=BF16, device="cuda")
    # one value a row, +-1, and codes of -2 .. 2 with scale 1
    col = torch.randint(0, N, (M,), device="cuda", generator=g)
    sign = torch.randint(0, 2, (M,), device="cuda", generator=g) * 2 - 1
    dy[torch.arange(M, device="cuda"), col] = sign.bfloat16()
    codes = torch.empty(M, K, dtype=torch.int8, device="cuda")
    want = torch.zeros(N, K, device="cuda")
    for r in range(0, M, 20000):
        part = torch.randint(-2, 3, (20000, K), device="cuda", generator=g, dtype=torch.int16)
        codes[r:r + 20000] = part.to(torch.int8)
        want.index_add_(0, col[r:r + 20000], part.float() * sign[r:r + 20000, None])
    assert torch.equal(gpu.grad_weight_int8(dy, codes, torch.ones(M, device="cuda")), want)


def _pair(gpu):
    # whole tiles on widened values both ways; all tiles in parts, on widened values
    steps = _Step(gpu, 500, 3088, 4112, "gelu_tanh", 1), _Step(gpu, 4001, 2064, 2064, "silu", 2)
    assert _route(gpu, 500, 3088, 4112, 256, "whole") and _route(gpu, 500, 4112, 3088, 256, "whole")
    assert _route(gpu, 4001, 2064, 2064, 256, "cut")
    return steps


def test_two_streams_at_once(gpu):
    announce("training step with the largest tile: two streams")
    a, b = _pair(gpu)
    ra, rb = a.run(), b.run()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(sa):
            oa = a.run()
        with torch.cuda.stream(sb):
            ob = b.run()
        torch.cuda.synchronize()
        assert _same(oa, ra) and _same(ob, rb)


def test_captured_steps_replay_the_eager_results(gpu):
    announce("training step with the largest tile: graphs")
    steps = _pair(gpu)
    refs = [s.run() for s in steps]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in steps:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.run()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run())
        graphs.append(g)
    for turn in range(3):
        for o in outs:
            for t in o.values():
                t.fill_(7)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert _same(outs[0], refs[0]) and _same(outs[1], refs[1]), turn
        assert _same(steps[turn % 2].run(), refs[turn % 2])
        torch.cuda.synchronize()
