"""The 8-bit operators on several streams, inside captured graphs and on another device.

Every call only enqueues work on the caller's stream and keeps nothing: two streams at once
give the bits of one, and a captured pass (its workspaces from the graph's own pool) gives
the eager results on every replay, with eager work between the replays."""

import pytest
import torch

from helpers import announce

pytestmark = pytest.mark.gpu


class _Pass:
    """The block path at sizes that take every route: the one-launch product, a split of K
    with its reduction, the largest tile, and both forms of the head norm."""

    def __init__(self, mxq, seed, device="cuda"):
        self.mxq = mxq
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(s, device=device, generator=g)   # noqa: E731
        self.x1, self.x2, self.x3 = r(3, 2048).bfloat16(), r(40, 13824).bfloat16(), r(600, 1040)
        self.w = [mxq.quantize_int8(r(n, k)) for n, k in ((300, 2048), (512, 13824), (1536, 1040))]
        self.b = r(512)
        self.cos, self.sin = r(700, 32), r(700, 32)
        self.pos = torch.randint(0, 700, (600,), device=device, generator=g)
        self.wn = r(64).abs()

    def run(self):
        m = self.mxq
        y1 = m.gemm_w8a8_fused(self.x1, *self.w[0])
        q2, s2 = m.quantize_int8(self.x2)
        y2 = m.gemm_w8a8(q2, s2, *self.w[1], bias=self.b, out_dtype=torch.float32)
        y3 = m.gemm_w8a8_fused(self.x3, *self.w[2])
        q, k = y3[:, :512].view(600, 8, 64), y3[:, 512:1024].view(600, 8, 64)
        n = m.qk_norm_rope(q, k, self.wn, self.wn, self.cos, self.sin, positions=self.pos, style="halves")
        c = m.quantize_qk_norm_rope(q, k, self.wn, self.wn, self.cos, self.sin, positions=self.pos)
        d = m.dequantize_int8(c[0].view(-1, 64), c[1].view(-1))
        s = m.gemm_w8a8(c[0][:, 3], c[1][:, 3], c[2][:, 3], c[3][:, 3], out_dtype=torch.float32)
        return [y1, q2, s2, y2, y3, *n, *c, d, s]


def _same(xs, ys):
    return [i for i, (x, y) in enumerate(zip(xs, ys)) if not torch.equal(x, y)] == []


def test_two_streams_at_once(gpu):
    announce("8-bit operators: two streams")
    a, b = _Pass(gpu, 1), _Pass(gpu, 2)
    ra, rb = a.run(), b.run()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(sa):
            oa = a.run()
        with torch.cuda.stream(sb):
            ob = b.run()
        with torch.cuda.stream(sa):
            oc = a.run()
        torch.cuda.synchronize()
        assert _same(oa, ra) and _same(ob, rb) and _same(oc, ra)


def test_captured_passes_replay_the_eager_results(gpu):
    """Two graphs of the same operators, replayed in turn and at once on two streams."""
    announce("8-bit operators: graphs")
    passes = [_Pass(gpu, 3), _Pass(gpu, 4)]
    refs = [p.run() for p in passes]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p in passes:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            p.run()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(p.run())
        graphs.append(g)
    for turn in range(3):
        for o in outs:
            for t in o:
                t.fill_(7)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert _same(outs[0], refs[0]) and _same(outs[1], refs[1]), turn
        assert _same(passes[turn % 2].run(), refs[turn % 2])       # eager work between the replays
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert _same(outs[0], refs[0]) and _same(outs[1], refs[1])


def test_graph_reads_new_inputs(gpu):
    announce("8-bit operators: graph with new inputs")
    x = torch.randn(2, 1024, device="cuda").bfloat16()
    w, ws = gpu.quantize_int8(torch.randn(96, 1024, device="cuda"))
    gpu.gemm_w8a8_fused(x, w, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = gpu.gemm_w8a8_fused(x, w, ws)
    for seed in range(4):
        x.copy_(torch.randn(2, 1024, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, gpu.gemm_w8a8(*gpu.quantize_int8(x), w, ws))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_on_another_device(gpu):
    announce("8-bit operators: another device")
    ref = _Pass(gpu, 5).run()
    assert torch.cuda.current_device() == 0
    p = _Pass(gpu, 5, "cuda:1")
    out = p.run()
    torch.cuda.synchronize("cuda:1")
    assert torch.cuda.current_device() == 0 and all(t.device.index == 1 for t in out)
    assert len(out) == len(ref)
    with torch.cuda.device(1):
        assert _same(out, p.run())


def test_tensors_on_two_devices_are_refused(gpu):
    w, ws = gpu.quantize_int8(torch.randn(8, 64, device="cuda"))
    with pytest.raises(ValueError, match="GPU tensor"):
        gpu.gemm_w8a8(w, ws, w.cpu(), ws)
    with pytest.raises(ValueError, match="GPU tensor"):
        gpu.gemm_w8a8_fused(torch.randn(8, 64, device="cuda"), w, ws, bias=torch.zeros(8))
