"""The norm, activation and weight gradient together with the 8-bit products, as a training step of a feed-forward
block runs them: on one stream, on two, inside captured graphs, and on another device.

Every call only enqueues work on the caller's stream and keeps nothing: two streams at once give the bits of one, and a
captured pass (its workspaces from the graph's own pool) gives the eager results on every replay."""

import numpy as np
import pytest
import torch

import oracle
from oracle import training as tr
from helpers import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _np(t):
    return t.detach().double().cpu().numpy()


class _Step:
    """y = act(norm(x) W1^T + b1) W2^T: forward with every activation kept in 8 bits, and backward from those."""

    def __init__(self, mxq, T, C, F, act, seed, device="cuda"):
        self.mxq, self.act = mxq, act
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s: torch.randn(s, device=device, generator=g)   # noqa: E731
        self.x, self.w, self.b = r(T, C).mul_(2).add_(0.3).bfloat16(), (1 + 0.2 * r(C)).bfloat16(), (0.1 * r(C)).bfloat16()
        self.w1, self.w2 = (r(F, C) * C ** -0.5).bfloat16(), (r(C, F) * F ** -0.5).bfloat16()
        self.b1, self.dz = 0.1 * r(F), r(T, C).bfloat16()
        self.q1, self.q2 = mxq.quantize_int8(self.w1), mxq.quantize_int8(self.w2)
        # for the products of the backward pass: channels are then columns of the weights
        self.t1, self.t2 = mxq.quantize_int8(self.w1.t().contiguous()), mxq.quantize_int8(self.w2.t().contiguous())
        self.acc = r(C, F)

    def run(self):
        m = self.mxq
        n, ns, mean, rstd, xc, xs = m.quantize_layer_norm(self.x, self.w, self.b, eps=1e-5, save="int8")
        u = m.gemm_w8a8(n, ns, *self.q1, bias=self.b1)
        h, hs, uc, us = m.quantize_activation(u, self.act, save="int8")
        z = m.gemm_w8a8(h, hs, *self.q2)
        acc = self.acc.clone()
        dw2 = m.grad_weight_int8(self.dz, h, hs, out=acc, accumulate=True)
        dh = m.gemm_w8a8_fused(self.dz, *self.t2)
        du = m.activation_backward(dh, uc, us, self.act)
        dw1 = m.grad_weight_int8(du, n, ns, out_dtype=BF16)
        dn = m.gemm_w8a8_fused(du, *self.t1)
        dx, dw, db = m.layer_norm_backward(dn, xc, mean, rstd, self.w, x_scales=xs)
        y, mean2, rstd2 = m.layer_norm(self.x, self.w, self.b, eps=1e-5, save="x")
        dx2, dw_2, db_2 = m.layer_norm_backward(dn, self.x, mean2, rstd2, self.w)
        return dict(n=n, ns=ns, mean=mean, rstd=rstd, xc=xc, xs=xs, u=u, h=h, hs=hs, uc=uc, us=us, z=z, dw2=dw2, dh=dh, du=du, dw1=dw1,
                    dn=dn, dx=dx, dw=dw, db=db, y=y, mean2=mean2, rstd2=rstd2, dx2=dx2, dw_2=dw_2, db_2=db_2)


def _same(a, b):
    return [k for k in a if not torch.equal(a[k], b[k])] == []


@pytest.mark.parametrize("T,C,F,act", [(1, 64, 128, "silu"), (77, 640, 1360, "gelu_tanh"), (515, 1040, 4112, "gelu_tanh"), (1100, 512, 2064, "silu")])
def test_step_against_the_oracle(gpu, T, C, F, act):
    """Each stage on the values that the stages before it gave, within the tolerance of its own tests."""
    announce(f"training step {T}x{C}x{F} {act}")
    s = _Step(gpu, T, C, F, act, T + C)
    r = s.run()
    deq = lambda c, q: oracle.dequantize_int8(c.cpu().numpy(), q.cpu().numpy())   # noqa: E731

    def near(got, ref, size, steps, half):
        assert np.all(np.abs(_np(got) - ref) <= steps * size + half * np.abs(ref) * (1 + 2.0 ** -10))

    ref, mean, rstd, size = tr.layer_norm(_np(s.x), _np(s.w), _np(s.b), 1e-5)
    near(r["y"], ref, size, 2.0 ** -18, 2.0 ** -8)
    hs = _np(r["ns"])[:, None]
    assert np.all(np.abs(_np(r["n"]) * hs - ref) <= (0.5 + 127 * 2.0 ** -22) * hs + 2.0 ** -18 * size + 2.0 ** -24 * np.abs(ref))
    assert torch.equal(r["mean"], r["mean2"]) and torch.equal(r["rstd"], r["rstd2"])
    assert all(torch.equal(a, b) for a, b in zip((r["xc"], r["xs"]), gpu.quantize_int8(s.x)))
    u = _np(r["u"])
    ref, z = tr.activation(u, act)
    tol = 2.0 ** -24 * (6 * z + 16) * np.abs(ref) + 2.0 ** -100 * np.abs(u)
    hs = _np(r["hs"])[:, None]
    assert np.all(np.abs(_np(r["h"]) * hs - ref) <= (0.5 + 127 * 2.0 ** -22) * hs + tol)
    rc, rs = tr.activation_checkpoint(r["u"].float().cpu().numpy(), act)
    assert np.array_equal(r["uc"].cpu().numpy(), rc) and np.array_equal(r["us"].cpu().numpy(), rs)
    slope, z, size = tr.activation_slope(deq(r["uc"], r["us"]), act)
    d = _np(r["dh"])
    near(r["du"], d * slope, (12 * z + 32) * size * np.abs(d), 2.0 ** -24, 2.0 ** -8)
    ref, size = tr.grad_weight_int8(_np(s.dz), r["h"].cpu().numpy(), _np(r["hs"]).astype(np.float32))
    ref = ref + _np(s.acc)
    near(r["dw2"], ref, size + 2.0 ** -6 * np.abs(_np(s.acc)), 1e-5, 2.0 ** -24)
    ref, size = tr.grad_weight_int8(_np(r["du"]), r["n"].cpu().numpy(), _np(r["ns"]).astype(np.float32))
    near(r["dw1"], ref, size * 1.01, 1e-5, 2.0 ** -8)
    for dx, dw, db, x in ((r["dx"], r["dw"], r["db"], deq(r["xc"], r["xs"])), (r["dx2"], r["dw_2"], r["db_2"], _np(s.x))):
        ex, ew, eb, sx, sw, sb = tr.layer_norm_backward(_np(r["dn"]), x, _np(r["mean"]), _np(r["rstd"]), _np(s.w))
        near(dx, ex, sx, 2.0 ** -18, 2.0 ** -8)
        near(dw, ew, sw, 2.0 ** -17, 2.0 ** -24)
        near(db, eb, sb, 2.0 ** -17, 2.0 ** -24)


def _pair(mxq):
    # the two take different kernels: short and long rows, parts of M with their joining, the largest tile
    return _Step(mxq, 1500, 256, 2064, "gelu_tanh", 1), _Step(mxq, 700, 2816, 2832, "silu", 2)


def test_two_streams_at_once(gpu):
    announce("training step: two streams")
    a, b = _pair(gpu)
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


def test_captured_steps_replay_the_eager_results(gpu):
    """Two graphs, replayed in turn and at once on two streams, with eager work between the replays."""
    announce("training step: graphs")
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
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert _same(outs[0], refs[0]) and _same(outs[1], refs[1])


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_on_another_device(gpu):
    announce("training step: another device")
    s = _Step(gpu, 300, 640, 1360, "silu", 5, "cuda:1")
    assert torch.cuda.current_device() == 0
    out = s.run()
    torch.cuda.synchronize("cuda:1")
    assert torch.cuda.current_device() == 0 and all(t.device.index == 1 for t in out.values())
    with torch.cuda.device(1):
        assert _same(out, s.run())


def test_tensors_on_two_devices_are_refused(gpu):
    x, w = torch.randn(8, 64, device="cuda"), torch.ones(64)
    with pytest.raises(ValueError, match="GPU tensor"):
        gpu.layer_norm(x, w)
    _, mean, rstd = gpu.layer_norm(x, save="x")
    with pytest.raises(ValueError, match="GPU tensor"):
        gpu.layer_norm_backward(x, x, mean.cpu(), rstd)
    _, c, s = gpu.activation(x, save="int8")
    with pytest.raises(ValueError, match="GPU tensor"):
        gpu.activation_backward(x, c, s.cpu())
    with pytest.raises(ValueError, match="GPU tensor"):
        gpu.grad_weight_int8(x.bfloat16(), c.cpu(), s)
