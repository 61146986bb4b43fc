"""Workloads of the layer norm (plain, to 8-bit codes, and its gradient) and of activations kept in 8 bits
for the backward pass (the FFN's activation and its derivative, the weight gradient of an 8-bit product).

`own` false: elementary torch operations; true: the library's entry points."""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-6
LIMIT = {"gelu_tanh": 4.0, "silu": 8.0}   # beyond it the derivative is flat, and the checkpoint saturates


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a 5120-wide transformer: latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 5120, "type": "bf16", "affine": True, "pad": 0},
        # every latent token of Wan2.2, ahead of cross attention
        {"name": "norm_wan", "op": "norm", "rows": 75600, "cols": 5120, "type": "bf16", "affine": True, "pad": 0},
        # to the codes of an 8-bit product (and their dequantization): odd row count, rows of a wider buffer, binary32
        {"name": "norm_int8_ragged", "op": "norm_int8", "rows": 1001, "cols": 1360, "type": "fp32", "affine": True, "pad": 16},
        # the gradient from the kept input
        {"name": "norm_grad_wan", "op": "norm_grad", "rows": 75600, "cols": 5120, "type": "bf16", "affine": True, "pad": 0},
        # forward and backward with the input kept in 8 bits
        {"name": "norm_train_wan", "op": "norm_train", "rows": 75600, "cols": 5120, "type": "bf16", "affine": True, "pad": 0},
        # the same, small and ragged, binary32
        {"name": "norm_train_ragged", "op": "norm_train", "rows": 4099, "cols": 2064, "type": "fp32", "affine": True, "pad": 48},
        # one token's FFN activation to the codes of the second product (and their dequantization): latency
        {"name": "act_int8_token", "op": "act_int8", "rows": 1, "cols": 13824, "type": "bf16", "act": "gelu_tanh", "pad": 0},
        # the Wan2.2 FFN's activation, forward with an 8-bit checkpoint and backward from it
        {"name": "act_train_wan", "op": "act_train", "rows": 75600, "cols": 13824, "type": "bf16", "act": "gelu_tanh", "pad": 0},
        # the same with the other activation, odd rows of a wider buffer, binary32
        {"name": "act_train_ragged", "op": "act_train", "rows": 777, "cols": 1936, "type": "fp32", "act": "silu", "pad": 16},
        # weight gradient of a small layer, nothing a multiple of a tile
        {"name": "wgrad_ragged", "op": "wgrad", "M": 1001, "N": 2056, "K": 1360, "out": "fp32", "pad": 16},
        # one image's tokens through a square projection
        {"name": "wgrad_image", "op": "wgrad", "M": 3584, "N": 5120, "K": 5120, "out": "bf16", "pad": 0},
        # the Wan2.2 FFN-up layer
        {"name": "wgrad_wan", "op": "wgrad", "M": 75600, "N": 13824, "K": 5120, "out": "fp32", "pad": 0},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm_int8", "norm_grad", "norm_train", "act_int8", "act_train", "wgrad", "wgrad", "wgrad"])
    pad = rng.choice([0, 0, 16, 48])
    if op == "wgrad":
        N, K = _log(rng, 16, 14000, 8), _log(rng, 16, 14000, 16)
        most = int(min(75600, 8e12 / (2 * N * K)))   # tokens
        return {"op": op, "M": _log(rng, 1, most), "N": N, "K": K, "out": rng.choice(["bf16", "fp32"]), "pad": pad}
    c = {"op": op, "rows": _log(rng, 1, 60000), "cols": _log(rng, 64, 14000, 16), "type": rng.choice(["bf16", "bf16", "fp32"]), "pad": pad}
    if op.startswith("norm"):
        c["affine"] = rng.random() < 0.75
    else:
        c["act"] = rng.choice(["gelu_tanh", "silu"])
    return c


# ---------------------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _rows(g, rows, cols, dtype, pad, ch=None, shift=None):
    """N(0, 1), times a scale and plus an offset for each channel, as rows of a buffer `pad` columns wider."""
    wide = torch.zeros((rows, cols + pad), dtype=dtype, device=DEV)
    for r in range(0, rows, 16384):   # in slices: the binary32 draw of a large case stays small
        v = _randn(g, min(16384, rows - r), cols)
        if ch is not None:
            v = v * ch
        if shift is not None:
            v = v + shift
        wide[r:r + 16384, :cols] = v
    return wide[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, st = case["op"], {"case": case}
    if op == "wgrad":
        M, N, K, pad = case["M"], case["N"], case["K"], case["pad"]
        st["dy"] = _rows(g, M, N, torch.bfloat16, pad, ch=torch.full((N,), 0.02, device=DEV))
        # the codes and scales that the forward product took: they are kept, and nothing else is
        ch = torch.exp(_randn(g, K))
        codes = torch.zeros((M, K + pad), dtype=torch.int8, device=DEV)
        st["scales"] = torch.empty(M, dtype=torch.float32, device=DEV)
        for r in range(0, M, 16384):
            codes[r:r + 16384, :K], st["scales"][r:r + 16384] = _quantize(_randn(g, min(16384, M - r), K) * ch)
        st["codes"] = codes[:, :K]
        return st
    rows, cols, dtype, pad = case["rows"], case["cols"], TYPES[case["type"]], case["pad"]
    if op.startswith("act"):
        st["u"] = _rows(g, rows, cols, dtype, pad, ch=torch.exp(0.5 * _randn(g, cols)), shift=0.3 * _randn(g, cols) - 0.2)
    else:
        # the residual stream: outlier channels, some of them with a mean of their own
        st["x"] = _rows(g, rows, cols, dtype, pad, ch=torch.exp(_randn(g, cols)), shift=_randn(g, cols))
        st["w"] = (1 + 0.2 * _randn(g, cols)).to(dtype) if case["affine"] else None
        st["b"] = (0.2 * _randn(g, cols)).to(dtype) if case["affine"] else None
    if op in ("norm_grad", "norm_train", "act_train"):
        st["dy"] = _rows(g, rows, cols, dtype, pad)
    if op == "norm_grad":   # what the forward pass left
        mean, rstd = zip(*(_stats(st["x"][r:r + 16384])[1:] for r in range(0, rows, 16384)))
        st["mean"], st["rstd"] = torch.cat(mean), torch.cat(rstd)
    return st


# ---------------------------------------------------------------------------------- plain forms
def _quantize(x, limit=None):
    x = x.float()
    if limit is not None:
        x = x.clamp(-limit, limit)
    amax = x.abs().amax(dim=-1)
    tiny = amax < 2.0 ** -118
    # the binary32 quotients, through 64 bits (correctly rounded either way)
    s = torch.where(tiny, torch.zeros_like(amax), (amax.double() / 127.0).float())
    inv = torch.where(tiny, torch.zeros_like(amax), (127.0 / amax.double()).float())
    return torch.round(x * inv[..., None]).to(torch.int8), s


def _values(codes, s):
    return codes.float() * s[:, None]


def _stats(x):
    x = x.float()
    mean = x.mean(dim=-1)
    d = x - mean[:, None]
    return d, mean, torch.rsqrt((d * d).mean(dim=-1) + EPS)


def _norm(st):
    d, mean, rstd = _stats(st["x"])
    y = d * rstd[:, None]
    if st["w"] is not None:
        y = y * st["w"].float() + st["b"].float()
    return y, mean, rstd


def _norm_grad(dy, x, mean, rstd, w):
    dy = dy.float()
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w.float()
    dx = rstd[:, None] * (g - g.mean(dim=-1, keepdim=True) - xh * (g * xh).mean(dim=-1, keepdim=True))
    # sums over all rows: in 64 bits
    return (dx,) if w is None else (dx, (dy * xh).sum(dim=0, dtype=torch.float64).float(), dy.sum(dim=0, dtype=torch.float64).float())


def _act(u, act):
    u = u.float()
    z = u if act == "silu" else 2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u * u * u)
    return u / (1 + torch.exp(-z))


def _act_grad(u, act):
    z = u if act == "silu" else 2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u * u * u)
    dz = 1.0 if act == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * u * u)
    s = 1 / (1 + torch.exp(-z))
    return s + u * s * (1 / (1 + torch.exp(z))) * dz


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "wgrad":
        x = _values(st["codes"], st["scales"]).bfloat16().float()   # the values as dequantize_int8 gives them
        return torch.matmul(st["dy"].float().t(), x).to(TYPES[c["out"]])
    dtype = TYPES[c["type"]]
    if op == "norm":
        return _norm(st)[0].to(dtype)
    if op == "norm_int8":
        codes, s = _quantize(_norm(st)[0])
        return _values(codes, s).bfloat16(), s
    if op == "norm_grad":
        dx, *rest = _norm_grad(st["dy"], st["x"], st["mean"], st["rstd"], st["w"])
        return (dx.to(dtype), *rest)
    if op == "norm_train":
        y, mean, rstd = _norm(st)
        dx, *rest = _norm_grad(st["dy"], _values(*_quantize(st["x"])), mean, rstd, st["w"])
        return (y.to(dtype), mean, rstd, dx.to(dtype), *rest)
    if op == "act_int8":
        codes, s = _quantize(_act(st["u"], c["act"]))
        return _values(codes, s).bfloat16(), s
    kept = _values(*_quantize(st["u"], LIMIT[c["act"]]))
    return _act(st["u"], c["act"]).to(dtype), (st["dy"].float() * _act_grad(kept, c["act"])).to(dtype)


# ---------------------------------------------------------------------------------- one pass
def _own(st):
    import mxfp4_microscaled_quantization_amd as mxq
    c = st["case"]
    op = c["op"]
    if op == "wgrad":
        return mxq.grad_weight_int8(st["dy"], st["codes"], st["scales"], out_dtype=TYPES[c["out"]])
    if op == "norm":
        return mxq.layer_norm(st["x"], st["w"], st["b"], eps=EPS)
    if op == "norm_int8":
        codes, s = mxq.quantize_layer_norm(st["x"], st["w"], st["b"], eps=EPS)
        return mxq.dequantize_int8(codes, s), s
    if op == "norm_grad":
        out = mxq.layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["w"])
        return out if st["w"] is not None else out[:1]
    if op == "norm_train":
        y, mean, rstd, codes, s = mxq.layer_norm(st["x"], st["w"], st["b"], eps=EPS, save="int8")
        out = mxq.layer_norm_backward(st["dy"], codes, mean, rstd, st["w"], x_scales=s)
        return (y, mean, rstd, *(out if st["w"] is not None else out[:1]))
    if op == "act_int8":
        codes, s = mxq.quantize_activation(st["u"], c["act"])
        return mxq.dequantize_int8(codes, s), s
    y, codes, s = mxq.activation(st["u"], c["act"], save="int8")
    return y, mxq.activation_backward(st["dy"], codes, s, c["act"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "wgrad":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * N + M * K + 4 * M + N * K * SIZE[case["out"]], "flops": 2 * M * N * K}
    rows, cols, b = case["rows"], case["cols"], SIZE[case["type"]]
    n = rows * cols
    if op.startswith("act"):
        return {"bytes": n * (b + 2) + 4 * rows if op == "act_int8" else n * 4 * b, "flops": n * (12 if op == "act_int8" else 32)}
    vectors = (2 * b * cols if case["affine"] else 0) if op != "norm_grad" else (b * cols if case["affine"] else 0)
    sums = 8 * cols if case["affine"] else 0
    if op == "norm":
        return {"bytes": 2 * n * b + vectors, "flops": 8 * n}
    if op == "norm_int8":
        return {"bytes": n * (b + 2) + 4 * rows + vectors, "flops": 10 * n}
    if op == "norm_grad":
        return {"bytes": 3 * n * b + 8 * rows + vectors + sums, "flops": 14 * n}
    return {"bytes": 4 * n * b + 8 * rows + vectors + sums, "flops": 24 * n}


# ---------------------------------------------------------------------------------- 64 bits
def _exact_rule(v, limit=None):
    """The values that the codes of the last axis stand for, and the scale: the two quotients, the product and the code each rounded once."""
    v = v.double()
    if limit is not None:
        v = torch.minimum(torch.maximum(v, torch.full_like(v, -limit)), torch.full_like(v, limit))
    top = v.abs().max(dim=-1).values
    alive = top >= math.ldexp(1.0, -118)
    one = torch.ones_like(top)
    step = torch.where(alive, top / 127.0, 0 * one).to(torch.float32)
    inv = torch.where(alive, 127.0 / torch.where(alive, top, one), 0 * one).to(torch.float32)
    # a product of two binary32 values is exact in 64 bits, and is rounded to 24 once
    code = (v * inv.double().unsqueeze(-1)).to(torch.float32).double()
    low = torch.floor(code)
    part = code - low
    up = (part > 0.5) | ((part == 0.5) & (torch.remainder(low, 2.0) == 1.0))
    return torch.where(up, low + 1, low) * step.double().unsqueeze(-1), step


def _exact_codes(y):
    """8-bit values of numbers that are not binary32 ones."""
    step = y.abs().max(dim=-1).values / 127.0
    return torch.round(y / step.unsqueeze(-1)) * step.unsqueeze(-1), step


def _exact_act(u, act):
    """The activation and its derivative, by tanh: logistic(2 t) = (1 + tanh(t)) / 2."""
    if act == "silu":
        t, dt = 0.5 * u, torch.full_like(u, 0.5)
    else:
        k = math.sqrt(2.0 / math.pi)
        t, dt = k * (u + 0.044715 * u ** 3), k * (1.0 + 3 * 0.044715 * u ** 2)
    h = torch.tanh(t)
    return 0.5 * u * (1.0 + h), 0.5 * (1.0 + h) + 0.5 * u * (1.0 - h * h) * dt


def _exact_slice(st, r, n):
    """Outputs of n rows from r, and their part of the sums over rows."""
    c = st["case"]
    op = c["op"]
    if op.startswith("act"):
        y, _ = _exact_act(st["u"][r:r + n].double(), c["act"])
        if op == "act_int8":
            v, s = _exact_codes(y)
            return [v.float(), s], []
        kept, _ = _exact_rule(st["u"][r:r + n], LIMIT[c["act"]])
        return [y, st["dy"][r:r + n].double() * _exact_act(kept, c["act"])[1]], []
    x = st["x"][r:r + n].double()
    w = None if st["w"] is None else st["w"].double()
    if op == "norm_grad":
        mean, rstd = st["mean"][r:r + n].double(), st["rstd"][r:r + n].double()
    else:
        mean = x.sum(dim=-1) / x.shape[-1]
        rstd = 1.0 / torch.sqrt(torch.var(x, dim=-1, unbiased=False) + EPS)
    outs = []
    if op != "norm_grad":
        y = (x - mean.unsqueeze(-1)) * rstd.unsqueeze(-1)
        y = y if w is None else torch.addcmul(st["b"].double(), y, w)
        if op == "norm_int8":
            v, s = _exact_codes(y)
            return [v.float(), s], []
        outs.append(y)
        if op == "norm":
            return outs, []
        outs += [mean, rstd]
        x, _ = _exact_rule(st["x"][r:r + n])
    dy = st["dy"][r:r + n].double()
    xh = (x - mean.unsqueeze(-1)) * rstd.unsqueeze(-1)
    g = dy if w is None else dy * w
    C = g.shape[-1]
    outs.append((g - g.sum(dim=-1, keepdim=True) / C - xh * ((g * xh).sum(dim=-1, keepdim=True) / C)) * rstd.unsqueeze(-1))
    return outs, [] if w is None else [torch.einsum("rc,rc->c", dy, xh), dy.sum(dim=0)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "wgrad":
        out = torch.zeros((case["N"], case["K"]), dtype=torch.float64, device=DEV)
        for r in range(0, case["M"], 8192):
            # a code times a binary32 scale is exact in 64 bits
            x = (st["codes"][r:r + 8192].double() * st["scales"][r:r + 8192].double()[:, None]).to(torch.float32).to(torch.bfloat16)
            out += st["dy"][r:r + 8192].double().t() @ x.double()
        return out
    outs, sums, n = None, None, 8192
    for r in range(0, case["rows"], n):
        o, s = _exact_slice(st, r, n)
        if outs is None:
            outs, sums = [[x] for x in o], s
        else:
            for have, x in zip(outs, o):
                have.append(x)
            sums = [a + x for a, x in zip(sums, s)]
    got = [torch.cat(x) for x in outs] + sums
    return got[0] if case["op"] == "norm" else tuple(got)
