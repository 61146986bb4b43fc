"""Workloads of the 8-bit operators: the row quantizer, the 8-bit product with token and channel
scales (separate and with the activations quantized by the call), and the norm and rotation of
queries and keys, plain and quantized.

`own` false: elementary torch operations; true: the library's entry points."""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a 5120-wide transformer, before a linear layer: latency
        {"name": "quant_token", "op": "quantize", "rows": 1, "cols": 5120, "type": "bf16", "pad": 0},
        # every token of the Wan2.2 FFN-down input
        {"name": "quant_wan_ffn_down", "op": "quantize", "rows": 75600, "cols": 13824, "type": "bf16", "pad": 0},
        # one token through the FFN-up weights: the weights' bytes count
        {"name": "gemm_token", "op": "gemm", "M": 1, "K": 5120, "N": 13824, "out": "bf16", "bias": True, "pad": 0},
        # a small batch of tokens through the FFN-down weights, long K
        {"name": "gemm_batch48", "op": "gemm", "M": 48, "K": 13824, "N": 5120, "out": "bf16", "bias": False, "pad": 0},
        # ragged everything: rows inside a wider buffer, K no multiple of a window, odd N, binary32 out
        {"name": "gemm_ragged", "op": "gemm", "M": 1001, "K": 1360, "N": 2051, "out": "fp32", "bias": True, "pad": 32},
        # the Wan2.2 FFN-up layer
        {"name": "gemm_wan_ffn_up", "op": "gemm", "M": 75600, "K": 5120, "N": 13824, "out": "bf16", "bias": True, "pad": 0},
        # one token, unquantized, through the FFN-down weights
        {"name": "fused_token", "op": "fused", "M": 1, "K": 13824, "N": 5120, "type": "bf16", "out": "bf16", "bias": True, "pad": 0},
        # one image's tokens through a QKV projection
        {"name": "fused_qkv", "op": "fused", "M": 3584, "K": 5120, "N": 15360, "type": "bf16", "out": "bf16", "bias": True, "pad": 0},
        # one new token with grouped heads, rotation by halves, position from an array
        {"name": "qk_token", "op": "qk", "T": 1, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "style": "halves", "type": "bf16",
         "table": 8192, "int8": False},
        # the queries and keys of every Wan2.2 latent token
        {"name": "qk_wan", "op": "qk", "T": 75600, "Hq": 40, "Hk": 40, "D": 128, "R": 128, "style": "interleaved",
         "type": "bf16", "table": 75600, "int8": False},
        # ragged: odd token count, 96-wide heads of which 64 are rotated, binary32, 8-bit out (and its dequantization)
        {"name": "qk_int8_ragged", "op": "qk", "T": 77, "Hq": 12, "Hk": 3, "D": 96, "R": 64, "style": "halves", "type": "fp32",
         "table": 4096, "int8": True},
        # a batch of 16 FLUX images' tokens, 8-bit queries and keys (and their dequantization)
        {"name": "qk_int8_flux", "op": "qk", "T": 57344, "Hq": 24, "Hk": 24, "D": 128, "R": 128, "style": "interleaved",
         "type": "bf16", "table": 3584, "int8": True},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)


def draw(rng):
    op = rng.choice(["quantize", "gemm", "fused", "qk", "qk"])
    pad = rng.choice([0, 0, 16, 48])
    if op == "quantize":
        rows, cols = _log(rng, 1, 80000), _log(rng, 16, 14000, 16)
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "bf16", "fp32"]), "pad": pad}
    if op in ("gemm", "fused"):
        K, N = _log(rng, 64, 14000, 16), _log(rng, 16, 14000)
        most = int(min(40000 if op == "gemm" else 8000, 5e12 / (2 * K * N)))   # tokens
        c = {"op": op, "M": _log(rng, 1, most), "K": K, "N": N,
             "out": rng.choice(["bf16", "bf16", "fp32"]), "bias": rng.random() < 0.5, "pad": pad}
        if op == "fused":
            c["type"] = rng.choice(["bf16", "bf16", "fp32"])
        return c
    d = rng.choice([64, 80, 96, 128, 128, 256])
    hk = rng.choice([1, 2, 3, 8, 24])
    return {"op": op, "T": _log(rng, 1, 30000), "Hq": hk * rng.choice([1, 1, 2, 4] if hk < 24 else [1]), "Hk": hk, "D": d,
            "R": rng.choice([d, d, d // 16 * 8]), "style": rng.choice(["interleaved", "halves"]), "type": rng.choice(["bf16", "bf16", "fp32"]),
            "table": _log(rng, 64, 40000), "int8": rng.random() < 0.5}


# ---------------------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _padded(t, pad):
    """The same values as rows of a buffer `pad` columns wider (a view with that row pitch)."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _activations(g, rows, cols, dtype):
    """N(0, 1) times a scale for each channel ~ LogNormal(0, 1): outlier channels."""
    ch = torch.exp(_randn(g, cols))
    out = torch.empty((rows, cols), dtype=dtype, device=DEV)
    for r in range(0, rows, 16384):   # in slices: the binary32 draw of a large case stays small
        out[r:r + 16384] = _randn(g, min(16384, rows - r), cols) * ch
    return out


def _codes(x):
    """8-bit codes and scales of an operand that the program has in hand."""
    q = torch.empty(x.shape, dtype=torch.int8, device=DEV)
    s = torch.empty(x.shape[0], dtype=torch.float32, device=DEV)
    for r in range(0, x.shape[0], 16384):
        q[r:r + 16384], s[r:r + 16384] = _quantize(x[r:r + 16384])
    return q, s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, st = case["op"], {"case": case}
    if op == "quantize":
        st["x"] = _padded(_activations(g, case["rows"], case["cols"], TYPES[case["type"]]), case["pad"])
    elif op in ("gemm", "fused"):
        M, N, K = case["M"], case["N"], case["K"]
        a = _activations(g, M, K, TYPES[case.get("type", "bf16")])
        st["w"], st["ws"] = _codes(_randn(g, N, K) * 0.02)
        if op == "gemm":
            q, st["as"] = _codes(a)
            st["a"] = _padded(q, case["pad"])
            st["w"] = _padded(st["w"], case["pad"])
        else:
            st["a"] = _padded(a, case["pad"])
        st["bias"] = _randn(g, N) * 0.5 if case["bias"] else None
    else:
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        # the output of the QKV projection: queries, keys and values side by side in a row
        qkv = _activations(g, T, (Hq + 2 * Hk) * D, TYPES[case["type"]])
        st["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        st["wq"], st["wk"] = ((1 + 0.2 * _randn(g, D)).to(TYPES[case["type"]]) for _ in range(2))
        P, R = case["table"], case["R"]
        freq = 10000.0 ** (-torch.arange(R // 2, device=DEV, dtype=torch.float64) * 2 / R)
        ang = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * freq
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["pos"] = torch.randint(0, P, (T,), generator=g, device=DEV)
    return st


# ---------------------------------------------------------------------------------- plain forms
def _quantize(x):
    x = x.float()
    amax = x.abs().amax(dim=-1)
    tiny = amax < 2.0 ** -118
    # the binary32 quotients, through 64 bits (correctly rounded either way)
    s = torch.where(tiny, torch.zeros_like(amax), (amax.double() / 127.0).float())
    inv = torch.where(tiny, torch.zeros_like(amax), (127.0 / amax.double()).float())
    return torch.round(x * inv[..., None]).to(torch.int8), s


def _product(q, s, w, ws, bias, dtype):
    # sums of 8-bit products pass 2^24: in 64 bits
    v = torch.matmul(q.double(), w.double().t())
    v *= s.double()[:, None]
    v *= ws.double()[None, :]
    if bias is not None:
        v += bias.double()
    return v.to(dtype)


def _norm_rope(x, w, cos, sin, R, style, eps=1e-6):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + eps) * w.float()
    rot, rest = y[..., :R], y[..., R:]
    c, s = cos[:, None, :], sin[:, None, :]
    if style == "interleaved":
        y0, y1 = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((y0 * c - y1 * s, y1 * c + y0 * s), dim=-1).flatten(-2)
    else:
        y0, y1 = rot[..., :R // 2], rot[..., R // 2:]
        rot = torch.cat((y0 * c - y1 * s, y1 * c + y0 * s), dim=-1)
    return torch.cat((rot, rest), dim=-1)


def _plain(st):
    c = st["case"]
    if c["op"] == "quantize":
        return _quantize(st["x"])
    if c["op"] == "gemm":
        return _product(st["a"], st["as"], st["w"], st["ws"], st["bias"], TYPES[c["out"]])
    if c["op"] == "fused":
        q, s = _quantize(st["a"])
        return _product(q, s, st["w"], st["ws"], st["bias"], TYPES[c["out"]])
    cos, sin = st["cos"][st["pos"]], st["sin"][st["pos"]]
    q = _norm_rope(st["q"], st["wq"], cos, sin, c["R"], c["style"])
    k = _norm_rope(st["k"], st["wk"], cos, sin, c["R"], c["style"])
    if not c["int8"]:
        return q.to(TYPES[c["type"]]), k.to(TYPES[c["type"]])
    (qc, qs), (kc, ks) = _quantize(q), _quantize(k)
    return (qc.float() * qs[..., None]).bfloat16(), qs, (kc.float() * ks[..., None]).bfloat16(), ks


# ---------------------------------------------------------------------------------- one pass
def _own(st):
    import mxfp4_microscaled_quantization_amd as mxq
    c = st["case"]
    if c["op"] == "quantize":
        return mxq.quantize_int8(st["x"])
    if c["op"] == "gemm":
        return mxq.gemm_w8a8(st["a"], st["as"], st["w"], st["ws"], bias=st["bias"], out_dtype=TYPES[c["out"]])
    if c["op"] == "fused":
        return mxq.gemm_w8a8_fused(st["a"], st["w"], st["ws"], bias=st["bias"], out_dtype=TYPES[c["out"]])
    args = (st["q"], st["k"], st["wq"], st["wk"], st["cos"], st["sin"])
    if not c["int8"]:
        return mxq.qk_norm_rope(*args, positions=st["pos"], eps=1e-6, style=c["style"])
    qc, qs, kc, ks = mxq.quantize_qk_norm_rope(*args, positions=st["pos"], eps=1e-6, style=c["style"])
    D = c["D"]
    q = mxq.dequantize_int8(qc.view(-1, D), qs.view(-1)).view(qc.shape)
    k = mxq.dequantize_int8(kc.view(-1, D), ks.view(-1)).view(kc.shape)
    return q, qs, k, ks


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (SIZE[case["type"]] + 1) + 4 * case["rows"], "flops": 2 * n}
    if op in ("gemm", "fused"):
        M, N, K = case["M"], case["N"], case["K"]
        a = M * K * SIZE[case["type"]] if op == "fused" else M * K + 4 * M
        return {"bytes": a + N * K + 4 * N * (2 if case["bias"] else 1) + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    T, H, D, b = case["T"], case["Hq"] + case["Hk"], case["D"], SIZE[case["type"]]
    n = T * H * D
    # the table rows that the tokens name, positions, and the outputs that run() returns
    tables = 8 * min(T, case["table"]) * (case["R"] // 2) + 8 * T
    return {"bytes": n * b + (n * 2 + 4 * T * H if case["int8"] else n * b) + tables, "flops": 8 * n}


# ---------------------------------------------------------------------------------- 64 bits
def _exact_rule(v32):
    """Codes and scale of the last axis from the rule itself: the two quotients, the product and the code each rounded once."""
    v = v32.double()
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
    return torch.where(up, low + 1, low), step


def _exact_turn(x, w, cos, sin, R, style, eps=1e-6):
    x = x.double()
    norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    y = x / torch.sqrt(norm ** 2 / x.shape[-1] + eps) * w.double()
    out = y.clone()
    first = torch.arange(0, R, 2, device=DEV) if style == "interleaved" else torch.arange(R // 2, device=DEV)
    second = first + (1 if style == "interleaved" else R // 2)
    z = torch.complex(y[..., first], y[..., second]) * torch.complex(cos.double(), sin.double())[:, None, :]
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q = torch.empty(st["x"].shape, dtype=torch.int8, device=DEV)
        s = torch.empty(st["x"].shape[0], dtype=torch.float32, device=DEV)
        for r in range(0, q.shape[0], 4096):
            c, s[r:r + 4096] = _exact_rule(st["x"][r:r + 4096])
            q[r:r + 4096] = c.to(torch.int8)
        return q, s
    if op in ("gemm", "fused"):
        out = torch.empty((case["M"], case["N"]), dtype=torch.float64, device=DEV)
        w = st["w"].double() * st["ws"].double()[:, None]
        for r in range(0, case["M"], 8192):
            a = st["a"][r:r + 8192]
            a, sa = _exact_rule(a) if op == "fused" else (a.double(), st["as"][r:r + 8192])
            out[r:r + 8192] = (a * sa.double()[:, None]) @ w.t()
            if st["bias"] is not None:
                out[r:r + 8192] += st["bias"].double()
        return out
    got = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        outs, steps = [], []
        for r in range(0, case["T"], 8192):
            p = st["pos"][r:r + 8192]
            y = _exact_turn(x[r:r + 8192], w, st["cos"][p], st["sin"][p], case["R"], case["style"])
            if case["int8"]:
                top = y.abs().max(dim=-1).values
                steps.append(top / 127.0)
                outs.append((torch.round(y / steps[-1].unsqueeze(-1)) * steps[-1].unsqueeze(-1)).float())
            else:
                outs.append(y)
        got.append(torch.cat(outs))
        if case["int8"]:
            got.append(torch.cat(steps))
    return tuple(got)
