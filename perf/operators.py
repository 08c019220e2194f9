"""Timing cases of the 8-bit feed-forward operators: RMS norm with the residual's addition, gated
activation, and the 2:4 product with its epilogue, each in a plain form and as the library's call.

`own` says which of the two `run` computes.  Activations are tokens x features.  8-bit values are
e4m3 with one fp32 scale per row (per token, or per output feature of a weight): a row y is held
as q = e4m3(y / s) with s = max(max|y| / 448, the smallest normal fp32), so that y is about q s.

  norm    h = x + residual;  y = h / sqrt(mean(h^2) + eps) * weight
  gate    a = act(gate) * up            (without `up`: act(gate))
  linear  Y = act(sw[m] sx[n] sum_k W[m][k] X[n][k] + bias[m]) + residual[n][m], W 2:4-sparse
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f8": F8}
BYTES = {"bf16": 2, "f32": 4, "f8": 1}
TINY = torch.finfo(torch.float32).tiny
EPS = 1e-6


def listed():
    return [
        # one token through the norm ahead of a layer, 8-bit output for the product behind it: latency
        {"name": "norm_1_token", "op": "norm", "tokens": 1, "width": 4096, "stream": "bf16", "out": "f8",
         "residual": True, "pad": 0},
        # a long prompt's norm, bf16 stream, 8-bit output
        {"name": "norm_prompt", "op": "norm", "tokens": 8192, "width": 8192, "stream": "bf16", "out": "f8",
         "residual": True, "pad": 0},
        # a final norm: an fp32 stream with padded rows and an odd width, bf16 output, no residual
        {"name": "norm_odd", "op": "norm", "tokens": 1571, "width": 1003, "stream": "f32", "out": "bf16",
         "residual": False, "pad": 5},
        # a few tokens of a decoding batch between the two feed-forward products
        {"name": "gate_4_tokens", "op": "gate", "tokens": 4, "width": 11264, "stream": "bf16", "out": "f8",
         "act": "silu", "up": True, "pad": 0},
        # a prompt's gated activation, 8-bit output
        {"name": "gate_prompt", "op": "gate", "tokens": 4096, "width": 8192, "stream": "bf16", "out": "f8",
         "act": "silu", "up": True, "pad": 0},
        # an odd width in fp32, GELU gate, bf16 output
        {"name": "gate_odd", "op": "gate", "tokens": 777, "width": 2051, "stream": "f32", "out": "bf16",
         "act": "gelu", "up": True, "pad": 3},
        # one token through a square projection that adds to the residual stream
        {"name": "linear_1_token", "op": "linear", "tokens": 1, "rows": 4096, "width": 4096, "out": "bf16",
         "bias": False, "act": "none", "residual": True},
        # a decoding batch through stacked gate and up weights
        {"name": "linear_24_tokens", "op": "linear", "tokens": 24, "rows": 16384, "width": 4096, "out": "bf16",
         "bias": False, "act": "none", "residual": False},
        # a short prompt, rows and tokens off every tile, fp32 output with bias and GELU
        {"name": "linear_odd", "op": "linear", "tokens": 517, "rows": 1000, "width": 4032, "out": "f32",
         "bias": True, "act": "gelu", "residual": False},
        # an encoder's stacked projections: 4096 tokens of 768 features
        {"name": "linear_encoder", "op": "linear", "tokens": 4096, "rows": 2304, "width": 768, "out": "bf16",
         "bias": True, "act": "none", "residual": False},
        # a prompt through an up projection with bias and activation
        {"name": "linear_prompt", "op": "linear", "tokens": 4096, "rows": 8192, "width": 4096, "out": "bf16",
         "bias": True, "act": "silu", "residual": False},
        # the library's headline shape, adding to the residual stream
        {"name": "linear_8192", "op": "linear", "tokens": 8192, "rows": 8192, "width": 8192, "out": "bf16",
         "bias": False, "act": "none", "residual": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "gate", "linear", "linear"])
    tokens = rng.choice([1, _spread(rng, 1, 64), _spread(rng, 1, 8192), _spread(rng, 64, 8192)])
    if op == "linear":
        return {"op": op, "tokens": tokens, "rows": _spread(rng, 32, 8192), "width": 64 * _spread(rng, 1, 128),
                "out": rng.choice(["bf16", "bf16", "f32"]), "bias": rng.random() < 0.5,
                "act": rng.choice(["none", "relu", "gelu", "silu"]), "residual": rng.random() < 0.5}
    case = {"op": op, "tokens": tokens, "width": _spread(rng, 64, 8192), "stream": rng.choice(["bf16", "bf16", "f32"]),
            "out": rng.choice(["f8", "f8", "bf16", "f32"]), "pad": rng.choice([0, 0, rng.randint(1, 17)])}
    if case["stream"] == "f32":
        case["tokens"] = min(tokens, 4096)
    if rng.random() < 0.5:
        case["width"] = max(64, case["width"] // 64 * 64)
    if op == "norm":
        case["residual"] = rng.random() < 0.7
    else:
        case["act"] = rng.choice(["silu", "gelu", "relu", "none"])
        case["up"] = rng.random() < 0.75
    return case


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, tokens, width, pad, dtype):
    """Rows of a wider buffer (`pad` more elements a row): N(0, 1) with a few features much larger, as in a
    residual stream."""
    full = _normal(g, tokens, width + pad)
    full[:, :: max(1, width // 7)] *= 8
    return full.to(dtype)[:, :width]


def _quantize(y):
    """Plain: rows of fp32 -> (e4m3, fp32 scale)."""
    s = (y.abs().amax(dim=1) / 448).clamp_min(TINY)
    return (y / s[:, None]).to(F8), s


def _pruned(g, rows, width):
    """N(0, 0.02^2) weights, the two smallest magnitudes of every four along a row dropped, as 8-bit rows."""
    w = (_normal(g, rows, width) * 0.02).reshape(rows, width // 4, 4)
    a, b, c, d = w.abs().unbind(dim=2)
    lo, hi = torch.minimum(a, b), torch.maximum(a, b)
    lo2, hi2 = torch.minimum(c, d), torch.maximum(c, d)
    third = torch.minimum(torch.maximum(lo, lo2), torch.minimum(hi, hi2))   # third largest of the four
    w = torch.where(w.abs() > third[:, :, None], w, torch.zeros_like(w))
    return _quantize(w.reshape(rows, width))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, n = case["op"], case["tokens"]
    st = dict(case)
    if op == "norm":
        dt = TYPES[case["stream"]]
        st["x"] = _rows(g, n, case["width"], case["pad"], dt)
        st["weight"] = 1 + 0.1 * _normal(g, case["width"])
        st["r"] = _rows(g, n, case["width"], case["pad"], dt) if case["residual"] else None
    elif op == "gate":
        w, dt = case["width"], TYPES[case["stream"]]
        both = _rows(g, n, 2 * w if case["up"] else w, case["pad"], dt)
        st["gate"], st["upv"] = both[:, :w], both[:, w:] if case["up"] else None   # one product's two halves
    else:
        m, k = case["rows"], case["width"]
        st["wq"], st["ws"] = _pruned(g, m, k)
        st["xq"], st["xs"] = _quantize(_rows(g, n, k, 0, torch.float32))
        st["b"] = 0.1 * _normal(g, m) if case["bias"] else None
        st["r"] = _normal(g, n, m).to(TYPES[case["out"]]) if case["residual"] else None
        if own:   # the weight as a program keeps it: compressed once, when it is loaded
            import structured_sparse_gemm_prune24_amd as p24
            st["w"] = p24.compress_f8(st["wq"].float() * st["ws"][:, None])
            st["x8"] = p24.Quantized8(st["xq"], st["xs"])
    return st


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * (0.5 + 0.5 * torch.erf(z * math.sqrt(0.5)))
    return z


def _give(y, out):
    if out == "f8":
        q, s = _quantize(y)
        return {"y": q, "scale": s}
    return {"y": y.to(TYPES[out])}


def _own(st):
    import structured_sparse_gemm_prune24_amd as p24
    out = TYPES[st["out"]]
    if st["op"] == "linear":
        return {"y": p24.spmm24_f8(st["w"], st["x8"], out_dtype=out, bias=st["b"], act=st["act"], residual=st["r"])}
    if st["op"] == "norm":
        y, h = p24.rms_norm(st["x"], st["weight"], residual=st["r"], eps=EPS, out_dtype=out)
    else:
        y, h = p24.gated_act(st["gate"], st["upv"], act=st["act"], out_dtype=out), None
    got = {"y": y.values, "scale": y.scale} if out == F8 else {"y": y}
    return got if h is None else {**got, "h": h}


def run(st):
    if own:
        return _own(st)
    if st["op"] == "norm":
        h = st["x"].float() if st["r"] is None else st["x"].float() + st["r"].float()
        y = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS) * st["weight"]
        got = _give(y, st["out"])
        return got if st["r"] is None else {**got, "h": h.to(st["x"].dtype)}
    if st["op"] == "gate":
        a = _act(st["gate"].float(), st["act"])
        return _give(a if st["upv"] is None else a * st["upv"].float(), st["out"])
    z = st["xq"].float() @ st["wq"].float().t()
    z = z * (st["xs"][:, None] * st["ws"])
    if st["b"] is not None:
        z = z + st["b"]
    z = _act(z, st["act"])
    if st["r"] is not None:
        z = z + st["r"].float()
    return {"y": z.to(TYPES[st["out"]])}


def exact(case, seed):
    """From the definitions in fp64; 8-bit values are the unrounded y / s."""
    st = prepare(case, seed)
    d = torch.float64

    def act(z):
        if case["act"] == "silu":
            return z * torch.sigmoid(z)
        if case["act"] == "gelu":
            return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
        return torch.where(z > 0, z, torch.zeros_like(z)) if case["act"] == "relu" else z

    if case["op"] == "linear":
        z = torch.mm(st["xq"].to(d) * st["xs"].to(d).unsqueeze(1), (st["wq"].to(d) * st["ws"].to(d).unsqueeze(1)).T)
        z = act(z + st["b"].to(d) if case["bias"] else z)
        return {"y": z + st["r"].to(d) if case["residual"] else z}
    extra = {}
    if case["op"] == "norm":
        y = st["x"].to(d)
        if case["residual"]:
            y = y + st["r"].to(d)
            extra["h"] = y
        y = y * torch.rsqrt(y.square().sum(1, keepdim=True) / case["width"] + EPS) * st["weight"].to(d)
    else:
        y = act(st["gate"].to(d))
        y = y * st["upv"].to(d) if case["up"] else y
    if case["out"] != "f8":
        return {"y": y, **extra}
    s = torch.clamp(torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 448, min=TINY)
    return {"y": y / s.unsqueeze(1), "scale": s, **extra}


def work(case):
    n, w, out = case["tokens"], case["width"], BYTES[case["out"]]
    if case["op"] == "linear":
        m = case["rows"]
        # half of the weights are kept, one byte and two position bits each
        byts = m * w // 2 + m * w // 8 + 4 * m + n * w + 4 * n + n * m * out
        byts += 4 * m * case["bias"] + n * m * out * case["residual"]
        return {"bytes": byts, "flops": n * m * w}
    stream = BYTES[case["stream"]]
    scale = 4 * n * (case["out"] == "f8")
    if case["op"] == "norm":
        return {"bytes": n * w * (stream * (3 if case["residual"] else 1) + out) + 4 * w + scale, "flops": 5 * n * w}
    return {"bytes": n * w * (stream * (2 if case["up"] else 1) + out) + scale, "flops": 10 * n * w}
