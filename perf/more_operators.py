"""Timing cases of the expert operators (routing, 2:4 products grouped by expert, combination) and of
the dense 8-bit product with a scale for each block of 128, each in a plain form and as the
library's calls.

`own` says which of the two `run` computes.  Activations are tokens x features; 8-bit values are e4m3.

  route    the k best experts of a token by its logits (ties to the lower expert; -inf: not open), their
           weights, and the rows sorted by expert: offsets, the token of a row, the row of a slot
  experts  Y[p] = act(sw[e] sx[r] W[e] X[r] + bias[e]) for the rows p of expert e, r = tokens[p] or p;
           W 2:4-sparse, one scale per feature and per row of X
  combine  y[t] = residual[t] + sum_j weights[t][j] Z[positions[t][j]]
  block    Y = act(W a + bias) + residual with a = act(x) up quantised by blocks of 128 along a token,
           W by blocks of 128 x 128; a block y is held as q = e4m3(y / s), s = max(max|y| / 448, 2^-126)
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
TINY = torch.finfo(torch.float32).tiny


def listed():
    return [
        # the router of one decoded token: latency
        {"name": "route_1_token", "op": "route", "tokens": 1, "experts": 128, "k": 8, "logits": "bf16",
         "score": "softmax", "normalize": True, "bias": False, "padded": 0},
        # a padded prompt batch through a sigmoid router with a selection bias
        {"name": "route_prompt", "op": "route", "tokens": 8192, "experts": 256, "k": 8, "logits": "f32",
         "score": "sigmoid", "normalize": True, "bias": True, "padded": 251},
        # one token through its 8 experts' stacked gate and up weights
        {"name": "experts_1_token", "op": "experts", "tokens": 1, "experts": 128, "k": 8, "rows": 2048,
         "width": 4096, "gather": True, "out": "bf16", "bias": False, "act": "none", "padded": 0},
        # a decoding batch that reaches every expert
        {"name": "experts_64_tokens", "op": "experts", "tokens": 64, "experts": 32, "k": 4, "rows": 4096,
         "width": 4096, "gather": True, "out": "bf16", "bias": False, "act": "none", "padded": 0},
        # a padded batch through few experts' down weights, fp32 output, sizes off every tile
        {"name": "experts_odd", "op": "experts", "tokens": 1571, "experts": 7, "k": 2, "rows": 1000,
         "width": 1088, "gather": False, "out": "f32", "bias": True, "act": "gelu", "padded": 40},
        # a prompt through the stacked gate and up weights of 64 experts
        {"name": "experts_prompt", "op": "experts", "tokens": 4096, "experts": 64, "k": 8, "rows": 4096,
         "width": 2048, "gather": True, "out": "bf16", "bias": False, "act": "none", "padded": 0},
        # a few tokens' rows back into their tokens
        {"name": "combine_8_tokens", "op": "combine", "tokens": 8, "k": 8, "width": 4096, "out": "bf16",
         "residual": True, "padded": 0},
        # a prompt's
        {"name": "combine_prompt", "op": "combine", "tokens": 4096, "k": 8, "width": 4096, "out": "bf16",
         "residual": True, "padded": 100},
        # one token through a dense square projection that adds to the residual stream
        {"name": "block_1_token", "op": "block", "tokens": 1, "rows": 4096, "width": 4096, "stream": "bf16",
         "up": False, "quant_act": "none", "out": "bf16", "bias": False, "act": "none", "residual": True},
        # a short prompt in fp32, rows, tokens and width off every tile
        {"name": "block_odd", "op": "block", "tokens": 517, "rows": 1000, "width": 4048, "stream": "f32",
         "up": False, "quant_act": "none", "out": "f32", "bias": True, "act": "silu", "residual": False},
        # a prompt's gated activation and down projection, adding to the residual stream
        {"name": "block_gated", "op": "block", "tokens": 2048, "rows": 4096, "width": 11264, "stream": "bf16",
         "up": True, "quant_act": "silu", "out": "bf16", "bias": False, "act": "none", "residual": True},
        # the library's headline shape
        {"name": "block_8192", "op": "block", "tokens": 8192, "rows": 8192, "width": 8192, "stream": "bf16",
         "up": False, "quant_act": "none", "out": "bf16", "bias": False, "act": "none", "residual": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "combine", "block", "block"])
    tokens = rng.choice([1, _spread(rng, 1, 64), _spread(rng, 1, 4096), _spread(rng, 64, 4096)])
    padded = rng.choice([0, 0, tokens // rng.randint(2, 40)])
    act = rng.choice(["none", "relu", "gelu", "silu"])
    if op == "route":
        score = rng.choice(["softmax", "sigmoid"])
        experts = rng.choice([8, 64, 128, _spread(rng, 2, 512)])
        return {"op": op, "tokens": tokens * rng.choice([1, 2]), "experts": experts, "k": rng.randint(1, min(16, experts)),
                "logits": rng.choice(["bf16", "f32"]), "score": score, "normalize": rng.random() < 0.6,
                "bias": score == "sigmoid" and rng.random() < 0.6, "padded": padded}
    if op == "combine":
        return {"op": op, "tokens": tokens, "k": rng.randint(1, 8), "width": _spread(rng, 64, 4096),
                "out": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.6, "padded": padded}
    if op == "experts":
        rows, width, experts = _spread(rng, 32, 4096), 64 * _spread(rng, 1, 64), _spread(rng, 2, 128)
        return {"op": op, "tokens": tokens, "experts": max(2, min(experts, (1 << 29) // (rows * width))),
                "k": rng.randint(1, 2 if experts < 8 else 8), "rows": rows, "width": width, "gather": rng.random() < 0.6,
                "out": rng.choice(["bf16", "bf16", "f32"]), "bias": rng.random() < 0.4, "act": act, "padded": padded}
    out = rng.choice(["bf16", "bf16", "f32"])
    # an fp32 output shows single 8-bit roundings: there the quantised values are the stream's own
    gated = out == "bf16" and rng.random() < 0.4
    return {"op": op, "tokens": tokens * rng.choice([1, 2]), "rows": _spread(rng, 16, 8192), "width": 16 * _spread(rng, 1, 512),
            "stream": rng.choice(["bf16", "bf16", "f32"]), "up": gated, "quant_act": rng.choice(["silu", "gelu"]) if gated else "none",
            "out": out, "bias": rng.random() < 0.4, "act": act, "residual": rng.random() < 0.5}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _stream(g, tokens, width):
    """N(0, 1) with a few features much larger, as in a residual stream."""
    x = _normal(g, tokens, width)
    x[:, :: max(1, width // 7)] *= 8
    return x


def _logits(g, case):
    """Router logits: some experts are more popular; the last `padded` tokens are open to none."""
    l = 1.5 * _normal(g, case["tokens"], case["experts"]) + 0.7 * _normal(g, case["experts"])
    l[case["tokens"] - case["padded"]:] = -math.inf
    return l


def _sorted(experts, count):
    """(offsets, tokens, positions) of the rows sorted by expert, from the chosen experts [tokens, k] (-1: none)."""
    flat = experts.reshape(-1).long()
    key = torch.where(flat < 0, count, flat)
    order = torch.sort(key, stable=True).indices
    ids = torch.arange(count, device=flat.device)
    counts = (flat[:, None] == ids).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rows = torch.arange(flat.numel(), device=flat.device)
    tokens = torch.where(rows < offsets[-1], order // experts.shape[1], -1)
    positions = torch.empty_like(flat)
    positions[order] = rows
    positions = torch.where(flat < 0, -1, positions).reshape(experts.shape)
    return offsets.int(), tokens.int(), positions.int()


def _best(score, logits, k):
    """The k best experts of each token, -1 where none is open; ties to the lower expert."""
    closed = logits == -math.inf
    top = torch.sort(torch.where(closed, -math.inf, score), dim=1, descending=True, stable=True).indices[:, :k]
    return torch.where(closed.gather(1, top), -1, top), top


def _scales(y, dims):
    top = y.abs().amax(dim=dims)
    return (top / torch.full_like(top, 448)).clamp_min(TINY)   # a quotient: by a number torch multiplies with its reciprocal


def _quantize_rows(y):
    """fp32 tokens x width -> e4m3, fp32 scales [tokens], one a row."""
    s = _scales(y, 1)
    return (y / s[:, None]).to(F8), s


def _quantize_blocks(y, tall):
    """e4m3 values and fp32 scales of blocks `tall` x 128: [rows / tall, blocks]."""
    n, w = y.shape
    p = torch.nn.functional.pad(y, (0, -w % 128, 0, -n % tall))
    p = p.reshape(p.shape[0] // tall, tall, p.shape[1] // 128, 128)
    s = _scales(p, (1, 3))
    q = (p / s[:, None, :, None]).to(F8)
    return q.reshape(p.shape[0] * tall, -1)[:n, :w].contiguous(), s


def _pruned(g, rows, width):
    """N(0, 0.02^2) weights, the two smallest magnitudes of every four along a row dropped, as 8-bit rows."""
    w = (_normal(g, rows, width) * 0.02).reshape(rows, width // 4, 4)
    a, b, c, d = w.abs().unbind(dim=2)
    lo, hi = torch.minimum(a, b), torch.maximum(a, b)
    lo2, hi2 = torch.minimum(c, d), torch.maximum(c, d)
    third = torch.minimum(torch.maximum(lo, lo2), torch.minimum(hi, hi2))
    w = torch.where(w.abs() > third[:, :, None], w, torch.zeros_like(w))
    return _quantize_rows(w.reshape(rows, width))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    n = case["tokens"]
    if case["op"] == "route":
        st["l"] = _logits(g, case).to(TYPES[case["logits"]])
        st["b"] = 0.1 * _normal(g, case["experts"]) if case["bias"] else None
        return st
    if case["op"] == "combine":
        rows = (n - case["padded"]) * case["k"]
        st["z"] = _normal(g, n * case["k"], case["width"]).to(TYPES[case["out"]])
        perm = torch.randperm(rows, generator=g, device="cuda").int()
        st["p"] = torch.cat([perm, perm.new_full((n * case["k"] - rows,), -1)]).reshape(n, case["k"])
        w = torch.rand(n, case["k"], generator=g, device="cuda")
        st["w"] = torch.where(st["p"] < 0, 0, w / w.sum(1, keepdim=True))
        st["r"] = _normal(g, n, case["width"]).to(TYPES[case["out"]]) if case["residual"] else None
        return st
    m, k = case["rows"], case["width"]
    if case["op"] == "experts":
        e = case["experts"]
        l = _logits(g, case)
        off, tok, _ = _sorted(_best(l, l, case["k"])[0], e)
        st["off"], st["tok"] = off, tok.clamp_min(0) if case["gather"] else None
        st["wq"], st["ws"] = torch.empty(e, m, k, device="cuda", dtype=F8), torch.empty(e, m, device="cuda")
        for i in range(e):
            st["wq"][i], st["ws"][i] = _pruned(g, m, k)
        st["xq"], st["xs"] = _quantize_rows(_stream(g, n if case["gather"] else n * case["k"], k))
        st["b"] = 0.1 * _normal(g, e, m) if case["bias"] else None
        # rows behind the last expert's stay as they were
        st["y"] = torch.zeros(n * case["k"], m, device="cuda", dtype=TYPES[case["out"]]) if case["padded"] else None
        counts = off[1:] - off[:-1]
        st["active"], st["cap"] = counts.nonzero()[:, 0], int(counts.max())   # of this routing
        if own:   # the weights as a program keeps them: compressed once, when they are loaded
            import structured_sparse_gemm_prune24_amd as p24
            st["we"] = p24.compress_f8_experts(q.float() * s[:, None] for q, s in zip(st["wq"], st["ws"]))
            st["x8"] = p24.Quantized8(st["xq"], st["xs"])
        return st
    st["wq"], st["ws"] = _quantize_blocks(0.02 * _normal(g, m, k), 128)
    dt = TYPES[case["stream"]]
    both = _stream(g, n, 2 * k if case["up"] else k).to(dt)
    st["x"], st["upv"] = both[:, :k], both[:, k:] if case["up"] else None      # one product's two halves
    st["b"] = 0.1 * _normal(g, m) if case["bias"] else None
    st["r"] = _normal(g, n, m).to(TYPES[case["out"]]) if case["residual"] else None
    if own:
        import structured_sparse_gemm_prune24_amd as p24
        st["w8"] = p24.Weight8Block(st["wq"], st["ws"])
    return st


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * (0.5 + 0.5 * torch.erf(z * math.sqrt(0.5)))
    return z


def _own(st):
    import structured_sparse_gemm_prune24_amd as p24
    if st["op"] == "route":
        r = p24.route(st["l"], st["k"], score=st["score"], bias=st["b"], normalize=st["normalize"])
        return {"experts": r.experts, "weights": r.weights, "offsets": r.offsets, "tokens": r.tokens, "positions": r.positions}
    out = TYPES[st["out"]]
    if st["op"] == "combine":
        return {"y": p24.combine_experts(st["z"], st["p"], st["w"], residual=st["r"])}
    if st["op"] == "experts":
        return {"y": p24.spmm24_f8_grouped(st["we"], st["x8"], st["off"], tokens=st["tok"], out_dtype=out, out=st["y"],
                                           bias=st["b"], act=st["act"])}
    x = p24.quantize_f8_block(st["x"], st["upv"], act=st["quant_act"])
    return {"y": p24.gemm_f8_block(st["w8"], x, out_dtype=out, bias=st["b"], act=st["act"], residual=st["r"])}


def _run_route(st):
    l = st["l"].float()
    # sums of a sigmoid and a bias are compared in 64 bits: 32 would tie experts that are none
    score = 1 / (1 + torch.exp(-l.double())) + (0 if st["b"] is None else st["b"].double()) if st["score"] == "sigmoid" else l
    experts, top = _best(score, l, st["k"])
    if st["score"] == "sigmoid":
        w = (1 / (1 + torch.exp(-l))).gather(1, top)
        w = torch.where(experts < 0, 0, w)
        w = w / w.sum(1, keepdim=True) if st["normalize"] else w
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        w = torch.where(experts < 0, 0, e.gather(1, top))
        w = w / (w if st["normalize"] else e).sum(1, keepdim=True)
    w = torch.where(experts < 0, 0, w)
    offsets, tokens, positions = _sorted(experts, st["experts"])
    return {"experts": experts.int(), "weights": w, "offsets": offsets, "tokens": tokens, "positions": positions}


def _run_experts(st):
    off, live = st["off"].long(), st["active"]
    lo, count = off[live], (off[1:] - off[:-1])[live]
    place = torch.arange(st["cap"], device=off.device)
    rows = torch.where(place < count[:, None], lo[:, None] + place, lo[:, None])   # of each expert, padded to the largest
    src = rows if st["tok"] is None else st["tok"].long()[rows]
    z = torch.bmm(st["xq"].float()[src], st["wq"][live].float().transpose(1, 2))
    z = z * st["xs"][src][:, :, None] * st["ws"][live][:, None, :]
    if st["b"] is not None:
        z = z + st["b"][live][:, None, :]
    z = _act(z, st["act"]).to(TYPES[st["out"]])
    every = torch.arange(st["tokens"] * st["k"], device=off.device)
    group = (every[:, None] >= off[live + 1]).sum(1)
    mine = group.clamp_max(live.numel() - 1)
    y = z[mine, (every - lo[mine]).clamp_max(st["cap"] - 1)]
    return {"y": torch.where((group < live.numel())[:, None], y, 0)}


def run(st):
    if own:
        return _own(st)
    if st["op"] == "route":
        return _run_route(st)
    if st["op"] == "experts":
        return _run_experts(st)
    if st["op"] == "combine":
        y = (st["z"].float()[st["p"].clamp_min(0).long()] * torch.where(st["p"] < 0, 0, st["w"])[:, :, None]).sum(1)
        return {"y": (y if st["r"] is None else y + st["r"].float()).to(TYPES[st["out"]])}
    a = _act(st["x"].float(), st["quant_act"])
    a = a if st["upv"] is None else a * st["upv"].float()
    q, s = _quantize_blocks(a, 1)
    n, k = a.shape
    a = q.float() * s.repeat_interleave(128, 1)[:, :k]
    w = st["wq"].float() * st["ws"].repeat_interleave(128, 0)[: st["rows"]].repeat_interleave(128, 1)[:, :k]
    z = a @ w.t()
    if st["b"] is not None:
        z = z + st["b"]
    z = _act(z, st["act"])
    if st["r"] is not None:
        z = z + st["r"].float()
    return {"y": z.to(TYPES[st["out"]])}


def exact(case, seed):
    """From the definitions in fp64; the quantised operands are the 8-bit values that they stand for."""
    st = prepare(case, seed)
    d = torch.float64

    def act(z, name):
        if name == "silu":
            return z * torch.sigmoid(z)
        if name == "gelu":
            return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
        return torch.where(z > 0, z, torch.zeros_like(z)) if name == "relu" else z

    if case["op"] == "route":
        l = st["l"].to(d)
        p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, dim=1), nan=0.0)
        score = p if st["b"] is None else p + st["b"].to(d)
        order = torch.argsort(-torch.where(torch.isinf(l), -math.inf, l if case["score"] == "softmax" else score), dim=1, stable=True)
        w = torch.gather(p, 1, order[:, : case["k"]])
        w = w.masked_fill(torch.isinf(torch.gather(l, 1, order[:, : case["k"]])), 0.0)
        if case["normalize"]:
            w = w / torch.clamp(w.sum(1, keepdim=True), min=1e-300)
        return {"experts": None, "weights": w, "offsets": None, "tokens": None, "positions": None}
    if case["op"] == "combine":
        y = torch.zeros(case["tokens"], case["width"], dtype=d, device="cuda") if st["r"] is None else st["r"].to(d)
        for j in range(case["k"]):
            p = st["p"][:, j].long()
            on = (p >= 0).to(d) * st["w"][:, j].to(d)
            y = y + on.unsqueeze(1) * st["z"][p.clamp(min=0)].to(d)
        return {"y": y}
    if case["op"] == "experts":
        y = torch.zeros(case["tokens"] * case["k"], case["rows"], dtype=d, device="cuda")
        ends = st["off"].tolist()
        for i in range(case["experts"]):
            r = torch.arange(ends[i], ends[i + 1], device="cuda")
            if r.numel() == 0:
                continue
            src = st["tok"][r].long() if case["gather"] else r
            x = st["xq"][src].to(d) * st["xs"][src].to(d).unsqueeze(1)
            z = torch.mm(x, (st["wq"][i].to(d) * st["ws"][i].to(d).unsqueeze(1)).T)
            y[r] = act(z + st["b"][i].to(d) if case["bias"] else z, case["act"])
        return {"y": y}
    a = act(st["x"].to(d), case["quant_act"])
    if case["up"]:
        a = a * st["upv"].to(d)
    n, k = a.shape
    m = case["rows"]
    out = torch.zeros(n, m, dtype=d, device="cuda")
    for b in range(0, k, 128):
        part = a[:, b:b + 128]
        s = torch.clamp(torch.linalg.vector_norm(part, ord=math.inf, dim=1) / 448, min=TINY).float().to(d).unsqueeze(1)
        w = st["wq"][:, b:b + 128].to(d) * st["ws"][torch.arange(m, device="cuda") // 128, b // 128].to(d).unsqueeze(1)
        out += torch.mm((part / s).float().to(F8).to(d) * s, w.T)
    out = act(out + st["b"].to(d) if case["bias"] else out, case["act"])
    return {"y": out + st["r"].to(d) if case["residual"] else out}


def work(case):
    n = case["tokens"]
    if case["op"] == "route":
        e, k, size = case["experts"], case["k"], BYTES[case["logits"]]
        return {"bytes": n * e * size + n * k * 16 + 4 * (e + 1) + 4 * e * case["bias"], "flops": 4 * n * e}
    if case["op"] == "combine":
        rows = (n - case["padded"]) * case["k"]
        size = BYTES[case["out"]]
        return {"bytes": rows * case["width"] * size + n * case["width"] * size * (1 + case["residual"]) + 8 * n * case["k"],
                "flops": 2 * rows * case["width"]}
    m, k = case["rows"], case["width"]
    if case["op"] == "experts":
        e, rows = case["experts"], (n - case["padded"]) * case["k"]
        live = min(e, math.ceil(e * (1 - (1 - 1 / e) ** rows)))   # experts that rows reach, about
        x = (n - case["padded"] if case["gather"] else rows) * (k + 4) + 4 * rows * case["gather"]
        return {"bytes": live * (m * k * 5 // 8 + 4 * m * (1 + case["bias"])) + x + rows * m * BYTES[case["out"]],
                "flops": rows * m * k}
    size = BYTES[case["out"]]
    byts = m * k + n * k * BYTES[case["stream"]] * (1 + case["up"]) + n * m * size * (1 + case["residual"]) + 4 * m * case["bias"]
    return {"bytes": byts, "flops": 2 * n * m * k}
