"""Expert operators of libprune24.so (``include/prune24_experts.h``): routing, 2:4-sparse 8-bit
products grouped by expert with ragged numbers of rows, and the combination of a token's experts.

    w = p24.compress_f8_experts(W)                        # W [E, M, K], once per layer
    r = p24.route(logits, 8)                              # experts, weights, rows sorted by expert
    gu = p24.spmm24_f8_grouped(w_gate_up, xq, r.offsets, tokens=r.tokens)    # [tokens * 8, 2F]
    aq = p24.gated_act(gu[:, :F], gu[:, F:])
    z = p24.spmm24_f8_grouped(w_down, aq, r.offsets)
    y = p24.combine_experts(z, r.positions, r.weights, residual=h)
    y = p24.feed_forward_f8_experts(xq, logits, 8, w_gate_up, w_down, residual=h)   # all of it

Activations are tokens x features; 8-bit rows are those of f8.py.  How many rows an expert has stays on
the device: a layer can be captured in a graph.  No gradients (inference only).
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import P24_ERR_SHAPE, P24_ERR_UNSUPPORTED, P24Error, _check, lib
from .f8 import _ACTS_F8, _CODES, _STREAM_TYPES, F8, Quantized8, _act_code, _call, _rows, _vector, compress_f8, gated_act

P24_SCORE_SOFTMAX, P24_SCORE_SIGMOID = 0, 1
_SCORES = {"softmax": P24_SCORE_SOFTMAX, "sigmoid": P24_SCORE_SIGMOID}


@dataclass
class Routing:
    """Which experts the tokens go to, and the rows that this makes.  The tensors are parts of one allocation, which
    any of them keeps (from 65 tokens on with 4 bytes of scratch an expert for every 32 tokens)."""
    experts: object      # torch.int32 [tokens, k]: best first, -1 where no expert is open
    weights: object      # torch.float32 [tokens, k]
    offsets: object      # torch.int32 [E + 1]: expert e's rows are offsets[e] to offsets[e + 1]
    tokens: object       # torch.int32 [tokens * k]: the token of each row, -1 past the last row
    positions: object    # torch.int32 [tokens, k]: the row of each slot, -1 where there is none


@dataclass
class Experts24F8:
    """E compressed M x K matrices (Compressed24F8), one after the other."""
    data: object         # torch.uint8, flat
    scale: object        # torch.float32 [E, M]
    E: int
    M: int
    K: int


_CALL = None


def _fast():
    global _CALL
    _CALL = _call()
    return _CALL


def _ints(t, name, shape, dev):
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be a device tensor on {dev}")
    if t.dtype is not torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape}")
    return t.data_ptr()


def _floats(t, name, shape, dev):
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be a device tensor on {dev}")
    if t.dtype is not torch.float32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {shape}")
    return t.data_ptr()


def route(logits, k: int, score="softmax", bias=None, normalize=True, scale=1.0) -> Routing:
    """The k best experts of each token and its weights for them, and the rows sorted by expert.

    logits [tokens, E] fp32 or bf16; -inf closes an expert to a token (a row of -inf: a padded token).
    score "softmax" ranks by the logit and weighs by the softmax over the chosen experts (`normalize`)
    or over all; "sigmoid" ranks by sigmoid(logit) + bias (bias fp32 [E] or None) and weighs by the
    sigmoids, over their sum with `normalize` (NaN where the largest logit lies below -709.78: -inf closes
    experts, a type's lowest value does not).  Ties go to the lower expert.  Weights times `scale`."""
    code = _SCORES.get(score)
    if code is not None and (bias is None or code == P24_SCORE_SIGMOID) and math.isfinite(scale):
        got = (_CALL or _fast()).route(logits, k, code, bias, 1 if normalize else 0, scale)
        if got is not None:
            return Routing(*got)
    dev = logits.device
    ldl = _rows(logits, "logits", dev, _STREAM_TYPES)
    T, E = logits.shape
    if code is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    if not 1 <= k <= E:
        raise ValueError(f"k is {k}, not in 1 to {E} experts")
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    if bias is not None and score != "sigmoid":
        raise ValueError("a bias goes with score \"sigmoid\"")
    bp = None if bias is None else _vector(bias, "bias", E, dev)
    new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)  # noqa: E731
    ws = torch.empty(lib().experts_route_workspace(T, E), dtype=torch.uint8, device=dev)
    r = Routing(new(T, k), torch.empty((T, k), dtype=torch.float32, device=dev), new(E + 1), new(T * k), new(T, k))
    with torch.cuda.device(dev):
        _check(lib().experts_route(logits.data_ptr(), _CODES[logits.dtype], ldl, T, E, k, code, bp, int(bool(normalize)),
                                   scale, r.experts.data_ptr(), r.weights.data_ptr(), r.offsets.data_ptr(),
                                   r.tokens.data_ptr(), r.positions.data_ptr(), ws.data_ptr(), ws.numel(),
                                   torch.cuda.current_stream(dev).cuda_stream), "experts_route")
    return r


def compress_f8_experts(W) -> Experts24F8:
    """compress_f8 of each expert's matrix: W [E, M, K], or any iterable of [M, K] tensors."""
    parts = [compress_f8(w) for w in W]
    if not parts:
        raise ValueError("no experts")
    M, K = parts[0].M, parts[0].K
    if any((p.M, p.K) != (M, K) for p in parts):
        raise ValueError("the experts' matrices differ in shape")
    if len({p.data.device for p in parts}) > 1:
        raise ValueError("the experts' matrices lie on several devices")
    return Experts24F8(torch.cat([p.data for p in parts]), torch.stack([p.scale for p in parts]), len(parts), M, K)


def _experts_weight(c: Experts24F8, dev):
    d = c.data
    if not d.is_cuda or d.device != dev:
        raise ValueError(f"the weights are on {d.device}, the operation runs on {dev}")
    if d.dtype is not torch.uint8 or not d.is_contiguous() or d.numel() < c.E * lib().prune24_f8_bytes(c.M, c.K):
        raise ValueError(f"the weights' data is not the compressed form of {c.E} of {(c.M, c.K)}")
    return _floats(c.scale, "the weights' scale", (c.E, c.M), dev)


def spmm24_f8_grouped(c: Experts24F8, X: Quantized8, offsets, tokens=None, out_dtype=torch.bfloat16, out=None, bias=None,
                      act="none"):
    """Y[p] = act(W[e] X[tokens[p]] + bias[e]) for the rows p of each expert e, offsets[e] to offsets[e + 1].

    X.values [rows of X, K] e4m3 (rows 16-byte aligned), X.scale fp32; offsets int32 [E + 1], not
    falling; tokens int32 [rows]: which row of X a row takes, or None: row p itself; bias fp32 [E, M].  Y has one row for
    each entry of `tokens` (of X without), at most 65535 * 32.  Rows behind the last expert's are not written: they keep what
    `out` held."""
    v = X.values
    if out is None and out_dtype in _STREAM_TYPES and act in _ACTS_F8:
        Y = (_CALL or _fast()).grouped(c.data, c.scale, c.E, c.M, c.K, v, X.scale, offsets, tokens, _CODES[out_dtype], bias,
                                       _ACTS_F8[act])
        if Y is not None:
            return Y
    dev = v.device
    ldx = _rows(v, "X.values", dev, (F8,))
    n, K = v.shape
    if K != c.K:
        raise ValueError(f"X has {K} features, the weights have K = {c.K}")
    ws = _experts_weight(c, dev)
    xs = _vector(X.scale, "X.scale", n, dev)
    op = _ints(offsets, "offsets", (c.E + 1,), dev)
    rows, tp = n, None
    if tokens is not None:
        rows = tokens.numel()
        tp = _ints(tokens, "tokens", (rows,), dev)
    bp = None if bias is None else _floats(bias, "bias", (c.E, c.M), dev)
    a = _act_code(act)
    if out is None:
        if out_dtype not in _STREAM_TYPES:
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        out = torch.empty((rows, c.M), dtype=out_dtype, device=dev)
        ldy = c.M
    else:
        ldy = _rows(out, "out", dev, _STREAM_TYPES, (rows, c.M))
    with torch.cuda.device(dev):
        _check(lib().spmm24_f8_grouped(c.data.data_ptr(), ws, c.E, c.M, K, v.data_ptr(), ldx, xs, n, op, tp, rows,
                                       out.data_ptr(), _CODES[out.dtype], ldy, bp, a,
                                       torch.cuda.current_stream(dev).cuda_stream), "spmm24_f8_grouped")
    return out


def combine_experts(Z, positions, weights, residual=None, out_dtype=None, out=None):
    """y[t] = residual[t] + sum_j weights[t][j] Z[positions[t][j]], positions outside Z's rows adding nothing.

    Z [rows, width] fp32 or bf16; positions int32, weights fp32 [tokens, k]; y has the residual's type,
    else Z's, unless out_dtype or `out` says otherwise; `out` may be the residual itself."""
    if out is None and (out_dtype is None or out_dtype in _STREAM_TYPES):
        y = (_CALL or _fast()).combine(Z, positions, weights, residual, -1 if out_dtype is None else _CODES[out_dtype])
        if y is not None:
            return y
    dev = Z.device
    ldz = _rows(Z, "Z", dev, _STREAM_TYPES)
    if positions.dim() != 2:
        raise ValueError("positions must be 2-D")
    T, k = positions.shape
    pp = _ints(positions, "positions", (T, k), dev)
    wp = _floats(weights, "weights", (T, k), dev)
    shape = (T, Z.shape[1])
    if out is None:
        out_dtype = out_dtype or (Z.dtype if residual is None else residual.dtype)
        if out_dtype not in _STREAM_TYPES:
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        out = torch.empty(shape, dtype=out_dtype, device=dev)
        ldy = shape[1]
    else:
        ldy = _rows(out, "out", dev, _STREAM_TYPES, shape)
    rp, ldr = None, 0
    if residual is not None:
        ldr = _rows(residual, "residual", dev, (out.dtype,), shape)
        rp = residual.data_ptr()
    with torch.cuda.device(dev):
        _check(lib().experts_combine(Z.data_ptr(), _CODES[Z.dtype], ldz, Z.shape[0], pp, wp, T, k, shape[1], rp, ldr,
                                     out.data_ptr(), _CODES[out.dtype], ldy, torch.cuda.current_stream(dev).cuda_stream),
               "experts_combine")
    return out


def feed_forward_f8_experts(xq: Quantized8, logits, k: int, w_gate_up: Experts24F8, w_down: Experts24F8, act="silu",
                            residual=None, out_dtype=torch.bfloat16, score="softmax", bias=None, normalize=True, scale=1.0):
    """One feed-forward layer of experts on 8-bit 2:4 weights: the tokens' k experts by `logits` (route), each
    W_down (act(gate) * up) with gate and up the halves of W_gate_up xq, weighed and added to the residual.

    xq: 8-bit rows of the norm [tokens, width]; logits [tokens, E]; w_gate_up E of 2F x width, gate rows
    first; w_down E of width x F.  The result has the residual's type, else out_dtype.  tokens * k is at most
    65535 * 32, the products' rows."""
    if w_gate_up.E != w_down.E or w_gate_up.M % 2 or w_gate_up.M // 2 != w_down.K or w_down.M != w_gate_up.K:
        raise ValueError(f"W_gate_up is {(w_gate_up.E, w_gate_up.M, w_gate_up.K)}, W_down "
                         f"{(w_down.E, w_down.M, w_down.K)}: not E of 2F x width and width x F")
    if logits.dim() != 2 or logits.shape != (xq.values.shape[0], w_gate_up.E):
        raise ValueError(f"logits is {tuple(logits.shape)}, not {(xq.values.shape[0], w_gate_up.E)}")
    out_dtype = out_dtype if residual is None else residual.dtype
    r = route(logits, k, score=score, bias=bias, normalize=normalize, scale=scale)
    gu = spmm24_f8_grouped(w_gate_up, xq, r.offsets, tokens=r.tokens, out_dtype=out_dtype)
    f = w_down.K
    aq = gated_act(gu[:, :f], gu[:, f:], act=act)
    z = spmm24_f8_grouped(w_down, aq, r.offsets, out_dtype=out_dtype)
    return combine_experts(z, r.positions, r.weights, residual=residual)
