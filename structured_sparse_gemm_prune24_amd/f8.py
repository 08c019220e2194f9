"""8-bit feed-forward operators of libprune24.so (``include/prune24_f8.h``): RMS norm with the
residual's addition, gated activation, and the product with 2:4-sparse 8-bit weights.

    w = p24.compress_f8(W)                              # W [M, K], once per weight
    xq, h = p24.rms_norm(x, g, residual=r)              # 8-bit rows of the norm, and x + r
    gu = p24.spmm24_f8(w_gate_up, xq)                   # [tokens, M] bf16
    aq = p24.gated_act(gu[:, :F], gu[:, F:])            # 8-bit rows of silu(gate) * up
    y = p24.spmm24_f8(w_down, aq, residual=h)           # adds to the residual stream
    y, h = p24.feed_forward_f8(x, r, g, w_gate_up, w_down)   # the four together

Activations are tokens x features.  8-bit values are e4m3 with one fp32 scale per row.  As in the
rest of the binding this is argument marshalling only, and the operators have no backward pass:
they take tensors that require gradients, as they are, and return results without history.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from . import P24_BF16, P24_ERR_SHAPE, P24_ERR_UNSUPPORTED, P24_F32, P24Error, _ACTS, _check, _w_code, lib

P24_F8 = 2
P24_ACT_SILU = 3
_ACTS_F8 = {**_ACTS, "silu": P24_ACT_SILU}
F8 = torch.float8_e4m3fn
_CODES = {torch.float32: P24_F32, torch.bfloat16: P24_BF16, F8: P24_F8}


@dataclass
class Quantized8:
    """Rows held in 8 bits: row t is about values[t] * scale[t]."""
    values: object       # torch.float8_e4m3fn [tokens, width]
    scale: object        # torch.float32 [tokens]


@dataclass
class Compressed24F8:
    """A 2:4-compressed M x K matrix of e4m3 values with one scale per row."""
    data: object         # torch.uint8, flat: values and positions in operand order
    scale: object        # torch.float32 [M]
    M: int
    K: int


_CALL = None


def _call():
    """_f8_call.so: each call's checks, outputs and launch in one step where its arguments are of the
    plain form, else None (csrc/f8_call.cpp); the code below then makes the call or names what is wrong."""
    global _CALL
    if _CALL is None:
        L = lib()
        try:
            from . import _f8_call as c
        except ImportError as e:
            raise RuntimeError("_f8_call.so is missing: build it with __graft_entry__.build() "
                               "or python structured_sparse_gemm_prune24_amd/build.py") from e
        c.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                 for f in (L.rms_norm, L.gated_act, L.spmm24_f8, L.experts_route, L.spmm24_f8_grouped, L.experts_combine,
                           L.quantize_f8_block, L.gemm_f8_block, L.experts_route_workspace)))
        _CALL = c
    return _CALL


def _rows(t, name, dev, dtypes, shape=None):
    """Leading dimension of a 2-D device tensor with unit stride along its rows (a single row or
    column has no stride of its own)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA/HIP device tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the operation runs on {dev}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, not one of {[str(d) for d in dtypes]}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    n, w = t.shape
    if shape is not None and (n, w) != shape:
        raise ValueError(f"{name} is {(n, w)}, not {shape}")
    s0, s1 = t.stride()
    if s1 != 1 and w > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return s0 if n > 1 else max(s0, w)


def _vector(t, name, n, dev):
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be a device tensor on {dev}")
    if t.dtype is not torch.float32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 vector of {n} values")
    return t.data_ptr()


def _act_code(act):
    code = _ACTS_F8.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS_F8)}")
    return code


_STREAM_TYPES = (torch.bfloat16, torch.float32)


def _row_output(out, out_dtype, shape, dev):
    """(what is returned, tensor of y, its leading dimension, dtype code, pointer of the scales)."""
    if out is None:
        code = _CODES.get(out_dtype)
        if code is None:
            raise ValueError("out_dtype must be torch.float8_e4m3fn, torch.bfloat16 or torch.float32")
        y = torch.empty(shape, dtype=out_dtype, device=dev)
        if code != P24_F8:
            return y, y, shape[1], code, None
        scale = torch.empty(shape[0], dtype=torch.float32, device=dev)
        return Quantized8(y, scale), y, shape[1], code, scale.data_ptr()
    if isinstance(out, Quantized8):
        ld = _rows(out.values, "out.values", dev, (F8,), shape)
        return out, out.values, ld, P24_F8, _vector(out.scale, "out.scale", shape[0], dev)
    return out, out, _rows(out, "out", dev, _STREAM_TYPES, shape), _CODES[out.dtype], None


def rms_norm(x, weight, residual=None, eps=1e-6, out_dtype=F8, out=None, h=None):
    """(y, h) with h = x + residual and y = h / sqrt(mean(h^2) + eps) * weight over each row.

    x, residual [tokens, width] fp32 or bf16; weight fp32 [width].  y is a Quantized8 for
    out_dtype torch.float8_e4m3fn (the default), else a bf16 or fp32 tensor; h has x's dtype, and
    is None without a residual.  `out` (a Quantized8 or tensor) and `h` give the outputs' place;
    h may be x or residual itself.  No gradients (inference only)."""
    if out is None and h is None and out_dtype in _CODES:
        got = (_CALL or _call()).norm(x, weight, residual, eps, _CODES[out_dtype])
        if got is not None:
            y, s, h = got
            return (y if s is None else Quantized8(y, s)), h
    dev = x.device
    ldx = _rows(x, "x", dev, _STREAM_TYPES)
    shape = tuple(x.shape)
    wp = _vector(weight, "weight", shape[1], dev)
    if not (eps >= 0 and math.isfinite(eps)):
        raise ValueError("eps must be finite and not negative")
    rp = hp = None
    ldr = ldh = 0
    if residual is not None:
        ldr = _rows(residual, "residual", dev, (x.dtype,), shape)
        rp = residual.data_ptr()
        if h is None:
            h = torch.empty(shape, dtype=x.dtype, device=dev)
            ldh = shape[1]
        else:
            ldh = _rows(h, "h", dev, (x.dtype,), shape)
        hp = h.data_ptr()
    elif h is not None:
        raise ValueError("h is the sum with a residual: there is none")
    got, y, ldy, code, sp = _row_output(out, out_dtype, shape, dev)
    _check(lib().rms_norm(x.data_ptr(), _CODES[x.dtype], ldx, rp, ldr, wp, eps, shape[0], shape[1], hp, ldh,
                          y.data_ptr(), code, ldy, sp, torch.cuda.current_stream(dev).cuda_stream), "rms_norm")
    return got, h


def gated_act(gate, up=None, act="silu", out_dtype=F8, out=None):
    """act(gate) * up (act(gate) without `up`), act "silu", "gelu", "relu" or "none".

    gate, up [tokens, width] fp32 or bf16, for instance the two halves of one product's output
    rows.  Returns a Quantized8 for out_dtype torch.float8_e4m3fn (the default), else a bf16 or
    fp32 tensor; `out` gives its place.  With act "none" and no `up` it quantizes the rows.  No
    gradients (inference only)."""
    if out is None and out_dtype in _CODES and act in _ACTS_F8:
        got = (_CALL or _call()).gate(gate, up, _ACTS_F8[act], _CODES[out_dtype])
        if got is not None:
            y, s, _ = got
            return y if s is None else Quantized8(y, s)
    dev = gate.device
    ldg = _rows(gate, "gate", dev, _STREAM_TYPES)
    shape = tuple(gate.shape)
    a = _act_code(act)
    upp, ldu = None, 0
    if up is not None:
        ldu = _rows(up, "up", dev, (gate.dtype,), shape)
        upp = up.data_ptr()
    got, y, ldy, code, sp = _row_output(out, out_dtype, shape, dev)
    _check(lib().gated_act(gate.data_ptr(), _CODES[gate.dtype], ldg, upp, ldu, a, shape[0], shape[1], y.data_ptr(),
                           code, ldy, sp, torch.cuda.current_stream(dev).cuda_stream), "gated_act")
    return got


def compress_f8(W) -> Compressed24F8:
    """Magnitude 2:4 prune of W (cuda fp32 or bf16, [M, K], K % 64 == 0) into 8-bit rows."""
    dev = W.device
    ldw = _rows(W, "W", dev, _STREAM_TYPES)
    M, K = W.shape
    n = lib().prune24_f8_bytes(M, K)
    if n == 0 and M * K:
        raise P24Error(P24_ERR_UNSUPPORTED if K % 64 else P24_ERR_SHAPE, "prune24_compress_f8")
    data = torch.empty(n, dtype=torch.uint8, device=dev)
    scale = torch.empty(M, dtype=torch.float32, device=dev)
    _check(lib().prune24_compress_f8(W.data_ptr(), _w_code(W), M, K, ldw, data.data_ptr(), scale.data_ptr(),
                                     torch.cuda.current_stream(dev).cuda_stream), "prune24_compress_f8")
    return Compressed24F8(data, scale, M, K)


def _weight(c: Compressed24F8, dev):
    """Pointer of a compressed weight's scales, after checking its buffers."""
    d = c.data
    if not d.is_cuda or d.device != dev:
        raise ValueError(f"the weight is on {d.device}, the operation runs on {dev}")
    if d.dtype is not torch.uint8 or not d.is_contiguous() or d.numel() < lib().prune24_f8_bytes(c.M, c.K):
        raise ValueError(f"the weight's data is not the compressed form of {(c.M, c.K)}")
    return _vector(c.scale, "the weight's scale", c.M, dev)


def decompress_f8(c: Compressed24F8):
    """Dense fp32 [M, K]: value times scale at the kept positions, zeros elsewhere."""
    dev = c.data.device
    _weight(c, dev)
    out = torch.empty((c.M, c.K), dtype=torch.float32, device=dev)
    _check(lib().prune24_decompress_f8(c.data.data_ptr(), c.scale.data_ptr(), c.M, c.K, out.data_ptr(), c.K,
                                       torch.cuda.current_stream(dev).cuda_stream), "prune24_decompress_f8")
    return out


def spmm24_f8(c: Compressed24F8, X: Quantized8, out_dtype=torch.bfloat16, out=None, bias=None, act="none",
              residual=None):
    """Y = act(W X^T + bias) + residual as [tokens, M] for an 8-bit 2:4 weight and 8-bit rows X.

    X.values [tokens, K] e4m3 (rows 16-byte aligned), X.scale fp32 [tokens]; bias fp32 [M];
    act "none", "relu", "gelu" or "silu"; residual [tokens, M] of the output's dtype, bf16 or
    fp32, and may be `out` itself.  No gradients (inference only)."""
    v = X.values
    if out is None and out_dtype in _STREAM_TYPES and act in _ACTS_F8:
        Y = (_CALL or _call()).product(c.data, c.scale, c.M, c.K, v, X.scale, _CODES[out_dtype], bias, _ACTS_F8[act],
                                       residual)
        if Y is not None:
            return Y
    dev = v.device
    ldx = _rows(v, "X.values", dev, (F8,))
    N, K = v.shape
    if K != c.K:
        raise ValueError(f"X has {K} features, W has K = {c.K}")
    ws = _weight(c, dev)
    xs = _vector(X.scale, "X.scale", N, dev)
    bp = None if bias is None else _vector(bias, "bias", c.M, dev)
    a = _act_code(act)
    shape = (N, c.M)
    if out is None:
        if out_dtype not in _STREAM_TYPES:
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        out = torch.empty(shape, dtype=out_dtype, device=dev)
        ldy = c.M
    else:
        ldy = _rows(out, "out", dev, _STREAM_TYPES, shape)
    rp, ldr = None, 0
    if residual is not None:
        ldr = _rows(residual, "residual", dev, (out.dtype,), shape)
        rp = residual.data_ptr()
    _check(lib().spmm24_f8(c.data.data_ptr(), ws, c.M, K, v.data_ptr(), ldx, xs, N, out.data_ptr(),
                           _CODES[out.dtype], ldy, bp, a, rp, ldr, torch.cuda.current_stream(dev).cuda_stream), "spmm24_f8")
    return out


def feed_forward_f8(x, residual, weight, w_gate_up: Compressed24F8, w_down: Compressed24F8, act="silu", eps=1e-6):
    """One feed-forward layer on 8-bit 2:4 weights: (y, h) with h = x + residual and
    y = W_down (act(gate) * up) + h, where gate and up are the halves of W_gate_up norm(h).

    x, residual [tokens, width]; w_gate_up 2F x width, gate rows first; w_down width x F.  No
    gradients (inference only)."""
    if w_gate_up.M % 2 or w_gate_up.M // 2 != w_down.K or w_down.M != x.shape[-1]:
        raise ValueError(f"W_gate_up is {(w_gate_up.M, w_gate_up.K)}, W_down {(w_down.M, w_down.K)}: "
                         f"not 2F x {x.shape[-1]} and {x.shape[-1]} x F")
    xq, h = rms_norm(x, weight, residual=residual, eps=eps)
    h = x if h is None else h
    gu = spmm24_f8(w_gate_up, xq, out_dtype=x.dtype)
    f = w_down.K
    aq = gated_act(gu[:, :f], gu[:, f:], act=act)
    return spmm24_f8(w_down, aq, out_dtype=x.dtype, residual=h), h
