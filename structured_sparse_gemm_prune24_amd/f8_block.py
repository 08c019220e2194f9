"""The dense 8-bit product with a scale for each block of 128 (``include/prune24_f8_block.h``): for the
layers of a pruned model that stay dense.

    w = p24.quantize_weight_f8_block(W)                   # W [M, K]: a scale per 128 x 128 weights
    xb = p24.quantize_f8_block(x)                         # a scale per token and 128 features
    y = p24.gemm_f8_block(w, xb, residual=h)              # [tokens, M]
    ab = p24.quantize_f8_block(gate, up, act="silu")      # 8-bit values of silu(gate) * up
    y, h = p24.feed_forward_f8_block(x, r, g, w_gate_up, w_down)

Activations are tokens x features; values are e4m3.  A model's own 8-bit weights with 128 x 128 scales
are a Weight8Block as they are.  No gradients (inference only).
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _check, _w_code, lib
from .f8 import _ACTS_F8, _CODES, _STREAM_TYPES, F8, _act_code, _call, _rows, _vector, rms_norm


@dataclass
class Rows8Block:
    """Rows in 8 bits: values[t, k] * scale[k // 128, t]."""
    values: object       # torch.float8_e4m3fn [tokens, width]
    scale: object        # torch.float32 [ceil(width / 128), tokens]


@dataclass
class Weight8Block:
    """A dense M x K matrix in 8 bits: values[m, k] * scale[m // 128, k // 128]."""
    values: object       # torch.float8_e4m3fn [M, K]
    scale: object        # torch.float32 [ceil(M / 128), ceil(K / 128)]


_CALL = None


def _fast():
    global _CALL
    _CALL = _call()
    return _CALL


def _blocks(n):
    return (n + 127) // 128


def _scale_rows(t, name, shape, dev):
    """Leading dimension of the blocks' scales, tokens side by side."""
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be a device tensor on {dev}")
    if t.dtype is not torch.float32 or tuple(t.shape) != shape or (t.stride(1) != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be an fp32 tensor of shape {shape} with unit stride along its last dimension")
    return t.stride(0) if shape[0] > 1 else max(t.stride(0), shape[1])


def _aligned_rows(shape, dev):
    """New e4m3 rows that start on 16 bytes."""
    return torch.empty((shape[0], (shape[1] + 15) // 16 * 16), dtype=F8, device=dev)[:, :shape[1]]


def quantize_f8_block(x, up=None, act="none") -> Rows8Block:
    """act(x) * up (act(x) without `up`) in 8 bits, a scale per token and 128 features.

    x, up [tokens, width] fp32 or bf16, for instance the two halves of one product's output rows; act
    "none", "relu", "gelu" or "silu".  No gradients (inference only)."""
    if act in _ACTS_F8:
        got = (_CALL or _fast()).quantize(x, up, _ACTS_F8[act])
        if got is not None:
            return Rows8Block(*got)
    dev = x.device
    ldx = _rows(x, "x", dev, _STREAM_TYPES)
    shape = tuple(x.shape)
    if shape[1] < 1:
        raise ValueError("x has no features")
    a = _act_code(act)
    upp, ldu = None, 0
    if up is not None:
        ldu = _rows(up, "up", dev, (x.dtype,), shape)
        upp = up.data_ptr()
    values = _aligned_rows(shape, dev)
    scale = torch.empty((_blocks(shape[1]), shape[0]), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().quantize_f8_block(x.data_ptr(), _CODES[x.dtype], ldx, upp, ldu, a, shape[0], shape[1],
                                       values.data_ptr(), values.stride(0), scale.data_ptr(), shape[0],
                                       torch.cuda.current_stream(dev).cuda_stream), "quantize_f8_block")
    return Rows8Block(values, scale)


def quantize_weight_f8_block(W) -> Weight8Block:
    """W (cuda fp32 or bf16, [M, K]) in 8 bits, a scale per 128 x 128 block."""
    dev = W.device
    ldw = _rows(W, "W", dev, _STREAM_TYPES)
    M, K = W.shape
    values = _aligned_rows((M, K), dev)
    scale = torch.empty((_blocks(M), _blocks(K)), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().quantize_weight_f8_block(W.data_ptr(), _w_code(W), M, K, ldw, values.data_ptr(), values.stride(0),
                                              scale.data_ptr(), torch.cuda.current_stream(dev).cuda_stream),
               "quantize_weight_f8_block")
    return Weight8Block(values, scale)


def gemm_f8_block(w: Weight8Block, X: Rows8Block, out_dtype=torch.bfloat16, out=None, bias=None, act="none", residual=None):
    """Y = act(W X^T + bias) + residual as [tokens, M] for a dense 8-bit weight and 8-bit rows.

    W and X of the same K, a multiple of 16, their rows 16-byte aligned; bias fp32 [M]; act "none", "relu",
    "gelu" or "silu"; residual [tokens, M] of the output's dtype, bf16 or fp32, and may be `out` itself.  No
    gradients (inference only)."""
    v = X.values
    if out is None and out_dtype in _STREAM_TYPES and act in _ACTS_F8:
        Y = (_CALL or _fast()).block_product(w.values, w.scale, v, X.scale, _CODES[out_dtype], bias, _ACTS_F8[act], residual)
        if Y is not None:
            return Y
    dev = v.device
    ldx = _rows(v, "X.values", dev, (F8,))
    N, K = v.shape
    ldw = _rows(w.values, "the weight", dev, (F8,))
    M, wk = w.values.shape
    if K != wk:
        raise ValueError(f"X has {K} features, W has K = {wk}")
    ldxs = _scale_rows(X.scale, "X.scale", (_blocks(K), N), dev)
    if tuple(w.scale.shape) != (_blocks(M), _blocks(K)) or not w.scale.is_contiguous() or \
            w.scale.dtype is not torch.float32 or w.scale.device != dev:
        raise ValueError(f"the weight's scale must be a contiguous fp32 tensor of shape {(_blocks(M), _blocks(K))} on {dev}")
    bp = None if bias is None else _vector(bias, "bias", M, dev)
    a = _act_code(act)
    shape = (N, M)
    if out is None:
        if out_dtype not in _STREAM_TYPES:
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        out = torch.empty(shape, dtype=out_dtype, device=dev)
        ldy = M
    else:
        ldy = _rows(out, "out", dev, _STREAM_TYPES, shape)
    rp, ldr = None, 0
    if residual is not None:
        ldr = _rows(residual, "residual", dev, (out.dtype,), shape)
        rp = residual.data_ptr()
    with torch.cuda.device(dev):
        _check(lib().gemm_f8_block(w.values.data_ptr(), ldw, w.scale.data_ptr(), M, K, v.data_ptr(), ldx,
                                   X.scale.data_ptr(), ldxs, N, out.data_ptr(), _CODES[out.dtype], ldy, bp, a, rp, ldr,
                                   torch.cuda.current_stream(dev).cuda_stream), "gemm_f8_block")
    return out


def feed_forward_f8_block(x, residual, weight, w_gate_up: Weight8Block, w_down: Weight8Block, act="silu", eps=1e-6):
    """One feed-forward layer on dense 8-bit weights, as feed_forward_f8 on pruned ones: (y, h) with
    h = x + residual and y = W_down (act(gate) * up) + h, gate and up the halves of W_gate_up norm(h).

    x, residual [tokens, width]; w_gate_up 2F x width, gate rows first; w_down width x F."""
    (m1, k1), (m2, k2) = w_gate_up.values.shape, w_down.values.shape
    if m1 % 2 or m1 // 2 != k2 or m2 != x.shape[-1]:
        raise ValueError(f"W_gate_up is {(m1, k1)}, W_down {(m2, k2)}: not 2F x {x.shape[-1]} and {x.shape[-1]} x F")
    n, h = rms_norm(x, weight, residual=residual, eps=eps, out_dtype=x.dtype)
    h = x if h is None else h
    gu = gemm_f8_block(w_gate_up, quantize_f8_block(n), out_dtype=x.dtype)
    a = quantize_f8_block(gu[:, :k2], gu[:, k2:], act=act)
    return gemm_f8_block(w_down, a, out_dtype=x.dtype, residual=h), h
