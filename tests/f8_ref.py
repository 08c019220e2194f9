"""Plain references of the 8-bit feed-forward operators (test infrastructure): fp64 formulas, the
8-bit row format, the compressed layout written value by value, and a lane-level model of the
sparse 8-bit matrix instruction.

v_smfmac_f32_32x32x64_fp8_fp8 (A 32 x 64 with two of every four k kept, B 64 x 32, D 32 x 32 fp32):
  A lane L: row L % 32, logical k 32 (L // 32) .. +32, as 16 stored values; lane L's word gives, for
    stored value i, its position p = bits [2 i, 2 i + 2) inside group i // 2 of four k.
  B lane L: column L % 32; elements e < 16 are k = 16 (L // 32) + e, e >= 16 are
    k = 32 + 16 (L // 32) + (e - 16).
  D lane L, element i: row 8 (i // 4) + 4 (L // 32) + i % 4, column L % 32.
"""
import numpy as np
import torch

F8 = torch.float8_e4m3fn
TINY = np.float32(2.0 ** -126)
U = 2.0 ** -24                       # half a step of fp32
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, F8: 2.0 ** -4}


def f8_bits(v) -> np.ndarray:
    """fp32 array -> e4m3 bits, round to nearest even (on the CPU)."""
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(F8).view(torch.uint8).numpy()


def f8_values(bits) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(bits)).view(F8).to(torch.float64).numpy()


def compress(W):
    """(bits [M, K/2], positions [M, K/2], scale [M]) of fp32 W: the two largest magnitudes of every
    four, ties to the lower index, over the row's scale."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    M, K = W.shape
    key = (W.view(np.uint32) & 0x7FFFFFFF).reshape(M, K // 4, 4).astype(np.int64)
    order = np.argsort(-key, axis=2, kind="stable")[:, :, :2]
    pos = np.sort(order, axis=2)
    top = (W.view(np.uint32) & 0x7FFFFFFF).max(axis=1).view(np.float32)
    scale = (top / np.float32(448)).astype(np.float32)
    scale = np.where(scale < TINY, TINY, scale)
    kept = np.take_along_axis(W.reshape(M, K // 4, 4), pos, axis=2)
    with np.errstate(invalid="ignore"):
        bits = f8_bits(kept / scale[:, None, None])
    return bits.reshape(M, K // 2), pos.reshape(M, K // 2), scale


def pack(bits, pos, M, K) -> np.ndarray:
    """The compressed layout of include/prune24_f8.h as bytes."""
    groups, steps = (M + 127) // 128, 2 * ((K + 127) // 128)
    vb = np.zeros((groups * 128, steps * 32), dtype=np.uint8)
    pb = np.tile(np.array([0, 1], dtype=np.int64), (groups * 128, steps * 16))
    vb[:M, :K // 2] = bits
    pb[:M, :K // 2] = pos
    out = np.zeros((groups, steps, 5120), dtype=np.uint8)
    for g in range(groups):
        for s in range(steps):
            for b in range(4):
                r0 = 128 * g + 32 * b
                v = vb[r0:r0 + 32, 32 * s:32 * s + 32].reshape(32, 2, 16).transpose(1, 0, 2)   # lane L = 32 h + r
                out[g, s, 1024 * b:1024 * (b + 1)] = v.reshape(-1)
                p = pb[r0:r0 + 32, 32 * s:32 * s + 32].reshape(32, 2, 16).transpose(1, 0, 2).reshape(64, 16)
                words = np.zeros(64, dtype=np.uint32)
                for i in range(16):
                    words |= p[:, i].astype(np.uint32) << np.uint32(2 * i)
                out[g, s, 4096 + 256 * b:4096 + 256 * (b + 1)] = words.view(np.uint8)
    return out.reshape(-1)


def decompress(bits, pos, scale, K) -> np.ndarray:
    """Dense fp64 [M, K] of q * s."""
    M = bits.shape[0]
    out = np.zeros((M, K // 4, 4))
    np.put_along_axis(out, pos.reshape(M, K // 4, 2), (f8_values(bits) * scale[:, None].astype(np.float64)).reshape(M, K // 4, 2), axis=2)
    return out.reshape(M, K)


def smfmac64_model(a_lanes, b_lanes, words):
    """a_lanes [64, 16], b_lanes [64, 32] (fp64 values), words [64] uint32 -> [64, 16]."""
    A, B = np.zeros((32, 64)), np.zeros((64, 32))
    for L in range(64):
        h = L // 32
        for i in range(16):
            A[L % 32, 32 * h + 4 * (i // 2) + ((int(words[L]) >> (2 * i)) & 3)] += a_lanes[L, i]
        for e in range(32):
            B[16 * h + e if e < 16 else 16 + 16 * h + e, L % 32] = b_lanes[L, e]
    D = A @ B
    out = np.zeros((64, 16))
    for L in range(64):
        for i in range(16):
            out[L, i] = D[8 * (i // 4) + 4 * (L // 32) + i % 4, L % 32]
    return out


def act(z, name):
    """The activations in fp64 (torch, either device)."""
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / 2.0 ** 0.5)
    return torch.where(z < 0, torch.zeros_like(z), z) if name == "relu" else z


def act_error(z, name, out=torch.float32):
    """Bound of the kernel's relative error of act(z), as multiples of |act(z)|: each fp32 operation
    and each of the hardware's exp2 and reciprocal (one ulp, 2 U) counts, and a rounding in the
    exponent of exp grows with the exponent (|z| for SiLU, z^2 / 2 for GELU, three roundings each).
    GELU's fit is 3.3e-8 off for an fp32 output (within the 40 U), 1.8e-5 for the others."""
    if name == "silu":
        return (3 * z.abs() + 8) * U
    if name == "gelu":
        return (1.5 * z * z + 40) * U + (0 if out == torch.float32 else 1.8e-5)
    return torch.zeros_like(z)


def row_scale(y):
    """fp64 scale of the rows of y."""
    return (y.abs().amax(dim=1) / 448).clamp_min(float(TINY))
