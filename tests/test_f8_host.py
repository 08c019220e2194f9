"""Host-side checks of the 8-bit feed-forward operators (no GPU): exports, argument refusals of the
C entry points and of the binding (fake pointers, never dereferenced), and the compressed layout
driven through the lane-level model of the sparse 8-bit matrix instruction."""

import numpy as np
import pytest

from f8_ref import F8, compress, decompress, f8_values, pack, smfmac64_model

torch = pytest.importorskip("torch")
p24 = pytest.importorskip("structured_sparse_gemm_prune24_amd")
OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP = (p24.P24_OK, p24.P24_ERR_NULL, p24.P24_ERR_SHAPE, p24.P24_ERR_ALIGN,
                                        p24.P24_ERR_DTYPE, p24.P24_ERR_UNSUPPORTED)
P = 1 << 20
F32, BF16, E4 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    return p24.lib()


def test_exports(L):
    syms = p24.header_symbols(p24.F8_HEADER_PATH)
    assert len(syms) == len(set(syms)) and set(syms) == set(p24._F8_SIGNATURES)
    for s in syms:
        assert hasattr(L, s), s


def test_bytes(L):
    assert L.prune24_f8_bytes(1, 64) == 2 * 5120             # 128 rows, 128 columns
    assert L.prune24_f8_bytes(128, 128) == 2 * 5120
    assert L.prune24_f8_bytes(129, 192) == 2 * 4 * 5120
    assert L.prune24_f8_bytes(8192, 8192) == 64 * 128 * 5120
    assert L.prune24_f8_bytes(4, 96) == 0 and L.prune24_f8_bytes(-1, 64) == 0


def _norm(L, **k):
    v = dict(x=P, xd=BF16, ldx=64, r=None, ldr=0, w=P, eps=1e-6, t=4, n=64, h=None, ldh=0, y=P, yd=E4, ldy=64, s=P)
    v.update(k)
    return L.rms_norm(v["x"], v["xd"], v["ldx"], v["r"], v["ldr"], v["w"], v["eps"], v["t"], v["n"], v["h"], v["ldh"],
                      v["y"], v["yd"], v["ldy"], v["s"], None)


@pytest.mark.parametrize("code,args", [
    (DTYPE, dict(xd=2)), (DTYPE, dict(xd=7)), (DTYPE, dict(yd=3)), (SHAPE, dict(t=-1)), (SHAPE, dict(n=0)),
    (SHAPE, dict(n=65537, ldx=65537, ldy=65537)), (SHAPE, dict(ldx=63)), (SHAPE, dict(ldy=63)),
    (SHAPE, dict(r=P, ldr=63, h=P, ldh=64)), (SHAPE, dict(r=P, ldr=64, h=P, ldh=63)), (SHAPE, dict(eps=-1.0)),
    (SHAPE, dict(eps=float("nan"))), (SHAPE, dict(eps=float("inf"))), (UNSUP, dict(t=1 << 22)), (SHAPE, dict(t=1 << 31)),
    (NULL, dict(x=None)), (NULL, dict(y=None)), (NULL, dict(s=None)), (NULL, dict(w=None)),
    (NULL, dict(r=P, ldr=64, ldh=64)), (UNSUP, dict(h=P, ldh=64)), (ALIGN, dict(x=P + 1)), (ALIGN, dict(w=P + 2)),
    (ALIGN, dict(s=P + 2)), (ALIGN, dict(xd=F32, x=P + 2)), (ALIGN, dict(yd=F32, y=P + 2)),
    (ALIGN, dict(r=P + 1, ldr=64, h=P, ldh=64)), (ALIGN, dict(r=P, ldr=64, h=P + 1, ldh=64)),
    (OK, dict(t=0, x=None, y=None, w=None, s=None))])
def test_norm_refusals(L, code, args):
    assert _norm(L, **args) == code


@pytest.mark.parametrize("code,args", [
    (UNSUP, dict(act=4)), (UNSUP, dict(act=-1)), (DTYPE, dict(xd=2)), (DTYPE, dict(yd=-1)), (SHAPE, dict(n=0)),
    (SHAPE, dict(ldu=63)), (SHAPE, dict(ldg=1)), (NULL, dict(g=None)), (NULL, dict(y=None)), (NULL, dict(s=None)),
    (ALIGN, dict(u=P + 1)), (OK, dict(t=0))])
def test_gate_refusals(L, code, args):
    v = dict(g=P, xd=BF16, ldg=64, u=P, ldu=64, act=3, t=4, n=64, y=P, yd=E4, ldy=64, s=P)
    v.update(args)
    assert L.gated_act(v["g"], v["xd"], v["ldg"], v["u"], v["ldu"], v["act"], v["t"], v["n"], v["y"], v["yd"], v["ldy"],
                       v["s"], None) == code


@pytest.mark.parametrize("code,args", [
    (DTYPE, dict(d=2)), (SHAPE, dict(M=-1)), (UNSUP, dict(K=96, ld=96)), (SHAPE, dict(ld=60)), (UNSUP, dict(M=1 << 24)),
    (UNSUP, dict(M=1 << 20, K=1 << 20, ld=1 << 20)), (NULL, dict(W=None)), (NULL, dict(data=None)), (NULL, dict(s=None)),
    (ALIGN, dict(W=P + 2)), (ALIGN, dict(data=P + 8)), (ALIGN, dict(s=P + 1)), (OK, dict(M=0))])
def test_compress_refusals(L, code, args):
    v = dict(W=P, d=F32, M=8, K=64, ld=64, data=P, s=P)
    v.update(args)
    assert L.prune24_compress_f8(v["W"], v["d"], v["M"], v["K"], v["ld"], v["data"], v["s"], None) == code
    if "d" not in args:
        W = v["W"]
        assert L.prune24_decompress_f8(v["data"], v["s"], v["M"], v["K"], W, v["ld"], None) == code


@pytest.mark.parametrize("code,args", [
    (DTYPE, dict(yd=2)), (UNSUP, dict(act=9)), (SHAPE, dict(N=-1)), (SHAPE, dict(ldx=48)), (SHAPE, dict(ldy=31)),
    (SHAPE, dict(r=P, ldr=31)), (UNSUP, dict(K=96, ldx=96)), (UNSUP, dict(K=0)), (UNSUP, dict(ldx=1 << 23)),
    (UNSUP, dict(M=1 << 24, ldy=1 << 24)), (UNSUP, dict(N=1 << 21)), (NULL, dict(data=None)), (NULL, dict(ws=None)),
    (NULL, dict(X=None)), (NULL, dict(xs=None)), (NULL, dict(Y=None)), (ALIGN, dict(data=P + 4)), (ALIGN, dict(X=P + 4)),
    (ALIGN, dict(ldx=72)), (ALIGN, dict(Y=P + 1)), (ALIGN, dict(r=P + 1, ldr=32)), (ALIGN, dict(b=P + 2)),
    (ALIGN, dict(xs=P + 2)), (ALIGN, dict(ws=P + 2)), (OK, dict(N=0, X=None)), (OK, dict(M=0, ldy=0, data=None))])
def test_product_refusals(L, code, args):
    v = dict(data=P, ws=P, M=32, K=64, X=P, ldx=64, xs=P, N=4, Y=P, yd=BF16, ldy=32, b=None, act=0, r=None, ldr=0)
    v.update(args)
    assert L.spmm24_f8(v["data"], v["ws"], v["M"], v["K"], v["X"], v["ldx"], v["xs"], v["N"], v["Y"], v["yd"], v["ldy"],
                       v["b"], v["act"], v["r"], v["ldr"], None) == code


def test_rows_of_no_values_have_scales(L):
    assert L.prune24_compress_f8(None, F32, 8, 0, 0, None, None, None) == NULL
    assert L.prune24_compress_f8(None, F32, 0, 0, 0, None, None, None) == OK


def test_a_single_token_has_no_stride(L):
    """One token's leading dimension passes the checks on it, and the call comes to its other arguments."""
    for ldx in (72, 1 << 23):
        many, one = (L.spmm24_f8(None, P, 32, 64, P, ldx, P, n, P, BF16, 32, None, 0, None, 0, None) for n in (2, 1))
        assert one == NULL and many == (UNSUP if ldx == 1 << 23 else NULL)


class _Dev:
    """A tensor's face for the binding's checks: a CPU tensor that says it is on the device."""

    def __init__(self, t, dev="cuda:0"):
        self.t, self.device, self.is_cuda = t, torch.device(dev), True

    def __getattr__(self, k):
        return getattr(self.t, k)


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    q = p24.Quantized8(torch.zeros(4, 64).to(F8), torch.ones(4))
    c = p24.Compressed24F8(torch.zeros(10240, dtype=torch.uint8), torch.ones(32), 32, 64)
    for call in (lambda: p24.rms_norm(x, w), lambda: p24.gated_act(x), lambda: p24.compress_f8(w[None]),
                 lambda: p24.spmm24_f8(c, q)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    dx, dw = _Dev(x), _Dev(w)
    with pytest.raises(ValueError, match="unit stride"):
        p24.rms_norm(_Dev(torch.zeros(64, 4, dtype=torch.bfloat16).t()), dw)
    with pytest.raises(ValueError, match="2-D"):
        p24.rms_norm(_Dev(x[0]), dw)
    with pytest.raises(ValueError, match="not one of"):
        p24.rms_norm(_Dev(x.half()), dw)
    with pytest.raises(ValueError, match="weight"):
        p24.rms_norm(dx, _Dev(w[:63]))
    with pytest.raises(ValueError, match="weight"):
        p24.rms_norm(dx, _Dev(w.double()))
    with pytest.raises(ValueError, match="residual is"):
        p24.rms_norm(dx, dw, residual=_Dev(x.float()))
    with pytest.raises(ValueError, match="residual is"):
        p24.rms_norm(dx, dw, residual=_Dev(x[:3]))
    with pytest.raises(ValueError, match="residual is on"):
        p24.rms_norm(dx, dw, residual=_Dev(x, "cuda:1"))
    with pytest.raises(ValueError, match="there is none"):
        p24.rms_norm(dx, dw, h=dx)
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="eps"):
            p24.rms_norm(dx, dw, eps=eps)
    with pytest.raises(ValueError, match="out_dtype"):
        p24.rms_norm(dx, dw, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="act"):
        p24.gated_act(dx, act="tanh")
    with pytest.raises(ValueError, match="up is"):
        p24.gated_act(dx, _Dev(x[:, :63]))
    dq = p24.Quantized8(_Dev(q.values), _Dev(q.scale))
    dc = p24.Compressed24F8(_Dev(c.data), _Dev(c.scale), 32, 64)
    with pytest.raises(ValueError, match="features"):
        p24.spmm24_f8(p24.Compressed24F8(dc.data, dc.scale, 32, 128), dq)
    with pytest.raises(ValueError, match="compressed form"):
        p24.spmm24_f8(p24.Compressed24F8(_Dev(c.data[:5120]), dc.scale, 32, 64), dq)
    with pytest.raises(ValueError, match="compressed form"):
        p24.decompress_f8(p24.Compressed24F8(_Dev(c.data.to(torch.int32)), dc.scale, 32, 64))
    with pytest.raises(ValueError, match="weight's scale"):
        p24.spmm24_f8(p24.Compressed24F8(dc.data, _Dev(torch.ones(31)), 32, 64), dq)
    with pytest.raises(ValueError, match="the weight is on"):
        p24.spmm24_f8(p24.Compressed24F8(_Dev(c.data, "cuda:1"), dc.scale, 32, 64), dq)
    with pytest.raises(ValueError, match="act"):
        p24.spmm24_f8(dc, dq, act="swish")
    with pytest.raises(ValueError, match="bias"):
        p24.spmm24_f8(dc, dq, bias=_Dev(torch.zeros(31)))
    with pytest.raises(ValueError, match="X.scale"):
        p24.spmm24_f8(dc, p24.Quantized8(dq.values, _Dev(torch.ones(5))))
    with pytest.raises(ValueError, match="out_dtype"):
        p24.spmm24_f8(dc, dq, out_dtype=F8)
    with pytest.raises(ValueError, match="out is"):
        p24.spmm24_f8(dc, dq, out=_Dev(torch.zeros(4, 31)))
    with pytest.raises(ValueError, match="W_gate_up"):
        p24.feed_forward_f8(dx, None, dw, dc, dc)


def test_a_single_row_has_no_stride_of_its_own():
    from structured_sparse_gemm_prune24_amd import f8
    t = torch.as_strided(torch.zeros(64), (1, 64), (1, 1))
    assert f8._rows(_Dev(t), "t", torch.device("cuda:0"), (torch.float32,)) == 64
    t = torch.as_strided(torch.zeros(64), (4, 1), (16, 7))
    assert f8._rows(_Dev(t), "t", torch.device("cuda:0"), (torch.float32,)) == 16


@pytest.mark.parametrize("seed", range(2))
def test_layout_through_the_lane_model(seed):
    """The packed bytes, read as the kernel's lanes read them and multiplied by the instruction's
    model, are the product of the pruned matrix: exact on whole numbers."""
    rng = np.random.default_rng(seed)
    M, K, N = 96, 192, 32
    W = rng.integers(-6, 7, (M, K)).astype(np.float32)
    W[:, 0] = 7
    bits, pos, scale = compress(W)
    data = pack(bits, pos, M, K).reshape(-1, 5120)          # one row group: [step]
    X = rng.integers(-8, 9, (N, K)).astype(np.float64)
    got = np.zeros((M, N))
    for rb in range(3):
        D = np.zeros((64, 16))
        for s in range(K // 64):
            piece = data[s]
            a = f8_values(piece[1024 * rb:1024 * (rb + 1)].reshape(64, 16))
            words = piece[4096 + 256 * rb:4096 + 256 * (rb + 1)].view(np.uint32)
            b = np.zeros((64, 32))
            for lane in range(64):
                n, h = lane % 32, lane // 32
                b[lane] = np.concatenate([X[n, 64 * s + 16 * h:][:16], X[n, 64 * s + 32 + 16 * h:][:16]])
            D += smfmac64_model(a, b, words)
        for lane in range(64):
            for i in range(16):
                got[32 * rb + 8 * (i // 4) + 4 * (lane // 32) + i % 4, lane % 32] = D[lane, i]
    want = decompress(bits, pos, scale, K) @ X.T / scale[:, None]
    assert np.array_equal(got, want)
