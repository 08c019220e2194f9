"""Host-side checks of the expert operators and of the block-scaled 8-bit ones (no GPU): exports, argument
refusals of the C entry points and of the binding (fake pointers, never dereferenced), and the places that their
direct-to-LDS loads read, computed by the functions that the kernels use."""
import ctypes
import os
import subprocess

import pytest

from test_f8_host import _Dev

torch = pytest.importorskip("torch")
p24 = pytest.importorskip("structured_sparse_gemm_prune24_amd")
OK, NULL, SHAPE, ALIGN, DTYPE, UNSUP, WS = (p24.P24_OK, p24.P24_ERR_NULL, p24.P24_ERR_SHAPE, p24.P24_ERR_ALIGN,
                                            p24.P24_ERR_DTYPE, p24.P24_ERR_UNSUPPORTED, p24.P24_ERR_WORKSPACE)
P = 1 << 20
F32, BF16, E4 = 0, 1, 2
F8 = torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    return p24.lib()


@pytest.mark.parametrize("header,table", [("EXPERTS_HEADER_PATH", "_EXPERTS_SIGNATURES"),
                                          ("F8_BLOCK_HEADER_PATH", "_F8_BLOCK_SIGNATURES")])
def test_exports(L, header, table):
    syms = p24.header_symbols(getattr(p24, header))
    assert len(syms) == len(set(syms)) and set(syms) == set(getattr(p24, table))
    for s in syms:
        assert hasattr(L, s), s


# ---- C entry points ---------------------------------------------------------
@pytest.mark.parametrize("code,args", [
    (DTYPE, dict(d=2)), (SHAPE, dict(T=-1)), (SHAPE, dict(E=0, k=0)), (SHAPE, dict(k=0)), (SHAPE, dict(k=9)), (SHAPE, dict(ld=7)),
    (SHAPE, dict(scale=INF)), (SHAPE, dict(scale=NAN)), (UNSUP, dict(score=2)), (UNSUP, dict(score=-1)), (UNSUP, dict(b=P)),
    (UNSUP, dict(E=1025, ld=1025)), (UNSUP, dict(E=64, k=33, ld=64)), (UNSUP, dict(T=(1 << 18) + 1)), (NULL, dict(l=None)),
    (NULL, dict(e=None)), (NULL, dict(w=None)), (NULL, dict(o=None)), (NULL, dict(t=None)), (NULL, dict(p=None)),
    (NULL, dict(T=65, ws=None)), (ALIGN, dict(l=P + 1)), (ALIGN, dict(d=F32, l=P + 2)), (ALIGN, dict(e=P + 2)),
    (ALIGN, dict(o=P + 1)), (ALIGN, dict(t=P + 3)), (ALIGN, dict(p=P + 2)), (ALIGN, dict(w=P + 2)),
    (ALIGN, dict(score=1, b=P + 1)), (ALIGN, dict(T=65, ws=P + 2)), (WS, dict(T=65, n=4 * 8 * 4 - 1)), (WS, dict(T=65, n=0))])
def test_route_refusals(L, code, args):
    v = dict(l=P, d=BF16, ld=8, T=4, E=8, k=2, score=0, b=None, norm=1, scale=1.0, e=P, w=P, o=P, t=P, p=P, ws=P, n=1 << 20)
    v.update(args)
    assert L.experts_route(v["l"], v["d"], v["ld"], v["T"], v["E"], v["k"], v["score"], v["b"], v["norm"], v["scale"], v["e"],
                           v["w"], v["o"], v["t"], v["p"], v["ws"], v["n"], None) == code


def test_route_workspace(L):
    assert L.experts_route_workspace(64, 256) == 0 and L.experts_route_workspace(0, 8) == 0
    assert L.experts_route_workspace(65, 8) == 4 * 8 * 4           # three groups of 32 tokens, and the sums
    assert L.experts_route_workspace(8192, 256) == 257 * 256 * 4
    assert L.experts_route_workspace(100, 0) == 0


@pytest.mark.parametrize("code,args", [
    (DTYPE, dict(yd=2)), (UNSUP, dict(act=9)), (SHAPE, dict(E=0)), (SHAPE, dict(R=-1)), (SHAPE, dict(xr=-1)), (SHAPE, dict(ldx=48)),
    (SHAPE, dict(ldy=31)), (SHAPE, dict(xr=5)), (SHAPE, dict(xr=0, t=P)), (UNSUP, dict(E=1025)), (UNSUP, dict(K=96, ldx=96)),
    (UNSUP, dict(K=0)), (UNSUP, dict(ldx=1 << 23)), (UNSUP, dict(M=1 << 24, ldy=1 << 24)), (UNSUP, dict(R=1 << 21, xr=1 << 21)),
    (UNSUP, dict(t=P, xr=1 << 26)), (UNSUP, dict(t=P, xr=(1 << 31) - 1)), (NULL, dict(data=None)), (NULL, dict(ws=None)),
    (NULL, dict(X=None)), (NULL, dict(xs=None)), (NULL, dict(Y=None)), (NULL, dict(o=None)), (ALIGN, dict(data=P + 4)),
    (ALIGN, dict(X=P + 4)), (ALIGN, dict(ldx=72)), (ALIGN, dict(Y=P + 1)), (ALIGN, dict(b=P + 2)), (ALIGN, dict(xs=P + 2)),
    (ALIGN, dict(ws=P + 2)), (ALIGN, dict(o=P + 2)), (ALIGN, dict(t=P + 1)), (OK, dict(R=0, xr=0, X=None)),
    (OK, dict(M=0, ldy=0, data=None))])
def test_grouped_refusals(L, code, args):
    v = dict(data=P, ws=P, E=3, M=32, K=64, X=P, ldx=64, xs=P, xr=4, o=P, t=None, R=4, Y=P, yd=BF16, ldy=32, b=None, act=0)
    v.update(args)
    assert L.spmm24_f8_grouped(v["data"], v["ws"], v["E"], v["M"], v["K"], v["X"], v["ldx"], v["xs"], v["xr"], v["o"], v["t"],
                               v["R"], v["Y"], v["yd"], v["ldy"], v["b"], v["act"], None) == code


@pytest.mark.parametrize("code,args", [
    (DTYPE, dict(zd=2)), (DTYPE, dict(yd=2)), (SHAPE, dict(T=-1)), (SHAPE, dict(R=-1)), (SHAPE, dict(R=1 << 31)), (SHAPE, dict(k=0)),
    (SHAPE, dict(n=0)), (SHAPE, dict(n=65537, ldz=65537, ldy=65537)), (SHAPE, dict(ldz=63)), (SHAPE, dict(ldy=63)),
    (SHAPE, dict(r=P, ldr=63)), (UNSUP, dict(k=33)), (UNSUP, dict(T=1 << 22)), (NULL, dict(z=None)), (NULL, dict(p=None)),
    (NULL, dict(w=None)), (NULL, dict(y=None)), (ALIGN, dict(z=P + 1)), (ALIGN, dict(y=P + 1)), (ALIGN, dict(r=P + 1, ldr=64)),
    (ALIGN, dict(p=P + 2)), (ALIGN, dict(w=P + 2)), (OK, dict(T=0, z=None, y=None))])
def test_combine_refusals(L, code, args):
    v = dict(z=P, zd=BF16, ldz=64, R=8, p=P, w=P, T=4, k=2, n=64, r=None, ldr=0, y=P, yd=BF16, ldy=64)
    v.update(args)
    assert L.experts_combine(v["z"], v["zd"], v["ldz"], v["R"], v["p"], v["w"], v["T"], v["k"], v["n"], v["r"], v["ldr"], v["y"],
                             v["yd"], v["ldy"], None) == code


@pytest.mark.parametrize("code,args", [
    (DTYPE, dict(d=2)), (UNSUP, dict(act=4)), (SHAPE, dict(T=-1)), (SHAPE, dict(n=0)), (SHAPE, dict(ld=63)), (SHAPE, dict(ldv=63)),
    (SHAPE, dict(u=P, ldu=63)), (SHAPE, dict(lds=3)), (UNSUP, dict(n=1 << 24, ld=1 << 24, ldv=1 << 24)),
    (UNSUP, dict(T=65535 * 16 + 1, lds=1 << 21)), (NULL, dict(x=None)), (NULL, dict(v=None)), (NULL, dict(s=None)),
    (ALIGN, dict(x=P + 1)), (ALIGN, dict(u=P + 1, ldu=64)), (ALIGN, dict(s=P + 2)), (OK, dict(T=0, x=None, lds=0))])
def test_quantize_refusals(L, code, args):
    a = dict(x=P, d=BF16, ld=64, u=None, ldu=0, act=0, T=4, n=64, v=P, ldv=64, s=P, lds=4)
    a.update(args)
    assert L.quantize_f8_block(a["x"], a["d"], a["ld"], a["u"], a["ldu"], a["act"], a["T"], a["n"], a["v"], a["ldv"], a["s"],
                               a["lds"], None) == code


@pytest.mark.parametrize("code,args", [
    (DTYPE, dict(d=2)), (SHAPE, dict(M=-1)), (SHAPE, dict(ld=63)), (SHAPE, dict(ldv=63)), (UNSUP, dict(M=1 << 22)),
    (UNSUP, dict(K=1 << 22, ld=1 << 22, ldv=1 << 22)), (NULL, dict(W=None)), (NULL, dict(v=None)), (NULL, dict(s=None)),
    (ALIGN, dict(W=P + 2)), (ALIGN, dict(s=P + 1)), (OK, dict(M=0, W=None))])
def test_quantize_weight_refusals(L, code, args):
    a = dict(W=P, d=F32, M=8, K=64, ld=64, v=P, ldv=64, s=P)
    a.update(args)
    assert L.quantize_weight_f8_block(a["W"], a["d"], a["M"], a["K"], a["ld"], a["v"], a["ldv"], a["s"], None) == code


@pytest.mark.parametrize("code,args", [
    (DTYPE, dict(yd=2)), (UNSUP, dict(act=9)), (SHAPE, dict(N=-1)), (SHAPE, dict(M=-1)), (SHAPE, dict(ldx=48)), (SHAPE, dict(ldw=48)),
    (SHAPE, dict(ldxs=3)), (SHAPE, dict(ldy=31)), (SHAPE, dict(r=P, ldr=31)), (UNSUP, dict(K=72, ldx=80, ldw=80)),
    (UNSUP, dict(K=0)), (UNSUP, dict(ldx=1 << 23)), (UNSUP, dict(ldw=1 << 23)), (UNSUP, dict(M=1 << 24, ldy=1 << 24)),
    (UNSUP, dict(N=65535 * 16 + 1, ldxs=1 << 21)), (UNSUP, dict(ldxs=1 << 30)), (NULL, dict(W=None)), (NULL, dict(ws=None)),
    (NULL, dict(X=None)), (NULL, dict(xs=None)), (NULL, dict(Y=None)), (ALIGN, dict(W=P + 8)), (ALIGN, dict(X=P + 8)),
    (ALIGN, dict(ldw=72)), (ALIGN, dict(ldx=72)), (ALIGN, dict(Y=P + 1)), (ALIGN, dict(r=P + 1, ldr=32)), (ALIGN, dict(b=P + 2)),
    (ALIGN, dict(ws=P + 2)), (ALIGN, dict(xs=P + 2)), (OK, dict(N=0, X=None)), (OK, dict(M=0, ldy=0, W=None))])
def test_block_product_refusals(L, code, args):
    v = dict(W=P, ldw=64, ws=P, M=32, K=64, X=P, ldx=64, xs=P, ldxs=4, N=4, Y=P, yd=BF16, ldy=32, b=None, act=0, r=None, ldr=0)
    v.update(args)
    assert L.gemm_f8_block(v["W"], v["ldw"], v["ws"], v["M"], v["K"], v["X"], v["ldx"], v["xs"], v["ldxs"], v["N"], v["Y"], v["yd"],
                           v["ldy"], v["b"], v["act"], v["r"], v["ldr"], None) == code


# ---- binding ----------------------------------------------------------------
def _raises(match, call):
    with pytest.raises(ValueError, match=match):
        call()


def test_routing_and_combination_refusals():
    l, b = torch.zeros(4, 8), torch.zeros(8)
    _raises("device tensor", lambda: p24.route(l, 2))
    d = _Dev(l)
    _raises("score", lambda: p24.route(d, 2, score="tanh"))
    for k in (0, 9, -1):
        _raises("k is", lambda: p24.route(d, k))
    _raises("scale", lambda: p24.route(d, 2, scale=INF))
    _raises("bias goes", lambda: p24.route(d, 2, bias=_Dev(b)))
    _raises("bias", lambda: p24.route(d, 2, score="sigmoid", bias=_Dev(b[:7])))
    _raises("not one of", lambda: p24.route(_Dev(l.half()), 2))
    _raises("unit stride", lambda: p24.route(_Dev(torch.zeros(8, 4).t()), 2))
    z, p, w = torch.zeros(8, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    _raises("device tensor", lambda: p24.combine_experts(z, p, w))
    dz, dp, dw = _Dev(z), _Dev(p), _Dev(w)
    _raises("positions", lambda: p24.combine_experts(dz, _Dev(p.long()), dw))
    _raises("2-D", lambda: p24.combine_experts(dz, _Dev(p[0]), dw))
    _raises("weights", lambda: p24.combine_experts(dz, dp, _Dev(w[:, :1])))
    _raises("weights", lambda: p24.combine_experts(dz, dp, _Dev(w.double())))
    _raises("residual is", lambda: p24.combine_experts(dz, dp, dw, residual=_Dev(torch.zeros(4, 15)), out=_Dev(torch.zeros(4, 16))))
    _raises("out_dtype", lambda: p24.combine_experts(dz, dp, dw, out_dtype=torch.float16))
    _raises("out is", lambda: p24.combine_experts(dz, dp, dw, out=_Dev(torch.zeros(3, 16))))


def test_grouped_binding_refusals():
    c = p24.Experts24F8(torch.zeros(2 * 10240, dtype=torch.uint8), torch.ones(2, 32), 2, 32, 64)
    q = p24.Quantized8(torch.zeros(4, 64).to(F8), torch.ones(4))
    off = torch.zeros(3, dtype=torch.int32)
    _raises("device tensor", lambda: p24.spmm24_f8_grouped(c, q, off))
    dc = p24.Experts24F8(_Dev(c.data), _Dev(c.scale), 2, 32, 64)
    dq, do = p24.Quantized8(_Dev(q.values), _Dev(q.scale)), _Dev(off)
    _raises("features", lambda: p24.spmm24_f8_grouped(p24.Experts24F8(dc.data, dc.scale, 2, 32, 128), dq, do))
    _raises("compressed form", lambda: p24.spmm24_f8_grouped(p24.Experts24F8(dc.data, dc.scale, 3, 32, 64), dq, do))
    _raises("weights' scale", lambda: p24.spmm24_f8_grouped(p24.Experts24F8(dc.data, _Dev(torch.ones(64)), 2, 32, 64), dq, do))
    _raises("weights are on", lambda: p24.spmm24_f8_grouped(p24.Experts24F8(_Dev(c.data, "cuda:1"), dc.scale, 2, 32, 64), dq, do))
    _raises("X.scale", lambda: p24.spmm24_f8_grouped(dc, p24.Quantized8(dq.values, _Dev(torch.ones(5))), do))
    _raises("offsets", lambda: p24.spmm24_f8_grouped(dc, dq, _Dev(off[:2])))
    _raises("offsets", lambda: p24.spmm24_f8_grouped(dc, dq, _Dev(off.long())))
    _raises("tokens", lambda: p24.spmm24_f8_grouped(dc, dq, do, tokens=_Dev(torch.zeros(2, 2, dtype=torch.int32))))
    _raises("bias", lambda: p24.spmm24_f8_grouped(dc, dq, do, bias=_Dev(torch.zeros(32))))
    _raises("act", lambda: p24.spmm24_f8_grouped(dc, dq, do, act="swish"))
    _raises("out_dtype", lambda: p24.spmm24_f8_grouped(dc, dq, do, out_dtype=F8))
    _raises("out is", lambda: p24.spmm24_f8_grouped(dc, dq, do, out=_Dev(torch.zeros(4, 31))))
    _raises("no experts", lambda: p24.compress_f8_experts([]))
    _raises("W_gate_up", lambda: p24.feed_forward_f8_experts(dq, _Dev(torch.zeros(4, 2)), 1, dc, dc))


def test_block_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = p24.Weight8Block(_Dev(torch.zeros(32, 64).to(F8)), _Dev(torch.ones(1, 1)))
    q = p24.Rows8Block(_Dev(torch.zeros(4, 64).to(F8)), _Dev(torch.ones(1, 4)))
    _raises("device tensor", lambda: p24.quantize_f8_block(x))
    _raises("device tensor", lambda: p24.quantize_weight_f8_block(x))
    _raises("no features", lambda: p24.quantize_f8_block(_Dev(x[:, :0])))
    _raises("act", lambda: p24.quantize_f8_block(_Dev(x), act="tanh"))
    _raises("up is", lambda: p24.quantize_f8_block(_Dev(x), _Dev(x[:, :63])))
    _raises("not one of", lambda: p24.quantize_f8_block(_Dev(x.half())))
    _raises("features", lambda: p24.gemm_f8_block(p24.Weight8Block(_Dev(torch.zeros(32, 128).to(F8)), w.scale), q))
    _raises("not one of", lambda: p24.gemm_f8_block(p24.Weight8Block(_Dev(torch.zeros(32, 64)), w.scale), q))
    _raises("weight's scale", lambda: p24.gemm_f8_block(p24.Weight8Block(w.values, _Dev(torch.ones(2, 1))), q))
    _raises("weight's scale", lambda: p24.gemm_f8_block(p24.Weight8Block(w.values, _Dev(torch.ones(1, 1), "cuda:1")), q))
    _raises("X.scale", lambda: p24.gemm_f8_block(w, p24.Rows8Block(q.values, _Dev(torch.ones(4, 1)))))
    _raises("X.scale", lambda: p24.gemm_f8_block(w, p24.Rows8Block(q.values, _Dev(torch.ones(1, 8)[:, ::2]))))
    _raises("bias", lambda: p24.gemm_f8_block(w, q, bias=_Dev(torch.zeros(31))))
    _raises("act", lambda: p24.gemm_f8_block(w, q, act="swish"))
    _raises("out_dtype", lambda: p24.gemm_f8_block(w, q, out_dtype=F8))
    _raises("out is", lambda: p24.gemm_f8_block(w, q, out=_Dev(torch.zeros(4, 31))))
    _raises("W_gate_up", lambda: p24.feed_forward_f8_block(_Dev(x), None, _Dev(torch.ones(64)), w, w))


# ---- places of the loads ----------------------------------------------------
@pytest.fixture(scope="module")
def model(tmp_path_factory):
    here = os.path.dirname(os.path.abspath(__file__))
    so = str(tmp_path_factory.mktemp("reads") / "block_reads.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-shared", "-fPIC", os.path.join(here, "host_model", "block_reads.cpp"),
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    i64 = ctypes.c_int64
    lib.block_bad_reads.restype = lib.grouped_bad_reads.restype = ctypes.c_long
    lib.block_bad_reads.argtypes = [ctypes.c_int] + [i64] * 5
    lib.grouped_bad_reads.argtypes = [ctypes.c_int] + [i64] * 4
    return lib


@pytest.mark.parametrize("tile", range(9))
def test_block_tiles_read_inside_their_matrices(model, tile):
    """Values and scales: one token or row up to more than the widest tile, K of whole and part blocks and less
    than one, groups of waves with even and uneven parts of K, wide rows."""
    for M in (1, 9, 64, 127, 129, 256, 300, 520):
        for N in (1, 7, 33, 64, 130, 257):
            for K, pad in ((16, 0), (128, 0), (208, 48), (1040, 16), (1280, 4096)):
                assert model.block_bad_reads(tile, M, N, K, K + pad, N + pad // 16) == 0, (M, N, K, pad)


@pytest.mark.parametrize("tile", range(7))
def test_grouped_tiles_read_inside_their_rows(model, tile):
    """Rows of X by any index, as the kernel clips it, from one row up to more than a tile's."""
    for rows in (1, 7, 64, 129, 257):
        for x_rows in (1, 3, 300):
            for K, pad in ((64, 0), (192, 48), (1024, 16)):
                assert model.grouped_bad_reads(tile, rows, x_rows, K, K + pad) == 0, (rows, x_rows, K, pad)
