"""GPU parity of the 8-bit feed-forward operators against fp64 formulas: RMS norm, gated
activation, 2:4 compression into 8-bit rows, and the 2:4 product with its epilogue.

Tolerances count roundings (U = 2^-24 is half an fp32 step, relative).
Norm: the sum h is rounded once (U), its squares and their sum lose at most 8 values a chunk, 8
chunks a thread, 6 wave steps and 16 waves (94 U, half of that under the root), the root and the
quotients 6 U, the two products 2 U: 64 U of |y|, and twice that where y goes over the scale.
An 8-bit value is half an e4m3 step off: 2^-4 of itself, or 2^-10 (half the subnormal step) times
the scale.
Product: 8-bit products are exact in fp32; K / 2 of them are summed in fp32, each addition at most
one step (2 U) of the largest partial sum, which sum |w x| bounds.  With a bf16 output the 8-bit
matrix unit adds eight products at a time, seven of them cut to 2^-13 of the largest: another
7 * 2^-13 of sum |w x| at most.  (On small whole numbers nothing is cut: those are exact.)"""
import numpy as np
import pytest

from f8_ref import F8, HALF, TINY, U, act, act_error, compress as ref_compress, decompress, pack, row_scale, smfmac64_model
from gpu_util import need_gpu, torch

p24 = pytest.importorskip("structured_sparse_gemm_prune24_amd")
pytestmark = pytest.mark.gpu
D = torch.float64


def _rows(seed, tokens, width, pad, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    full = torch.randn(tokens, width + pad, generator=g, device="cuda")
    full[:, ::7] *= 8
    return full.to(dtype)[:, :width]


def _check_rows(got, y, rel, out):
    """got against fp64 y with relative error `rel` (a tensor or number) before the last rounding."""
    if out == F8:
        s = row_scale(y)
        worst = float(rel.max()) if torch.is_tensor(rel) else rel
        assert torch.all((got.scale.to(D) - s).abs() <= (worst + 4 * U) * s)
        v = got.values.to(D) * got.scale.to(D)[:, None]
        tol = (HALF[F8] + 2 * rel + 2 * worst + 8 * U) * y.abs() + 2.0 ** -10 * (1 + 2 * worst + 8 * U) * s[:, None]
        assert got.values.to(torch.float32).abs().max() <= 448
    else:
        v = got.to(D)
        assert got.dtype == out
        tol = (HALF[out] + rel * (1 + HALF[out])) * y.abs() + 1e-36     # fp32 subnormals may flush
    off = (v - y).abs()
    assert torch.all(off <= tol), float((off / tol.clamp_min(1e-300)).max())


NORM_SHAPES = [(1, 1, 0), (1, 64, 0), (3, 7, 2), (5, 511, 1), (4, 512, 0), (2, 513, 3), (7, 1003, 5), (2, 2048, 0),
               (3, 2049, 7), (1, 4096, 0), (9, 4097, 0), (2, 8192, 8), (2, 8193, 0), (1, 16385, 1), (2, 40001, 3),
               (1, 65536, 0), (2, 65536, 1), (300, 128, 0), (1025, 260, 4), (1030, 700, 1), (5, 120, 1), (9, 250, 1),
               (3, 4095, 0), (2, 5121, 2), (2, 9000, 1)]


@pytest.mark.parametrize("out", [F8, torch.bfloat16, torch.float32], ids=["f8", "bf16", "f32"])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32], ids=["xbf16", "xf32"])
@pytest.mark.parametrize("tokens,width,pad", NORM_SHAPES)
def test_norm(tokens, width, pad, stream, out):
    need_gpu()
    w = 1 + 0.1 * _rows(9, 1, width, 0, torch.float32)[0]
    for with_r in (False, True):
        x = _rows(1, tokens, width, pad, stream)
        r = _rows(2, tokens, width, pad + 1, stream) if with_r else None
        y, h = p24.rms_norm(x, w, residual=r, out_dtype=out)
        e = x.to(D) + r.to(D) if with_r else x.to(D)
        if with_r:
            assert h.dtype == stream
            assert torch.all((h.to(D) - e).abs() <= (U + HALF[stream] * (1 + U)) * e.abs())
        else:
            assert h is None
        e = e / torch.sqrt(e.square().mean(dim=1, keepdim=True) + 1e-6) * w.to(D)
        _check_rows(y, e, 64 * U, out)


@pytest.mark.parametrize("out", [F8, torch.bfloat16, torch.float32], ids=["f8", "bf16", "f32"])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32], ids=["xbf16", "xf32"])
@pytest.mark.parametrize("name", ["silu", "gelu", "relu", "none"])
@pytest.mark.parametrize("tokens,width,pad", [(1, 1, 0), (3, 7, 2), (4, 512, 0), (7, 1003, 5), (2, 4096, 8),
                                              (2, 8193, 0), (4, 11264, 0), (1, 40001, 1), (777, 130, 0)])
def test_gate(tokens, width, pad, name, stream, out):
    need_gpu()
    both = _rows(3, tokens, 2 * width, pad, stream)
    for with_up in (True, False):
        gate, up = both[:, :width], both[:, width:] if with_up else None
        got = p24.gated_act(gate, up, act=name, out_dtype=out)
        z = gate.to(D)
        e = act(z, name)
        rel = act_error(z, name, out) + U
        if with_up:
            e = e * up.to(D)
        _check_rows(got, e, rel, out)


@pytest.mark.parametrize("kind", ["zero", "nan", "inf", "tiny", "lowest"])
def test_special_rows(kind):
    """Rows of zeros, a NaN, an infinity, values under the smallest scale, the type's lowest value:
    next to ordinary rows, which must not change."""
    need_gpu()
    x = _rows(5, 6, 700, 0, torch.float32)
    clean = p24.gated_act(x, act="none")
    bad = x.clone()
    if kind == "zero":
        bad[2] = 0
    elif kind == "tiny":
        bad[2] = 2.0 ** -130
    else:
        bad[2, 333] = {"nan": float("nan"), "inf": float("inf"), "lowest": torch.finfo(torch.float32).min}[kind]
    got = p24.gated_act(bad, act="none")
    y, _ = p24.rms_norm(bad, torch.ones(700, device="cuda"))
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(got.values.view(torch.uint8)[keep], clean.values.view(torch.uint8)[keep])
    assert torch.equal(got.scale[keep], clean.scale[keep])
    v, s = got.values.float()[2], got.scale[2].item()
    vn, sn = y.values.float()[2], y.scale[2].item()
    if kind == "zero":
        assert s == sn == float(TINY) and not v.any() and not vn.any()
    elif kind == "tiny":
        assert s == float(TINY) and not torch.isnan(v).any()
        assert torch.equal(v * 2.0 ** -126, torch.full_like(v, 2.0 ** -130))     # 2^-4 is an e4m3 value
    elif kind == "nan":
        assert np.isnan(s) and np.isnan(sn) and torch.isnan(v).all() and torch.isnan(vn).all()
    elif kind == "inf":
        assert np.isinf(s) and torch.isnan(v[333]) and not v[:333].any() and not v[334:].any()
        assert np.isnan(sn)                          # inf / inf in the norm itself
    else:
        assert v[333] == -448 and np.isfinite(s)


def test_norm_in_place_and_outputs():
    need_gpu()
    x, r = _rows(6, 33, 1000, 4, torch.bfloat16), _rows(7, 33, 1000, 0, torch.bfloat16)
    w = torch.rand(1000, device="cuda")
    y0, h0 = p24.rms_norm(x, w, residual=r)
    for alias in ("x", "r"):
        a, b = x.clone(), r.clone()
        y, h = p24.rms_norm(a, w, residual=b, h=a if alias == "x" else b)
        assert h is (a if alias == "x" else b)
        assert torch.equal(h, h0) and torch.equal(y.values.view(torch.uint8), y0.values.view(torch.uint8))
    big = p24.Quantized8(torch.zeros(33, 1100, dtype=torch.uint8, device="cuda").view(F8)[:, 50:1050],
                         torch.zeros(33, device="cuda"))
    y, _ = p24.rms_norm(x, w, residual=r, out=big)
    assert y is big and torch.equal(big.scale, y0.scale)
    whole = torch.as_strided(big.values.view(torch.uint8), (33, 1100), (1100, 1), 0)
    assert torch.equal(whole[:, 50:1050], y0.values.view(torch.uint8))
    assert not whole[:, :50].any() and not whole[:, 1050:].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 64), (31, 64), (33, 192), (128, 128), (129, 320), (200, 1088)])
def test_compress(M, K, dtype):
    """Bit for bit: selection, ties, 8-bit values, positions, padding and scales."""
    need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(M * K)
    W = torch.randn(M, K + 3, generator=g, device="cuda").to(dtype)[:, :K]
    W[:, ::5] = 0.5          # ties
    W[0] = 0
    c = p24.compress_f8(W)
    bits, pos, scale = ref_compress(W.float().cpu().numpy())
    assert np.array_equal(c.scale.cpu().numpy(), scale)
    assert np.array_equal(c.data.cpu().numpy(), pack(bits, pos, M, K))
    dense = p24.decompress_f8(c).cpu().numpy()
    assert np.array_equal(dense, decompress(bits, pos, scale, K).astype(np.float32))


def _weight(seed, M, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return p24.compress_f8(0.02 * torch.randn(M, K, generator=g, device="cuda"))


def _product_ref(c, x, bias, name, r, out):
    W = p24.decompress_f8(c).to(D)        # checked on its own above
    X = x.values.to(D) * x.scale.to(D)[:, None]
    z = X @ W.T
    err = ((c.K + 16) * U + (7 * 2.0 ** -13 if out == torch.bfloat16 else 0)) * (X.abs() @ W.abs().T)
    if bias is not None:
        z = z + bias.to(D)
        err = err + 2 * U * z.abs()
    e = act(z, name)
    err = 1.13 * err + act_error(z, name, out) * e.abs()      # no activation's slope passes 1.13
    if r is not None:
        e = e + r.to(D)
        err = err + U * e.abs()
    return e, err


def _check_product(c, x, bias=None, name="none", r=None, out=torch.bfloat16, Y=None):
    Y = p24.spmm24_f8(c, x, out_dtype=out, bias=bias, act=name, residual=r) if Y is None else Y
    e, err = _product_ref(c, x, bias, name, r, out)
    tol = err + HALF[out] * (e.abs() + err) + 1e-36
    assert Y.dtype == out and tuple(Y.shape) == tuple(e.shape)
    off = (Y.to(D) - e).abs()
    assert torch.all(off <= tol), float((off / tol).max())
    return Y


SIZES = [(1, 32, 64), (1, 1, 64), (2, 33, 128), (1, 4096, 4096), (3, 100, 192), (24, 1000, 512), (31, 64, 64),
         (32, 257, 320), (33, 129, 1088), (64, 512, 256), (65, 300, 128), (127, 96, 4032), (128, 128, 128),
         (200, 640, 704), (257, 513, 64), (517, 1000, 448), (700, 2304, 768), (1000, 255, 2048), (2048, 1024, 320)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,M,K", SIZES)
def test_product(N, M, K, out):
    need_gpu()
    c = _weight(M + K, M, K)
    x = p24.gated_act(_rows(N, N, K, 0, torch.float32), act="none")
    _check_product(c, x, out=out)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    bias = torch.randn(M, generator=g, device="cuda")
    r = torch.randn(N, M + 3, generator=g, device="cuda").to(out)[:, :M]
    for name in ("none", "relu", "gelu", "silu"):
        _check_product(c, x, bias=bias, name=name, r=r if name != "relu" else None, out=out)
    _check_product(c, x, r=r, out=out)


TILES = ["tokens", "64x32", "64x64", "128x64", "128x128", "256x128", "256x192", "256x256"]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,M,K", [(1, 1, 64), (33, 65, 128), (70, 300, 192), (129, 257, 448), (257, 260, 1024),
                                   (100, 129, 1088), (300, 513, 1472), (64, 128, 4160), (300, 520, 64),
                                   (260, 264, 256), (90, 272, 384), (513, 512, 512)])
@pytest.mark.parametrize("tile", TILES)
def test_product_of_every_kernel(monkeypatch, tile, N, M, K, out):
    """Each kernel at tokens, rows and K off its tile, K's parts within a block even and uneven; rows that the
    tile reaches past the output stay untouched."""
    need_gpu()
    monkeypatch.setenv("P24_F8_TILE", tile)
    c = _weight(M + K, M, K)
    x = p24.gated_act(_rows(N, N, K, 0, torch.float32), act="none")
    full = torch.full((N + 2, M + 5), 7.0, dtype=out, device="cuda")
    y = full[1:N + 1, :M]
    p24.spmm24_f8(c, x, out=y)
    _check_product(c, x, out=out, Y=y)
    assert (full[0] == 7).all() and (full[-1] == 7).all() and (full[:, M:] == 7).all()
    r = _rows(5, N, M, 3, out)
    bias = _rows(6, 1, M, 0, torch.float32)[0].contiguous()
    for name in ("gelu", "silu"):
        _check_product(c, x, bias=bias, name=name, r=r, out=out)
    # a residual of whole 16-byte chunks, in place, next to the same one at odd rows
    if M % 8 == 0:
        r8 = _rows(5, N, M, 8, out)
        assert torch.equal(p24.spmm24_f8(c, x, residual=r8, out=r8.clone()), p24.spmm24_f8(c, x, residual=r8, out_dtype=out))
        odd = _rows(5, N, M, 9, out)
        odd.copy_(r8)
        assert torch.equal(p24.spmm24_f8(c, x, residual=odd, bias=bias, out_dtype=out),
                           p24.spmm24_f8(c, x, residual=r8, bias=bias, out_dtype=out))
        place = r8.clone()
        assert torch.equal(p24.spmm24_f8(c, x, residual=place, bias=bias, act="gelu", out=place),
                           p24.spmm24_f8(c, x, residual=r8, bias=bias, act="gelu", out_dtype=out))


@pytest.mark.parametrize("N,M,K", [(1, 64, 128), (5, 130, 4160), (40, 200, 192), (300, 300, 832), (600, 1500, 640)])
def test_product_integers(N, M, K):
    """Small whole numbers: every sum is exact in fp32, so the result is, whatever its order."""
    need_gpu()
    rng = np.random.default_rng(N)
    W = rng.integers(-6, 7, (M, K)).astype(np.float32)
    W[:, 0] = 7                                       # the row's largest: scale 7 / 448 = 2^-6
    c = p24.compress_f8(torch.from_numpy(W).cuda())
    q = torch.from_numpy(rng.integers(-4, 5, (N, K)).astype(np.float32)).cuda().to(F8)
    x = p24.Quantized8(q, torch.full((N,), 2.0, device="cuda"))
    dense = p24.decompress_f8(c)
    assert torch.equal(dense * 64, (dense * 64).round())
    want = (2 * q.to(D)) @ dense.to(D).T
    for out in (torch.float32, torch.bfloat16):
        assert torch.equal(p24.spmm24_f8(c, x, out_dtype=out), want.to(out))


def test_product_does_not_read_past_its_rows():
    """Tokens of a wider buffer whose other columns and rows are NaN, at every kernel's size."""
    need_gpu()
    for N, M, K in ((1, 96, 64), (20, 300, 192), (70, 300, 448), (300, 520, 320), (1000, 2048, 192)):
        big = torch.full((N + 5, K + 64), 0x7F, dtype=torch.uint8, device="cuda").view(F8)     # NaN
        src = p24.gated_act(_rows(N, N, K, 0, torch.float32), act="none")
        big[:N, :K] = src.values
        c = _weight(1, M, K)
        Y = p24.spmm24_f8(c, p24.Quantized8(big[:N, :K], src.scale))
        assert torch.equal(Y, p24.spmm24_f8(c, src))


def test_product_of_a_nan_token():
    """One token with a NaN scale: its row is NaN, the others keep their bits."""
    need_gpu()
    for N, M, K in ((3, 64, 128), (90, 300, 256), (500, 1024, 256)):
        c = _weight(2, M, K)
        x = p24.gated_act(_rows(N, N, K, 0, torch.float32), act="none")
        Y0 = p24.spmm24_f8(c, x, out_dtype=torch.float32)
        raw = _rows(N, N, K, 0, torch.float32).clone()
        raw[1, 5] = float("nan")
        Y = p24.spmm24_f8(c, p24.gated_act(raw, act="none"), out_dtype=torch.float32)
        assert torch.isnan(Y[1]).all()
        keep = [i for i in range(N) if i != 1]
        assert torch.equal(Y[keep], Y0[keep])


@pytest.mark.parametrize("N,M,K", [(1, 512, 256), (40, 300, 1024), (400, 1000, 320)])
def test_product_in_place_on_the_residual(N, M, K):
    need_gpu()
    c = _weight(3, M, K)
    x = p24.gated_act(_rows(4, N, K, 0, torch.float32), act="none")
    r = _rows(5, N, M, 9, torch.bfloat16)
    want = p24.spmm24_f8(c, x, residual=r, act="silu")
    full = torch.zeros(N, M + 9, dtype=torch.bfloat16, device="cuda")
    y = full[:, :M]
    y.copy_(r)
    got = p24.spmm24_f8(c, x, residual=y, out=y, act="silu")
    assert got is y and torch.equal(y, want) and not full[:, M:].any()


@pytest.mark.parametrize("N", [0, 1, 40, 600])
def test_no_tokens_repeat_and_empty(N):
    """Zero tokens are a no-op; the same call gives the same bits."""
    need_gpu()
    c = _weight(4, 300, 640)
    x = p24.gated_act(_rows(4, N, 640, 0, torch.bfloat16), act="gelu")
    a, b = p24.spmm24_f8(c, x), p24.spmm24_f8(c, x)
    assert tuple(a.shape) == (N, 300) and torch.equal(a, b)
    y, h = p24.rms_norm(_rows(1, N, 64, 0, torch.bfloat16), torch.ones(64, device="cuda"),
                        residual=_rows(2, N, 64, 0, torch.bfloat16))
    assert tuple(y.values.shape) == (N, 64) and tuple(h.shape) == (N, 64)


def _layer(seed, tokens, width, f):
    return (_rows(seed, tokens, width, 0, torch.bfloat16), _rows(seed + 1, tokens, width, 0, torch.bfloat16),
            torch.rand(width, device="cuda") + 0.5, _weight(11, 2 * f, width), _weight(12, width, f))


@pytest.mark.parametrize("tokens", [1, 24, 300])
def test_feed_forward(tokens):
    """The four calls together are the calls one by one, and near the layer in fp64 on the dequantized weights
    (8-bit rows on the way: half an e4m3 step of each value, averaged over the sums)."""
    need_gpu()
    x, r, g, wgu, wd = _layer(20, tokens, 512, 704)
    y, h = p24.feed_forward_f8(x, r, g, wgu, wd)
    xq, h2 = p24.rms_norm(x, g, residual=r)
    gu = p24.spmm24_f8(wgu, xq)
    y2 = p24.spmm24_f8(wd, p24.gated_act(gu[:, :704], gu[:, 704:]), residual=h2)
    assert torch.equal(h, h2) and torch.equal(y, y2)
    e = x.to(D) + r.to(D)
    n = e / torch.sqrt(e.square().mean(1, keepdim=True) + 1e-6) * g.to(D)
    z = n @ p24.decompress_f8(wgu).to(D).T
    a = act(z[:, :704], "silu") * z[:, 704:]
    want = a @ p24.decompress_f8(wd).to(D).T
    off = (y.to(D) - h.to(D)) - want
    # relative to the layer's own output: two quantizations (each value within 2^-4) and bf16 between and after
    assert off.norm() <= 0.15 * want.norm() + 2.0 ** -8 * h.to(D).norm()


def test_graph_and_streams():
    """One captured layer, replayed with eager work and new inputs in between, and a layer on a side stream."""
    need_gpu()
    x, r, g, wgu, wd = _layer(30, 40, 512, 704)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p24.feed_forward_f8(x, r, g, wgu, wd)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = p24.feed_forward_f8(x, r, g, wgu, wd)
    for k in range(4):
        nx, nr = _rows(40 + k, 40, 512, 0, torch.bfloat16), _rows(50 + k, 40, 512, 0, torch.bfloat16)
        ey, eh = p24.feed_forward_f8(nx, nr, g, wgu, wd)
        x.copy_(nx)
        r.copy_(nr)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(h, eh), k
    with torch.cuda.stream(side):
        sy, _ = p24.feed_forward_f8(x, r, g, wgu, wd)
    side.synchronize()
    assert torch.equal(sy, y)


@pytest.mark.parametrize("seed", range(4))
def test_smfmac_f8_lane_map(seed):
    """One wavefront, one instruction, whole numbers: the hardware's lane map is the model's, exactly."""
    need_gpu()
    import ctypes
    import os
    p24.lib()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "hw_probe", "libp24_smfmac_f8_probe.so")
    if not os.path.exists(path):
        pytest.fail(f"{path} is missing: build it with __graft_entry__.build()")
    f = ctypes.CDLL(path).p24probe_smfmac64_f8
    f.argtypes = [ctypes.c_void_p] * 5
    rng = np.random.default_rng(seed)
    a = rng.integers(-8, 9, (64, 16)).astype(np.float64)
    b = rng.integers(-8, 9, (64, 32)).astype(np.float64)
    nib = np.array([0x4, 0x8, 0xC, 0x9, 0xD, 0xE], dtype=np.uint32)[rng.integers(0, 6, (64, 8))]
    words = np.zeros(64, dtype=np.uint32)
    for q in range(8):
        words |= nib[:, q] << np.uint32(4 * q)
    ta, tb = (torch.from_numpy(v.astype(np.float32)).cuda().to(F8) for v in (a, b))
    tw = torch.from_numpy(words.view(np.int32)).cuda()
    d = torch.zeros(64, 16, device="cuda")
    assert f(ta.data_ptr(), tb.data_ptr(), tw.data_ptr(), d.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert np.array_equal(d.cpu().numpy().astype(np.float64), smfmac64_model(a, b, words))


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: their last rows are those of a call on the last rows alone."""
    need_gpu()
    tokens, width, last = 262200, 8256, 70
    x = torch.empty(tokens, width, dtype=torch.bfloat16, device="cuda")
    x[:-last] = 0
    x[-last:] = _rows(3, last, width, 0, torch.bfloat16)
    w = torch.rand(width, device="cuda")
    y, h = p24.rms_norm(x, w, residual=x)
    y1, h1 = p24.rms_norm(x[-last:], w, residual=x[-last:])
    assert torch.equal(h[-last:], h1) and torch.equal(y.values[-last:].view(torch.uint8), y1.values.view(torch.uint8))
    assert torch.equal(y.scale[-last:], y1.scale) and not h[:8].any()
    del h, h1
    a, a1 = p24.gated_act(x, x), p24.gated_act(x[-last:], x[-last:])
    assert torch.equal(a.values[-last:].view(torch.uint8), a1.values.view(torch.uint8))
    del a, x
    # whole numbers: the sums are exact in whichever order the two calls take
    q = torch.zeros(tokens, 128, device="cuda")
    q[-last:] = torch.randint(-4, 5, (last, 128), device="cuda").float()
    q = p24.Quantized8(q.to(F8), torch.ones(tokens, device="cuda"))
    c = p24.compress_f8(torch.cat([torch.full((width, 64), 7.0, device="cuda"),
                                   torch.randint(-6, 7, (width, 64), device="cuda").float()], 1))
    Y = p24.spmm24_f8(c, q)
    Y1 = p24.spmm24_f8(c, p24.Quantized8(q.values[-last:], q.scale[-last:]))
    assert torch.equal(Y[-last:], Y1) and Y1.any() and not Y[:8].any()


def test_example(monkeypatch, capsys):
    """The example runs and is as near the fp64 layer as two 8-bit roundings allow."""
    need_gpu()
    import os
    import runpy
    import sys
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward_f8.py")
    monkeypatch.setattr(sys, "argv", [path, "--tokens", "5", "--width", "256", "--hidden", "448", "--steps", "2"])
    runpy.run_path(path, run_name="__main__")
    line = capsys.readouterr().out
    assert "5 tokens, 256 -> 448 -> 256" in line and float(line.split("error")[1]) < 0.15


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32], ids=["xbf16", "xf32"])
@pytest.mark.parametrize("width,pad", [(32768, 0), (32769, 3), (53248, 0), (65529, 8), (65536, 0), (65536, 1)])
def test_norm_adds_few_squares_in_turn(width, pad, stream):
    """One value of 1 and the rest 2^-12: their squares are half an fp32 step of 1, so a thread that holds the 1
    loses every square it adds in turn.  At most 64 squares a thread, and 22 steps after: 43 U after the root, and
    8 U beside the sum."""
    need_gpu()
    x = torch.full((2, width + pad), 2.0 ** -12, dtype=stream, device="cuda")[:, :width]
    x[:, 0] = 1
    y, _ = p24.rms_norm(x, torch.ones(width, device="cuda"), out_dtype=torch.float32)
    e = x.to(D) / torch.sqrt(x.to(D).square().mean(dim=1, keepdim=True) + 1e-6)
    assert ((y.to(D) - e).abs() / e).max() <= 51 * U


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32], ids=["xbf16", "xf32"])
@pytest.mark.parametrize("width,pad", [(16385, 0), (40001, 3), (53248, 0), (65536, 1)])
def test_wide_norm_in_place(width, pad, stream):
    """Rows that are read twice, with h in the place of x or of the residual."""
    need_gpu()
    x, r = _rows(6, 3, width, pad, stream), _rows(7, 3, width, 0, stream)
    w = torch.rand(width, device="cuda")
    for out in (F8, torch.float32):
        y0, h0 = p24.rms_norm(x, w, residual=r, out_dtype=out)
        assert torch.equal(h0, x + r)
        for alias in ("x", "r"):
            a, b = x.clone(), r.clone()
            y, h = p24.rms_norm(a, w, residual=b, h=a if alias == "x" else b, out_dtype=out)
            assert torch.equal(h, h0)
            if out == F8:
                assert torch.equal(y.values.view(torch.uint8), y0.values.view(torch.uint8))
            else:
                assert torch.equal(y, y0)


@pytest.mark.parametrize("out", [F8, torch.bfloat16, torch.float32], ids=["f8", "bf16", "f32"])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32], ids=["xbf16", "xf32"])
@pytest.mark.parametrize("width", [7, 100, 250, 700, 2049, 4097, 9000, 20001, 40001])
def test_norm_of_rows_out_of_the_squares_range(width, stream, out):
    """Rows whose squares leave fp32, up to the type's largest and down to its smallest values, with an eps under
    and over them: the norm is the formula's, and the ordinary rows beside them keep their bits."""
    need_gpu()
    powers = [-130, -100, -63, -52, -45, -40, 50, 57, 60, 64, 90, 119]
    base = _rows(61, 2 * len(powers) + 3, width, 0, torch.float32)
    base = base.clamp(-60, 60)                               # below 2^6: the largest is 2^125
    base[:len(powers)] = torch.stack([base[i] * 2.0 ** p for i, p in enumerate(powers)])
    base[len(powers):2 * len(powers), width // 3] = torch.tensor([2.0 ** p for p in powers], device="cuda")   # one value
    base[2 * len(powers), 0] = torch.finfo(stream).min
    x = base.to(stream)
    w = 1 + 0.1 * _rows(9, 1, width, 0, torch.float32)[0]
    zero, clean = torch.zeros_like(x), x.clone()
    clean[:-2] = 1                                           # the ordinary rows in the same places (order of their sums)
    for eps in (0.0, 2.0 ** -120, 1e-6):
        ordinary, _ = p24.rms_norm(clean, w, eps=eps, out_dtype=out)
        for r in (None, zero):
            y, h = p24.rms_norm(x, w, residual=r, eps=eps, out_dtype=out)
            e = x.to(D)
            e = e / torch.sqrt(e.square().mean(dim=1, keepdim=True) + eps) * w.to(D)
            _check_rows(y, e, 64 * U, out)
            assert h is None or torch.equal(h, x)
            if out == F8:
                assert torch.equal(y.values[-2:].view(torch.uint8), ordinary.values[-2:].view(torch.uint8))
                assert torch.equal(y.scale[-2:], ordinary.scale[-2:])
            else:
                assert torch.equal(y[-2:], ordinary[-2:])


@pytest.mark.parametrize("kind", ["tiny", "lowest"])
def test_norm_of_special_rows(kind):
    """What the norm makes of the rows of test_special_rows that hold numbers only."""
    need_gpu()
    x = _rows(5, 6, 700, 0, torch.float32)
    if kind == "tiny":
        x[2] = 2.0 ** -130
    else:
        x[2, 333] = torch.finfo(torch.float32).min
    y, _ = p24.rms_norm(x, torch.ones(700, device="cuda"))
    v, s = y.values.float()[2], y.scale[2].item()
    if kind == "tiny":                                       # over sqrt(eps): 2^-130 1000, under the smallest scale
        assert s == float(TINY) and (v > 0).all()
    else:
        top = 700 ** 0.5                                     # all of the mean square is one value
        assert v[333] == -448 and not v[:333].any() and abs(s * 448 / top - 1) < 64 * U


@pytest.mark.parametrize("out", [F8, torch.float32], ids=["f8", "f32"])
@pytest.mark.parametrize("width", [65, 700, 2049, 8192, 16384, 40001])
def test_norm_of_mixed_rows(width, out):
    """Large, ordinary, small and no values in one row, in runs that fall to different threads; no eps."""
    need_gpu()
    x = _rows(71, 6, width, 0, torch.float32)
    part = max(1, width // 5)
    for row, powers in enumerate(([90, -60, 0], [-60, 90, -60], [0, -45, 62], [-50, -120, -42], [0, -60, -130], [120, -45, 30])):
        for i, p in enumerate(powers):
            x[row, i * part:(i + 1) * part] *= 2.0 ** p
        x[row, 4 * part:] = 0
    x.clamp_(-3e38, 3e38)
    w = 1 + 0.1 * _rows(9, 1, width, 0, torch.float32)[0]
    y, _ = p24.rms_norm(x, w, eps=0.0, out_dtype=out)
    e = x.to(D) / torch.sqrt(x.to(D).square().mean(dim=1, keepdim=True)) * w.to(D)
    _check_rows(y, e, 64 * U, out)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tile", TILES)
def test_product_of_scales_out_of_range(monkeypatch, tile, out):
    """Scales whose product leaves fp32 while the result does not: tokens of 2^-118 against weights of 2^-10, and
    tokens of 1e30 that meet only the zeros of weights of 1e15."""
    need_gpu()
    monkeypatch.setenv("P24_F8_TILE", tile)
    M, N, K = 96, 70, 4096
    c = p24.compress_f8(torch.full((M, K), 2.0 ** -10, device="cuda"))
    Y = p24.spmm24_f8(c, p24.gated_act(torch.full((N, K), 2.0 ** -118, device="cuda"), act="none"), out_dtype=out)
    assert ((Y.to(D) * 2.0 ** 117 - 1).abs() <= 4 * U).all()       # K / 2 products of 2^-128; whole numbers until the scales
    W, x = torch.zeros(M, K, device="cuda"), torch.zeros(N, K, device="cuda")
    W[:, 0::4], W[:, 1::4], x[:, 2::4], x[:, 3::4] = 1e15, -1e15, 1e30, 2e30
    Y = p24.spmm24_f8(p24.compress_f8(W), p24.gated_act(x, act="none"), out_dtype=out)
    assert (Y == 0).all()


def test_out_of_memory_is_torchs():
    """An output that does not fit raises torch.OutOfMemoryError, as torch's own calls and the calls with `out` do."""
    need_gpu()
    tokens, width = 1 << 14, 1 << 13
    x, w, c = torch.zeros(tokens, width, dtype=torch.bfloat16, device="cuda"), torch.ones(width, device="cuda"), _weight(1, width, 64)
    q = p24.gated_act(x[:, :64], act="none")
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (32 << 20)) / total)
    try:
        for call in (lambda: p24.rms_norm(x, w, out_dtype=torch.float32), lambda: p24.gated_act(x, out_dtype=torch.float32),
                     lambda: p24.gated_act(x), lambda: p24.spmm24_f8(c, q)):
            with pytest.raises(torch.OutOfMemoryError):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert not p24.gated_act(x).values.view(torch.uint8).any()


def test_arguments_that_are_no_numbers():
    """A weight whose sizes are no whole numbers is refused by the binding's checks."""
    need_gpu()
    import ctypes
    c = _weight(1, 32, 64)
    x = p24.gated_act(_rows(1, 4, 64, 0, torch.float32), act="none")
    for M, K in ((32.0, 64), (32, "64"), (None, 64)):
        with pytest.raises((TypeError, ValueError, ctypes.ArgumentError)):
            p24.spmm24_f8(p24.Compressed24F8(c.data, c.scale, M, K), x)


def test_a_token_of_rows_at_any_stride():
    """One token cut from a buffer whose rows are not 16 bytes apart."""
    need_gpu()
    for M, K in ((96, 64), (4096, 1024), (300, 192)):
        c = _weight(1, M, K)
        x = p24.gated_act(_rows(3, 1, K, 0, torch.float32), act="none")
        for pad in (1, 8, 24):
            buf = torch.zeros(3, K + pad, dtype=torch.uint8, device="cuda").view(F8)
            row = buf[:1, :K]
            row.copy_(x.values)
            assert row.stride(0) % 16
            want = p24.spmm24_f8(c, x)
            assert torch.equal(p24.spmm24_f8(c, p24.Quantized8(row, x.scale)), want)
            assert torch.equal(p24.spmm24_f8(c, p24.Quantized8(row, x.scale), out=torch.empty_like(want)), want)


@pytest.mark.parametrize("N,M,K", [(33, 65, 128), (70, 300, 192), (257, 260, 1024), (100, 136, 1088), (300, 513, 4160)])
@pytest.mark.parametrize("tile", TILES)
def test_integers_in_every_kernel(monkeypatch, tile, N, M, K):
    """Small whole numbers through each kernel, both outputs: exact, whatever the order of the sums."""
    need_gpu()
    monkeypatch.setenv("P24_F8_TILE", tile)
    rng = np.random.default_rng(N + K)
    W = rng.integers(-6, 7, (M, K)).astype(np.float32)
    W[:, 0] = 7                                       # the row's largest: scale 7 / 448 = 2^-6
    c = p24.compress_f8(torch.from_numpy(W).cuda())
    q = torch.from_numpy(rng.integers(-4, 5, (N, K)).astype(np.float32)).cuda().to(F8)
    x = p24.Quantized8(q, torch.full((N,), 2.0, device="cuda"))
    want = (2 * q.to(D)) @ p24.decompress_f8(c).to(D).T
    r = torch.from_numpy(rng.integers(-64, 65, (N, M)).astype(np.float32)).cuda()
    for out in (torch.float32, torch.bfloat16):
        assert torch.equal(p24.spmm24_f8(c, x, out_dtype=out), want.to(out))
        assert torch.equal(p24.spmm24_f8(c, x, out_dtype=out, residual=r.to(out)), (want + r.to(D)).to(out))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,M,K", [(960, 1152, 2112), (957, 1145, 2112), (8640, 256, 2112), (8630, 248, 2112)])
def test_one_group_of_waves_with_a_long_k(N, M, K, out):
    """More than 256 tiles of 64 x 64 and of 128 x 64, where one group of waves walks a long K alone and the
    residual takes over its stages."""
    need_gpu()
    c = _weight(M + K, M, K)
    x = p24.gated_act(_rows(N, N, K, 0, torch.float32), act="none")
    r, odd = _rows(5, N, M, 8, out), _rows(5, N, M, 9, out)
    odd.copy_(r)
    _check_product(c, x, out=out)
    Y = _check_product(c, x, r=r, name="silu", out=out)
    assert torch.equal(Y, p24.spmm24_f8(c, x, residual=odd, act="silu", out_dtype=out))


@pytest.mark.parametrize("N,M,K", [(6144, 2048, 128), (6100, 2040, 192)])
def test_a_full_round_of_blocks(N, M, K):
    """256 blocks of 256 x 192, the library's own choice of kernel."""
    need_gpu()
    c = _weight(M + K, M, K)
    x = p24.gated_act(_rows(N, N, K, 0, torch.float32), act="none")
    _check_product(c, x, r=_rows(5, N, M, 8, torch.bfloat16), name="silu")


def test_compress_of_rows_without_values():
    """K = 0: the scales of empty rows are the smallest, not memory as it was."""
    need_gpu()
    torch.full((5,), 7.0, device="cuda")              # what a fresh allocation would show
    for dtype in (torch.float32, torch.bfloat16):
        c = p24.compress_f8(torch.empty(5, 0, dtype=dtype, device="cuda"))
        assert torch.equal(c.scale, torch.full((5,), float(TINY), device="cuda"))
        assert c.data.numel() == 0 and tuple(p24.decompress_f8(c).shape) == (5, 0)
