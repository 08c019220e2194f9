"""GPU parity of the expert operators: routing against a brute force on the CPU, the grouped 2:4 products
and the combination against fp64 formulas, and a layer of them together.

Tolerances count roundings (U = 2^-24 is half an fp32 step, relative).
Routing: experts, offsets, tokens and positions are whole numbers and exact.  A weight: a logit's difference
from the largest is rounded once (at most |l - max| U of exp's argument), exp and the quotient's steps take
8 U, a sum of E terms E U.
Grouped product: as for the product it is made of (test_gpu_f8).
Combination: k products summed in fp32 and the residual: (k + 2) U of the sum of magnitudes."""
import gc
import math

import numpy as np
import pytest

from f8_ref import HALF, U, act, act_error
from gpu_util import need_gpu, torch

p24 = pytest.importorskip("structured_sparse_gemm_prune24_amd")
pytestmark = pytest.mark.gpu
D = torch.float64


@pytest.fixture
def large_blocks():
    """Blocks that a test leaves in the allocator's cache go back, before anything that lives on takes a part of one."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(seed, *shape):
    return torch.randn(*shape, generator=_gen(seed), device="cuda")


# ---- routing ----------------------------------------------------------------
def _route_ref(logits, k, score, bias, normalize, scale):
    """By Python's own comparisons: (experts, weights, offsets, tokens, positions)."""
    l = logits.double().cpu().numpy()
    T, E = l.shape
    with np.errstate(all="ignore"):
        sig = 1 / (1 + np.exp(-l))
    rank = sig + bias.double().cpu().numpy() if bias is not None else l
    experts, weights = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T):
        is_open = [e for e in range(E) if l[t, e] != -math.inf]
        nan_first = sorted(is_open, key=lambda e: (0 if math.isnan(rank[t, e]) else 1,
                                                   0 if math.isnan(rank[t, e]) else -rank[t, e], e))
        best = nan_first[:k]
        experts[t, :len(best)] = best
        if not best:
            continue
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                w = sig[t, best]
                total = w.sum() if normalize else 1.0
            else:
                top = l[t, is_open].max()          # NaN if any is
                w = np.exp(l[t, best] - top)
                total = w.sum() if normalize else np.exp(l[t, is_open] - top).sum()
            weights[t, :len(best)] = w / total * scale
    flat = experts.reshape(-1)
    rows = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if e >= 0:
            rows[e].append(i)
    offsets = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
    order = [i for r in rows for i in r]
    tokens, positions = np.full(T * k, -1), np.full(T * k, -1)
    for p, i in enumerate(order):
        tokens[p], positions[i] = i // k, p
    return experts, weights, offsets, tokens, positions.reshape(T, k)


def _check_route(logits, k, score="softmax", bias=None, normalize=True, scale=1.0):
    r = p24.route(logits, k, score=score, bias=bias, normalize=normalize, scale=scale)
    want = _route_ref(logits, k, score, bias, normalize, scale)
    for name, w in zip(("experts", None, "offsets", "tokens", "positions"), want):
        if name:
            got = getattr(r, name)
            assert got.dtype == torch.int32
            assert np.array_equal(got.cpu().numpy(), w), name
    assert r.weights.dtype == torch.float32
    got, w = r.weights.double().cpu().numpy(), want[1]
    finite = np.where(np.isfinite(logits.double().cpu().numpy()), logits.double().cpu().numpy(), 0.0)
    spread = 2 * np.abs(finite).max() if finite.size else 0.0
    tol = (2 * spread + 24 + logits.shape[1]) * U
    assert np.array_equal(np.isnan(got), np.isnan(w))
    ok = np.isnan(w) | (np.abs(got - w) <= tol * np.abs(w) + 1e-37)
    assert ok.all(), np.abs(got - w)[~ok].max()
    return r


ROUTES = [(1, 1, 1), (1, 128, 8), (3, 5, 5), (7, 64, 6), (40, 60, 4), (63, 8, 8), (64, 257, 3), (64, 1024, 32), (8195, 5, 2), (9000, 130, 3), (65, 512, 16), (33, 1000, 32),
          (200, 256, 8), (513, 16, 2), (1000, 31, 7), (2050, 128, 1), (300, 1024, 17)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", ROUTES)
def test_route(T, E, k, dtype):
    need_gpu()
    full = (2 * _randn(T + E, T, E + 3)).to(dtype)
    logits = full[:, :E]                       # rows at any alignment
    _check_route(logits, k)
    _check_route(logits, k, normalize=False, scale=2.5)
    _check_route(logits, k, score="sigmoid")
    bias = 0.3 * _randn(5, E)
    _check_route(logits, k, score="sigmoid", bias=bias, normalize=False)
    _check_route(logits, k, score="sigmoid", bias=bias, scale=0.5)


@pytest.mark.parametrize("T", [9, 300])
def test_route_of_ties_and_closed_experts(T):
    """Equal logits (both zeros among them) go to the lower expert; -inf closes experts, single ones, all but fewer
    than k, and whole tokens."""
    need_gpu()
    l = torch.round(_randn(3, T, 70))
    l[l == 0] = torch.where(torch.rand(int((l == 0).sum()), generator=_gen(1), device="cuda") < 0.5, -0.0, 0.0)
    l[torch.rand(T, 70, generator=_gen(2), device="cuda") < 0.2] = -math.inf
    l[1] = -math.inf
    l[-1] = -math.inf
    l[2, 3:] = -math.inf
    l[4] = 1.0
    l[5] = -math.inf
    l[5, 69] = -3e38
    for score in ("softmax", "sigmoid"):
        r = _check_route(l, 6, score=score)
        assert (r.experts[1] == -1).all() and (r.weights[1] == 0).all() and (r.positions[1] == -1).all()
        assert r.experts[4].tolist() == list(range(6)) and r.experts[5].tolist() == [69] + [-1] * 5
    _check_route(l, 6, score="sigmoid", bias=torch.zeros(70, device="cuda"))
    _check_route(torch.full((T, 70), -math.inf, device="cuda"), 6)


@pytest.mark.parametrize("T", [9, 300])
def test_route_of_nan_and_infinity(T):
    """NaN ranks above +inf; the weights are the formula's NaN, in that token alone."""
    need_gpu()
    l = _randn(4, T, 40)
    l[2, 17] = math.nan
    l[3, 5] = math.inf
    l[3, 9] = math.nan
    l[4, 30] = math.inf
    for score in ("softmax", "sigmoid"):
        r = _check_route(l, 4, score=score)
        assert r.experts[2, 0] == 17 and r.experts[3, :2].tolist() == [9, 5] and r.experts[4, 0] == 30
        assert torch.isfinite(r.weights[5:]).all()
    bias = torch.zeros(40, device="cuda")
    bias[7] = math.inf
    bias[8] = -math.inf
    _check_route(l, 4, score="sigmoid", bias=bias)


def test_route_of_many_choices():
    """More choices than the sorting blocks keep in registers."""
    need_gpu()
    _check_route(_randn(6, 3000, 24), 20)


def test_route_of_one_expert_for_all():
    need_gpu()
    l = _randn(6, 700, 12)
    l[:, 7] = 20.0
    r = _check_route(l, 1)
    assert r.offsets.tolist() == [0] * 8 + [700] * 5
    assert torch.equal(r.tokens, torch.arange(700, device="cuda", dtype=torch.int32))


@pytest.mark.parametrize("T,E,k", [(16384, 256, 8), (16385, 256, 1), (32768, 64, 2), (32800, 62, 2), (65504, 3, 1), (65505, 3, 1), (8192, 1021, 4),
                                   (70000, 5, 5)])
def test_route_of_many_tokens(T, E, k):
    """On both sides of where the counts are summed by a launch of their own; every token on one expert as well, the most a sum holds."""
    need_gpu()
    l = _randn(T + E, T, E)
    for logits in (l, torch.arange(E, 0, -1, device="cuda", dtype=torch.float32).repeat(T, 1)):
        r = p24.route(logits, k)
        chosen = r.experts.long()
        want = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(chosen, want)
        order = torch.sort(chosen.flatten(), stable=True).indices
        assert torch.equal(r.tokens.long(), order // k)
        at = torch.empty_like(order)
        at[order] = torch.arange(T * k, device="cuda")
        assert torch.equal(r.positions.long().flatten(), at)
        count = torch.bincount(chosen.flatten(), minlength=E)
        assert torch.equal(r.offsets.long(), torch.cat([count.new_zeros(1), count.cumsum(0)]))


def test_route_without_tokens():
    need_gpu()
    r = p24.route(torch.empty(0, 9, device="cuda"), 3)
    assert r.offsets.tolist() == [0] * 10 and r.tokens.numel() == 0 and r.experts.shape == (0, 3)


# ---- grouped products -------------------------------------------------------
def _weights(seed, E, M, K):
    return p24.compress_f8_experts(0.02 * _randn(seed + e, M, K) for e in range(E))


def _dense(c, e):
    n = p24.lib().prune24_f8_bytes(c.M, c.K)
    return p24.decompress_f8(p24.Compressed24F8(c.data[e * n:(e + 1) * n], c.scale[e], c.M, c.K)).to(D)


def _x(seed, n, K):
    return p24.gated_act(_randn(seed, n, K), act="none")


def _offsets(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def _check_grouped(c, x, counts, tokens=None, bias=None, name="none", out=torch.bfloat16, Y=None):
    off = _offsets(counts)
    Y = p24.spmm24_f8_grouped(c, x, off, tokens=tokens, out_dtype=out, bias=bias, act=name) if Y is None else Y
    X = x.values.to(D) * x.scale.to(D)[:, None]
    at = 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        W = _dense(c, e)
        src = torch.arange(at, at + n, device="cuda") if tokens is None else tokens[at:at + n].long()
        z = X[src] @ W.T
        err = ((c.K + 16) * U + (7 * 2.0 ** -13 if out == torch.bfloat16 else 0)) * (X[src].abs() @ W.abs().T)
        if bias is not None:
            z = z + bias[e].to(D)
            err = err + 2 * U * z.abs()
        want = act(z, name)
        err = 1.13 * err + act_error(z, name, out) * want.abs()
        tol = err + HALF[out] * (want.abs() + err) + 1e-36
        off_by = (Y[at:at + n].to(D) - want).abs()
        assert torch.all(off_by <= tol), (e, float((off_by / tol).max()))
        at += n
    return Y


TILES = ["tokens", "64x32", "64x64", "128x64", "128x128", "256x128", "256x192", "256x256"]
# experts' rows: none, one, a tile's edge, more than the widest tile; more experts than a wave has lanes
COUNTS = [[1], [0, 1, 0], [5, 0, 33, 64, 1], [300, 1, 0, 257], [0, 0, 0, 31], [2] * 70 + [0] * 60 + [3] * 5,
          [0] * 130 + [40, 7]]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tile", [None] + TILES)
def test_grouped(monkeypatch, tile, out):
    """Every kernel, gathered and not; rows outside the experts' ranges stay untouched."""
    need_gpu()
    if tile:
        monkeypatch.setenv("P24_F8_TILE", tile)
    for counts, (M, K) in zip(COUNTS, [(1, 64), (65, 192), (300, 448), (257, 1088), (40, 4160), (33, 128), (129, 320)]):
        c = _weights(M + K, len(counts), M, K)
        n, behind = sum(counts), 3
        x = _x(n, n + behind, K)
        full = torch.full((n + behind + 2, M + 5), 7.0, dtype=out, device="cuda")
        y = full[1:n + behind + 1, :M]
        p24.spmm24_f8_grouped(c, x, _offsets(counts), out=y)
        _check_grouped(c, x, counts, out=out, Y=y)
        assert (full[0] == 7).all() and (full[n + 1:] == 7).all() and (full[:, M:] == 7).all()
        few = _x(n + 1, max(1, n // 3), K)
        tokens = torch.randint(0, few.values.shape[0], (n + behind,), generator=_gen(9), device="cuda", dtype=torch.int32)
        tokens[n:] = -1
        bias = _randn(7, len(counts), M)
        for name in ("none", "gelu", "silu", "relu"):
            _check_grouped(c, few, counts, tokens=tokens, bias=bias, name=name, out=out)


@pytest.mark.parametrize("tile", [None] + TILES)
def test_grouped_is_each_experts_product(monkeypatch, tile):
    """Bit for bit the product of the expert's rows by the same kernel family, for whole numbers; and repeated calls agree."""
    need_gpu()
    if tile:
        monkeypatch.setenv("P24_F8_TILE", tile)
    counts, M, K = [70, 0, 3, 260, 129], 200, 512
    g = _gen(11)
    W = torch.randint(-4, 5, (5, M, K), generator=g, device="cuda").float()
    c = p24.compress_f8_experts(W)
    n = sum(counts)
    q = torch.randint(-4, 5, (n, K), generator=g, device="cuda").float()
    x = p24.Quantized8(q.to(torch.float8_e4m3fn), torch.ones(n, device="cuda"))
    y = p24.spmm24_f8_grouped(c, x, _offsets(counts), out_dtype=torch.float32)
    assert torch.equal(y, p24.spmm24_f8_grouped(c, x, _offsets(counts), out_dtype=torch.float32))
    at = 0
    for e, m in enumerate(counts):
        if m:
            want = q[at:at + m].to(D) @ _dense(c, e).T
            assert torch.all((y[at:at + m].to(D) - want).abs() <= 4 * U * want.abs() + K * U * 16), e
        at += m


@pytest.mark.parametrize("K", [448, 576, 640, 832])
@pytest.mark.parametrize("tile", [None, "128x128", "256x128", "256x192", "256x256"])
def test_grouped_over_several_tiles_a_block(monkeypatch, large_blocks, tile, K):
    """More tiles than the chip holds at once, of every fill, so that blocks go from one to the next; 4 to 7 steps of K,
    the last one half where K is odd in 64s."""
    need_gpu()
    if tile:
        monkeypatch.setenv("P24_F8_TILE", tile)
    E, M = 90, 1100
    counts = torch.randint(0, 601, (E,), generator=torch.Generator().manual_seed(K)).tolist()
    counts[3] = counts[64] = 0
    counts[10], counts[65], counts[89] = 1, 256, 257
    n = sum(counts)
    c = _weights(K, E, M, K)
    x = _x(K + 1, n, K)
    _check_grouped(c, x, counts)
    bias = _randn(5, E, M)
    few = _x(K + 2, 1001, K)
    tokens = torch.randint(0, 1001, (n,), generator=_gen(K), device="cuda", dtype=torch.int32)
    _check_grouped(c, few, counts, tokens=tokens, bias=bias, name="silu")
    y = p24.spmm24_f8_grouped(c, x, _offsets(counts))
    for _ in range(3):
        assert torch.equal(y, p24.spmm24_f8_grouped(c, x, _offsets(counts)))


def test_grouped_offsets_and_tokens_outside():
    """Offsets past the rows and tokens outside X reach nothing outside: what they do reach is defined."""
    need_gpu()
    c = _weights(1, 3, 70, 128)
    x = _x(2, 50, 128)
    full = torch.full((54, 70), 7.0, dtype=torch.bfloat16, device="cuda")
    p24.spmm24_f8_grouped(c, x, torch.tensor([-5, 20, 20, 1 << 30], dtype=torch.int32, device="cuda"), out=full[2:52])
    _check_grouped(c, x, [20, 0, 30], Y=full[2:52])
    assert (full[:2] == 7).all() and (full[52:] == 7).all()
    tokens = torch.arange(50, device="cuda", dtype=torch.int32)
    tokens[3], tokens[30] = 1 << 29, -7
    y = p24.spmm24_f8_grouped(c, x, _offsets([20, 0, 30]), tokens=tokens)
    tokens[3] = tokens[30] = 49
    _check_grouped(c, x, [20, 0, 30], tokens=tokens, Y=y)


@pytest.mark.parametrize("tile", [None] + TILES)
def test_grouped_of_a_nan_row(monkeypatch, tile):
    need_gpu()
    if tile:
        monkeypatch.setenv("P24_F8_TILE", tile)
    c = _weights(3, 2, 96, 192)
    x = _x(4, 90, 192)
    clean = p24.spmm24_f8_grouped(c, x, _offsets([50, 40]))
    x.values.view(torch.uint8)[60, 100] = 0x7F
    y = p24.spmm24_f8_grouped(c, x, _offsets([50, 40]))
    keep = [i for i in range(90) if i != 60]
    assert torch.isnan(y[60]).any() and torch.equal(y[keep], clean[keep])


def test_grouped_without_rows():
    need_gpu()
    c = _weights(1, 2, 70, 128)
    x = p24.Quantized8(torch.empty(0, 128, device="cuda").to(torch.float8_e4m3fn), torch.empty(0, device="cuda"))
    assert p24.spmm24_f8_grouped(c, x, _offsets([0, 0])).shape == (0, 70)


# ---- combination ------------------------------------------------------------
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("zt", [torch.bfloat16, torch.float32], ids=["zbf16", "zf32"])
@pytest.mark.parametrize("T,k,width,pad", [(1, 1, 1, 0), (1, 8, 4096, 0), (3, 5, 7, 2), (9, 4, 512, 1), (5, 2, 513, 3), (70, 8, 2049, 0),
                                           (6, 32, 8200, 5), (2, 3, 65536, 0), (4001, 2, 64, 0)])
def test_combine(T, k, width, pad, zt, out):
    need_gpu()
    rows = T * k + 3
    z = _randn(1, rows, width + pad).to(zt)[:, :width]
    pos = torch.randint(0, rows, (T, k), generator=_gen(2), device="cuda", dtype=torch.int32)
    w = torch.rand(T, k, generator=_gen(3), device="cuda")
    pos[0, -1] = -1
    pos[-1, 0] = rows
    w[0, -1] = math.nan           # of a slot without a row
    on = (pos >= 0) & (pos < rows)
    wz = torch.where(on, w, 0).to(D)[:, :, None] * z.to(D)[torch.where(on, pos, 0).long()]
    for r in (None, _randn(4, T, width + pad + 1).to(out)[:, :width]):
        want, size = wz.sum(1), wz.abs().sum(1)
        if r is not None:
            want, size = want + r.to(D), size + r.to(D).abs()
        err = (k + 2) * U * size
        y = p24.combine_experts(z, pos, w, residual=r, out_dtype=out)
        assert y.dtype == out
        assert torch.all((y.to(D) - want).abs() <= err + HALF[out] * (want.abs() + err) + 1e-36)
    place = r.clone() if pad else r
    assert torch.equal(p24.combine_experts(z, pos, w, residual=place, out=place), y)


# ---- together ---------------------------------------------------------------
def _layer(seed, tokens, width, f, E):
    wgu = _weights(seed, E, 2 * f, width)
    wd = _weights(seed + 100, E, width, f)
    h = _randn(seed + 1, tokens, width).bfloat16()
    xq, _ = p24.rms_norm(h, torch.ones(width, device="cuda"))
    return xq, h, _randn(seed + 2, tokens, E), wgu, wd


@pytest.mark.parametrize("tokens", [1, 5, 70, 600])
def test_layer(tokens):
    """Against the operators' own formulas in fp64, from the 8-bit rows in; padded tokens keep their residual.

    The second product's rows are 8-bit values of the first's: an element is within half an e4m3 step (2^-4) of
    itself or half the smallest step of its row's scale, and what bf16 lost before it."""
    need_gpu()
    width, f, E, k = 256, 192, 12, 3
    xq, h, l, wgu, wd = _layer(20, tokens, width, f, E)
    if tokens > 4:
        l[tokens - 2:] = -math.inf
    y = p24.feed_forward_f8_experts(xq, l, k, wgu, wd, residual=h)
    r = p24.route(l, k)
    X = xq.values.to(D) * xq.scale.to(D)[:, None]
    want = h.to(D).clone()
    tol = torch.zeros_like(want)
    for t in range(tokens):
        for j in range(k):
            e = int(r.experts[t, j])
            if e < 0:
                continue
            Wg, Wd = _dense(wgu, e), _dense(wd, e)
            g = Wg @ X[t]
            g_err = (7 * 2.0 ** -13 + (width + 16) * U) * (Wg.abs() @ X[t].abs())
            g_err = g_err + 2.0 ** -8 * (g.abs() + g_err)
            gate, up, ge, ue = g[:f], g[f:], g_err[:f], g_err[f:]
            a = act(gate, "silu") * up
            ae = 1.13 * ge * (up.abs() + ue) + act(gate, "silu").abs() * ue + 1e-5 * a.abs()
            ae = ae + 2.0 ** -4 * (a.abs() + ae) + 2.0 ** -10 / 448 * 1.01 * (a.abs() + ae).max()
            z = Wd @ a
            ze = Wd.abs() @ ae + (7 * 2.0 ** -13 + (f + 16) * U) * (Wd.abs() @ (a.abs() + ae))
            ze = ze + 2.0 ** -8 * (z.abs() + ze)
            w = float(r.weights[t, j])
            want[t] += w * z
            tol[t] += w * ze + 8 * U * w * z.abs()
    tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert torch.all((y.to(D) - want).abs() <= tol)
    if tokens > 4:
        assert torch.equal(y[tokens - 2:], h[tokens - 2:])


def test_graph_and_streams():
    """One captured layer, replayed with eager work, other logits and other rows in between; and one on a side stream."""
    need_gpu()
    xq, h, l, wgu, wd = _layer(30, 40, 256, 192, 12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p24.feed_forward_f8_experts(xq, l, 3, wgu, wd, residual=h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = p24.feed_forward_f8_experts(xq, l, 3, wgu, wd, residual=h)
    for i in range(4):
        nl, nh = _randn(50 + i, 40, 12), _randn(60 + i, 40, 256).bfloat16()
        if i == 2:
            nl[:, 1:] = -math.inf       # all tokens to one expert
        nx, _ = p24.rms_norm(nh, torch.ones(256, device="cuda"))
        want = p24.feed_forward_f8_experts(nx, nl, 3, wgu, wd, residual=nh)
        l.copy_(nl)
        h.copy_(nh)
        xq.values.view(torch.uint8).copy_(nx.values.view(torch.uint8))
        xq.scale.copy_(nx.scale)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
    with torch.cuda.stream(side):
        sy = p24.feed_forward_f8_experts(xq, l, 3, wgu, wd, residual=h)
    side.synchronize()
    assert torch.equal(sy, y)


@pytest.mark.parametrize("T", [20, 400])
def test_route_of_scores_that_32_bits_cannot_tell_apart(T):
    """Sigmoid and bias: experts whose scores differ by less than an fp32 step, at the edge of the chosen and among
    them, and far too many of them; saturated sigmoids tie in 64 bits too and go to the lower expert."""
    need_gpu()
    bias = torch.zeros(64, device="cuda")
    l = _randn(5, T, 64)
    step = torch.arange(64, device="cuda") * 1e-7
    l[0] = 3.0 + step                       # all of them near
    l[1] = 3.0 - step
    l[2, 10:14] = 4.0 + step[:4]            # a few among the chosen
    l[3, 40:42] = torch.tensor([4.0, 4.0000005], device="cuda")
    l[4] = 50.0                             # sigmoid 1 in 64 bits: ties
    l[5, ::2] = 40.0 + step[::2]
    order = torch.sort(l[6], descending=True).indices
    l[6, order[5]] = l[6, order[4]] - 1e-6  # across the edge of k = 5
    l[7, order[6]] = l[7].max() + 1         # and one that is just behind it
    for k in (5, 6, 15, 16, 20):
        _check_route(l, k, score="sigmoid", bias=bias)
        _check_route(l, k, score="sigmoid", bias=bias - 1000.0)     # the bias swallows the sigmoid's last bits in 32


def test_offsets_past_32_bits(large_blocks):
    """Outputs and combined rows of more than 2^31 elements: the last rows are those of a small call."""
    need_gpu()
    M, n = 32768, 70000
    c = _weights(5, 2, M, 64)
    x = _x(6, n, 64)
    y = p24.spmm24_f8_grouped(c, x, _offsets([30000, 40000]))
    small = p24.Quantized8(x.values[-5:], x.scale[-5:].contiguous())
    want = p24.spmm24_f8_grouped(c, small, _offsets([0, 5]))
    assert (y[-5:].float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()     # another kernel's sums
    assert want.any()
    pos = torch.arange(n - 1, n - 7, -1, dtype=torch.int32, device="cuda").reshape(3, 2)
    w = torch.rand(3, 2, generator=_gen(1), device="cuda")
    assert torch.equal(p24.combine_experts(y, pos, w), p24.combine_experts(y[-6:], pos - (n - 6), w))


def test_two_streams_at_once():
    """Two layers on two streams: no state between calls."""
    need_gpu()
    a, b = _layer(40, 300, 256, 192, 12), _layer(60, 200, 256, 192, 8)
    want = [p24.feed_forward_f8_experts(xq, l, 3, wgu, wd, residual=h) for xq, h, l, wgu, wd in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, (xq, h, l, wgu, wd) in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(p24.feed_forward_f8_experts(xq, l, 3, wgu, wd, residual=h))
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_example(monkeypatch, capsys):
    """The example runs and is near the fp64 layer: its output is rounded to bf16 twice (2^-8 of a value each at most),
    and what the layer adds to the residual, under a fiftieth of it at these weights (0.02 times the square root of
    256 and 192 inputs: values of 0.3 times 0.16, then 0.02), is 0.15 off at most by two 8-bit operands."""
    need_gpu()
    import os
    import runpy
    import sys
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "experts_f8.py")
    monkeypatch.setattr(sys, "argv", [path, "--tokens", "5", "--width", "256", "--hidden", "192", "--experts", "8", "--k", "2",
                                      "--steps", "2"])
    runpy.run_path(path, run_name="__main__")
    line = capsys.readouterr().out
    assert "5 tokens, 2 of 8 experts 256 -> 192 -> 256" in line
    assert float(line.split("error")[1]) <= 2 * 2.0 ** -8 + 0.15 / 50
