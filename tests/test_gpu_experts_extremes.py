"""GPU tests of the expert operators where their arguments leave the ordinary: sigmoids that leave fp32, offsets
that fall, the most rows; and the grouped product's every kernel on whole numbers.

U = 2^-24 is half an fp32 step, relative."""
import gc

import pytest

from f8_ref import U
from gpu_util import need_gpu, torch

p24 = pytest.importorskip("structured_sparse_gemm_prune24_amd")
pytestmark = pytest.mark.gpu
D = torch.float64


def _randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


@pytest.mark.parametrize("with_bias", [False, True], ids=["logits", "bias"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(7, 24, 5), (7, 24, 20), (150, 24, 5), (150, 600, 17)])
def test_sigmoids_that_leave_fp32_have_finite_quotients(T, E, k, dtype, with_bias):
    """Normalised weights of tokens whose logits all lie far below zero, against log-sigmoids in 64 bits.

    A weight is exp(l - max) / (1 + exp(l)) over their sum: the difference is rounded once (|l - max| U in exp's
    argument), each exp, the sums of at most k terms and the quotients take (24 + k) U; below 1e-37 fp32 has no
    normal numbers."""
    need_gpu()
    l = _randn(T + E, T, E)
    l[0] = l[0] - 95                                  # every sigmoid is 0 in fp32
    l[1] = 8 * l[1] - 80                              # some are
    l[2] = l[2] - 600
    l[3] = -88.0 - torch.arange(E, device="cuda") / 16
    l[4, 1:] = -3 - torch.arange(E - 1, device="cuda") / 2        # one ordinary logit or none above -3
    l[4, 0] = -5
    l[5] = l[5] - 3                                   # small, none lost
    l = l.to(dtype)
    bias = 0.3 * _randn(9, E) if with_bias else None
    r = p24.route(l, k, score="sigmoid", bias=bias, scale=2.0)
    x = l.to(D).gather(1, r.experts.long())
    low = x.clamp_max(0) - torch.log1p(torch.exp(-x.abs()))       # log sigmoid
    w = torch.exp(low - low.amax(1, keepdim=True))
    w = 2 * w / w.sum(1, keepdim=True)
    assert torch.isfinite(r.weights).all()
    spread = x.amax(1, keepdim=True) - x + 1
    off = (r.weights.to(D) - w).abs()
    assert torch.all(off <= (spread + 24 + k) * U * w + 1e-37), float((off / w).max())
    # a router's other tokens keep their bits
    ordinary = p24.route(l[6:].contiguous(), k, score="sigmoid", bias=bias, scale=2.0)
    assert torch.equal(r.weights[6:], ordinary.weights) and torch.equal(r.experts[6:], ordinary.experts)
    # unnormalised ones are the sigmoids, 0 where fp32 has none
    n = p24.route(l, k, score="sigmoid", bias=bias, normalize=False)
    y = torch.sigmoid(l.to(D).gather(1, n.experts.long()))
    assert torch.all((n.weights.to(D) - y).abs() <= (x.abs() + 24) * U * y + 1e-37)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tile", [None, "tokens", "64x32", "64x64", "128x64", "128x128", "256x128", "256x192", "256x256"])
def test_falling_offsets_write_nothing_outside(monkeypatch, tile, out):
    """Offsets that fall (no routing makes them) have no rows; the kernel for few rows may write some, none outside `out`.
    The same call with sums of counts, afterwards, is right."""
    need_gpu()
    if tile:
        monkeypatch.setenv("P24_F8_TILE", tile)
    E, rows, M, K = 70, 300, 300, 192
    one = p24.compress_f8(0.02 * _randn(1, M, K))
    c = p24.Experts24F8(one.data.repeat(E), one.scale.repeat(E, 1), E, M, K)
    x = p24.gated_act(_randn(2, rows, K), act="none")
    full = torch.full((rows + 8, M), 7.0, dtype=out, device="cuda")
    for offsets in ([0, 300] * 35 + [0], [300] * 35 + [0] * 36, [0] * 68 + [300, 0, 300], [(1 << 31) - 1, -(1 << 31)] * 35 + [0]):
        p24.spmm24_f8_grouped(c, x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=full[4:-4])
        torch.cuda.synchronize()
        assert (full[:4] == 7).all() and (full[-4:] == 7).all()
        if tile not in (None, "tokens"):
            assert (full == 7).all()
    good = torch.tensor([0] * 30 + [200] * 30 + [300] * 11, dtype=torch.int32, device="cuda")
    y = p24.spmm24_f8_grouped(c, x, good, out_dtype=out)
    X, W = x.values.to(D) * x.scale.to(D)[:, None], p24.decompress_f8(one).to(D)
    size = X.abs() @ W.abs().T
    # as in test_gpu_experts: K + 16 roundings of the sum, the 8-bit unit's cut, and the output's own
    err = ((K + 16) * U + (7 * 2.0 ** -13 if out == torch.bfloat16 else 0)) * size
    want = X @ W.T
    assert torch.all((y.to(D) - want).abs() <= err + (2.0 ** -8 if out == torch.bfloat16 else U) * (want.abs() + err) + 1e-36)


@pytest.fixture
def large_blocks():
    """Blocks that a test leaves in the allocator's cache go back."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tile", [None, "tokens"])
@pytest.mark.parametrize("E", [2, 1024])
def test_grouped_of_the_most_rows(monkeypatch, large_blocks, E, tile):
    """65535 * 32 rows through narrow weights, more tiles than the kernel for few rows has blocks.

    Whole numbers and scales of powers of two: exact."""
    need_gpu()
    if tile:
        monkeypatch.setenv("P24_F8_TILE", tile)
    rows, M, K = 65535 * 32, 32, 64
    W = torch.zeros(E, M, K, device="cuda")
    W[:, :, ::2] = torch.randint(-4, 5, (E, M, K // 2), device="cuda").float()
    W[:, :, 0] = 448                      # the rows' scale is 1
    c = p24.compress_f8_experts(W)
    assert (c.scale == 1).all()
    q = torch.randint(-2, 3, (rows, K), device="cuda").float()
    x = p24.Quantized8(q.to(torch.float8_e4m3fn), torch.ones(rows, device="cuda"))
    ends = torch.sort(torch.randint(0, rows + 1, (E - 1,))).values.tolist()
    y = p24.spmm24_f8_grouped(c, x, torch.tensor([0] + ends + [rows], dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    for e, (a, b) in enumerate(zip([0] + ends, ends + [rows])):
        if b > a:
            assert torch.equal(y[a:b], q[a:b] @ W[e].T), e


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tile", [None, "tokens", "64x32", "64x64", "128x64", "128x128", "256x128", "256x192", "256x256"])
def test_grouped_is_exact_on_whole_numbers(monkeypatch, large_blocks, tile, out):
    """Whole numbers with scales of powers of two, gathered and not, more tiles than the chip holds at once and 7 steps of K
    (blocks of the widest bf16 tiles load the next tile in a tile's last steps), 4 (they do not), 1 and a half.

    Exact: a row's largest weight is 448 and times 4 is 1792 < 2^11, so the 8-bit unit's cut at 2^-13 of the largest product
    leaves whole numbers whole; sums stay below 1792 + 832 * 16 < 2^24.  A bf16 output is their rounding.  Each expert's rows
    are also spmm24_f8's, bit for bit."""
    need_gpu()
    if tile:
        monkeypatch.setenv("P24_F8_TILE", tile)
    g = torch.Generator(device="cuda").manual_seed(3)
    whole = lambda low, high, *shape: torch.randint(low, high, shape, generator=g, device="cuda").float()  # noqa: E731
    for E, M, K, most in ((60, 1100, 832, 600), (30, 520, 448, 400), (7, 300, 192, 200), (3, 65, 64, 70)):
        counts = torch.randint(0, most + 1, (E,), generator=torch.Generator().manual_seed(K)).tolist()
        counts[0], counts[1], counts[-1] = 0, 257, 1
        offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
        ends = offsets.tolist()
        W = whole(-4, 5, E, M, K)
        W.view(E, M, K // 4, 4)[..., 1::2] = 0              # two of every four
        W[:, :, 0] = 448
        ws = torch.exp2(whole(-6, 3, E, M))
        c = p24.compress_f8_experts(W * ws[:, :, None])
        assert torch.equal(c.scale, ws)
        for x_rows in (ends[-1], 77):
            q, xs = whole(-4, 5, x_rows, K), torch.exp2(whole(-4, 5, x_rows))
            x = p24.Quantized8(q.to(torch.float8_e4m3fn), xs)
            tokens = None if x_rows == ends[-1] else torch.randint(0, x_rows, (ends[-1],), generator=g, device="cuda", dtype=torch.int32)
            y = p24.spmm24_f8_grouped(c, x, offsets, tokens=tokens, out_dtype=out)
            n = p24.lib().prune24_f8_bytes(M, K)
            for e in range(E):
                a, b = ends[e], ends[e + 1]
                if a == b:
                    continue
                src = slice(a, b) if tokens is None else tokens[a:b].long()
                want = (q[src].double() @ W[e].double().T) * xs[src].double()[:, None] * ws[e].double()
                assert torch.equal(y[a:b], want.float().to(out)), (E, e)
                if e % 10 == 1:
                    one = p24.Compressed24F8(c.data[e * n:(e + 1) * n], c.scale[e], M, K)
                    rows = p24.Quantized8(x.values[src].contiguous(), xs[src].contiguous())
                    assert torch.equal(y[a:b], p24.spmm24_f8(one, rows, out_dtype=out)), (E, e)
