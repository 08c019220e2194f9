"""The largest calls that the headers allow, on the host (no GPU): they get as far as the launch, which fails for want
of a device.  The pointers are fake and never dereferenced; with a device the calls are not made."""
import pytest

torch = pytest.importorskip("torch")
p24 = pytest.importorskip("structured_sparse_gemm_prune24_amd")
P = 1 << 20
MOST = 65535 * 32          # rows of a grouped product
F32, BF16 = 0, 1

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are fake: only where no kernel can start")


def _grouped(rows, E, M, K, dtype):
    return p24.lib().spmm24_f8_grouped(P, P, E, M, K, P, K, P, rows, P, None, rows, P, dtype, M, None, 0, None)


@pytest.mark.parametrize("tile", [None, "tokens", "64x32", "256x256"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("E", [1, 2, 64, 1024])
def test_grouped_takes_all_rows_that_it_allows(monkeypatch, E, dtype, tile):
    """Narrow weights prefer the kernel for few rows, whose grid does not hold all of them."""
    if tile:
        monkeypatch.setenv("P24_F8_TILE", tile)
    for M, K in ((1, 64), (32, 64), (32, 512), (64, 64), (4096, 1024)):
        for rows in (1, MOST - 64 * 1024, MOST):
            assert _grouped(rows, E, M, K, dtype) == -6, (M, K, rows)      # P24_ERR_HIP: no device
        assert _grouped(MOST + 1, E, M, K, dtype) == p24.P24_ERR_UNSUPPORTED
