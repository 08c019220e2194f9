"""GPU tests of the block-scaled quantisation: 8 bits that follow from the formula alone (the rounded quotient y / s,
then e4m3), for zeros of either sign and scales down to 2^-126."""
import numpy as np
import pytest

from gpu_util import need_gpu, torch
from test_gpu_f8_block import _blocks_ref

p24 = pytest.importorskip("structured_sparse_gemm_prune24_amd")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_quantize_keeps_the_sign_of_zeros(dtype):
    """-0 is e4m3's -0: of a row, of a gated row whose product is -0, of a block of zeros, of a weight."""
    need_gpu()
    x = torch.randn(9, 500, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[:, ::3] = 0.0
    x[:, 1::3] = -0.0
    x[2, 128:256] = -0.0
    q, s = _blocks_ref(x.float(), 1)
    assert (q == 0x80).any()
    got = p24.quantize_f8_block(x.cuda())
    assert np.array_equal(got.scale.cpu().numpy(), s.T)
    assert np.array_equal(got.values.contiguous().view(torch.uint8).cpu().numpy(), q)
    got = p24.quantize_f8_block(torch.ones_like(x).cuda(), x.cuda())
    assert np.array_equal(got.values.contiguous().view(torch.uint8).cpu().numpy(), q)
    W = x.repeat(20, 2)[:, :900]
    q, s = _blocks_ref(W.float(), 128)
    got = p24.quantize_weight_f8_block(W.cuda())
    assert np.array_equal(got.scale.cpu().numpy(), s)
    assert np.array_equal(got.values.contiguous().view(torch.uint8).cpu().numpy(), q)


def _near_borders(seed, rows, width, low, high, tall):
    """fp32 values whose quotients by their block's scale lie on and next to the borders between e4m3 values; the blocks'
    scales are spread over 2^low to 2^high."""
    rng = np.random.default_rng(seed)
    nr, nb = -(-rows // tall), -(-width // 128)
    top = np.float32(448) * np.exp2(rng.uniform(low, high, (nr, nb))).astype(np.float32)
    s = np.maximum((top / np.float32(448)).astype(np.float32), np.float32(2.0 ** -126))
    per = s.repeat(tall, 0)[:rows].repeat(128, 1)[:, :width].astype(np.float64)
    # borders: (m + 1/2) 2^k of the normal values, multiples of 2^-10 of the subnormal ones
    normal = (rng.integers(8, 16, per.shape) + 0.5) * np.exp2(rng.integers(-9, 5, per.shape).astype(np.float64))
    border = np.where(rng.random(per.shape) < 0.2, rng.integers(0, 17, per.shape) * 2.0 ** -10, normal)
    border = border * np.where(rng.random(per.shape) < 0.5, -1, 1)
    y = (per * border).astype(np.float32)
    for _ in range(2):
        step = rng.integers(-1, 2, per.shape)
        y = np.where(step == 0, y, np.nextafter(y, np.float32(np.inf) * np.where(step < 0, -1, 1).astype(np.float32)))
    y[::tall, ::128] = top                       # each block's largest
    return torch.from_numpy(y)


@pytest.mark.parametrize("low,high", [(-126, -125), (-125, -120), (-120, -100), (-100, -85), (-60, 60), (100, 118)])
def test_quantize_next_to_borders(low, high):
    need_gpu()
    for tokens, width in ((16, 4096), (33, 500)):
        x = _near_borders(1, tokens, width, low, high, 1)
        q, s = _blocks_ref(x, 1)
        got = p24.quantize_f8_block(x.cuda())
        assert np.array_equal(got.scale.cpu().numpy(), s.T)
        assert np.array_equal(got.values.contiguous().view(torch.uint8).cpu().numpy(), q)
        b = x.bfloat16()
        q, s = _blocks_ref(b.float(), 1)
        got = p24.quantize_f8_block(b.cuda())
        assert np.array_equal(got.scale.cpu().numpy(), s.T)
        assert np.array_equal(got.values.contiguous().view(torch.uint8).cpu().numpy(), q)
    W = _near_borders(2, 300, 1000, low, high, 128)
    q, s = _blocks_ref(W, 128)
    got = p24.quantize_weight_f8_block(W.cuda())
    assert np.array_equal(got.scale.cpu().numpy(), s)
    assert np.array_equal(got.values.contiguous().view(torch.uint8).cpu().numpy(), q)
