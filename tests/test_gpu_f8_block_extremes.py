"""GPU tests of the block-scaled quantisation: 8 bits that follow from the formula alone (the rounded quotient y / s,
then e4m3), for zeros of either sign."""
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
