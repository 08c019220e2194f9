"""GPU tests of the expert operators where their arguments leave the ordinary: sigmoids that leave fp32.

U = 2^-24 is half an fp32 step, relative."""
import numpy as np
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
