"""One feed-forward layer of experts on 8-bit 2:4-sparse weights beside a dense shared expert in 8 bits with
block scales, as a serving loop would run it.

    python examples/experts_f8.py [--tokens 1] [--width 2048] [--hidden 1024] [--experts 64] [--k 6] [--steps 50]

Random weights, compressed once; then RMS norm with the residual, the router's logits (a torch product: routers
stay in higher precision), the layer of experts and the shared expert, eagerly and as a replayed graph.
Prints the times, the bytes of weights that the chosen experts hold, and how far the output, residual included, is
from the same layer in fp64 on the dequantized weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_sparse_gemm_prune24_amd as p24  # noqa: E402


def timed(f, steps):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(steps):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / steps * 1e3


def expert(c, e):
    """Dense fp64 weight of expert e."""
    n = c.data.numel() // c.E
    return p24.decompress_f8(p24.Compressed24F8(c.data[e * n:(e + 1) * n], c.scale[e], c.M, c.K)).double()


def dense(w):
    m, k = w.values.shape
    return w.values.double() * w.scale.double().repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)[:, :k]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--k", type=int, default=6)
    ap.add_argument("--steps", type=int, default=50)
    o = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gate_up = p24.compress_f8_experts(0.02 * randn(2 * o.hidden, o.width) for _ in range(o.experts))
    down = p24.compress_f8_experts(0.02 * randn(o.width, o.hidden) for _ in range(o.experts))
    shared_up = p24.quantize_weight_f8_block(0.02 * randn(2 * o.hidden, o.width))
    shared_down = p24.quantize_weight_f8_block(0.02 * randn(o.width, o.hidden))
    router = 0.05 * randn(o.experts, o.width)
    x, r = randn(o.tokens, o.width).bfloat16(), randn(o.tokens, o.width).bfloat16()
    w = 1 + 0.1 * randn(o.width)

    def layer():
        n, h = p24.rms_norm(x, w, residual=r, out_dtype=torch.bfloat16)
        logits = n.float() @ router.t()
        y = p24.feed_forward_f8_experts(p24.gated_act(n, act="none"), logits, o.k, gate_up, down, residual=h)
        gu = p24.gemm_f8_block(shared_up, p24.quantize_f8_block(n))
        a = p24.quantize_f8_block(gu[:, :o.hidden], gu[:, o.hidden:], act="silu")
        return p24.gemm_f8_block(shared_down, a, residual=y), h, n, logits

    y, h, n, logits = layer()
    eager = timed(layer, o.steps)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = layer()[0]
    replay = timed(graph.replay, o.steps)
    assert torch.equal(y, y2)

    plan = p24.route(logits, o.k)
    n = n.double()
    want = torch.zeros_like(n)
    used = sorted(set(plan.experts.flatten().tolist()))
    for e in used:
        t, j = (plan.experts == e).nonzero(as_tuple=True)
        z = n[t] @ expert(gate_up, e).T
        z = (torch.nn.functional.silu(z[:, :o.hidden]) * z[:, o.hidden:]) @ expert(down, e).T
        want.index_add_(0, t, z * plan.weights[t, j].double()[:, None])
    z = n @ dense(shared_up).T
    want += (torch.nn.functional.silu(z[:, :o.hidden]) * z[:, o.hidden:]) @ dense(shared_down).T
    out = h.double() + want      # two bf16 roundings of it, and the 8-bit operands of `want`
    off = ((y.double() - out).norm() / out.norm()).item()
    mb = (gate_up.data.numel() + down.data.numel()) / o.experts * len(used) / 1e6
    print(f"{o.tokens} tokens, {o.k} of {o.experts} experts {o.width} -> {o.hidden} -> {o.width}: eager {eager:.1f} us, "
          f"graph {replay:.1f} us, {mb:.0f} MB of expert weights, relative error {off:.4f}")


if __name__ == "__main__":
    main()
