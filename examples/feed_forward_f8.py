"""One feed-forward layer on 8-bit 2:4-sparse weights, as a serving loop would run it.

    python examples/feed_forward_f8.py [--tokens 1] [--width 4096] [--hidden 11264] [--steps 50]

Random weights, compressed once; then the layer (RMS norm with the residual, stacked gate and up
product, gated activation, down product adding to the residual stream) eagerly and as a replayed
graph.  Prints the time of a layer, the weight bytes it read, and how far its output is from the
same layer in fp64 on the dequantized weights.
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


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=11264)
    ap.add_argument("--steps", type=int, default=50)
    o = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gate_up = p24.compress_f8(0.02 * randn(2 * o.hidden, o.width))
    down = p24.compress_f8(0.02 * randn(o.width, o.hidden))
    x, r = randn(o.tokens, o.width).bfloat16(), randn(o.tokens, o.width).bfloat16()
    w = 1 + 0.1 * randn(o.width)

    layer = lambda: p24.feed_forward_f8(x, r, w, gate_up, down)  # noqa: E731
    y, h = layer()
    eager = timed(layer, o.steps)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, _ = layer()
    replay = timed(graph.replay, o.steps)
    assert torch.equal(y, y2)

    d = torch.float64
    n = x.to(d) + r.to(d)
    n = n / torch.sqrt(n.square().mean(1, keepdim=True) + 1e-6) * w.to(d)
    z = n @ p24.decompress_f8(gate_up).to(d).T
    a = torch.nn.functional.silu(z[:, :o.hidden]) * z[:, o.hidden:]
    want = a @ p24.decompress_f8(down).to(d).T
    off = ((y.to(d) - h.to(d) - want).norm() / want.norm()).item()
    mb = (gate_up.data.numel() + down.data.numel()) / 1e6
    print(f"{o.tokens} tokens, {o.width} -> {o.hidden} -> {o.width}: eager {eager:.1f} us, graph {replay:.1f} us, "
          f"{mb:.0f} MB of weights ({mb / replay:.2f} TB/s), relative error {off:.3f}")


if __name__ == "__main__":
    main()
