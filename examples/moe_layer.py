"""A decode step's mixture-of-experts block on the library's operators, with
random weights:

    a  -> 4-bit projection             gemm_mxfp4
       -> residual addition and norm   rmsnorm
       -> router logits                gemm_bf16_f32
       -> experts and weights          route
       -> the experts' feed-forward    moe_mxfp4

    python examples/moe_layer.py --tokens 1 8 64

prints, for each number of tokens, the time of the block called step by step and
replayed as a HIP graph, and whether the two agree.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import latency_skinny_gemm_amd as skg  # noqa: E402


class MoeBlock:
    """Weights of one block; forward(a [T, hidden], residual [T, hidden]) ->
    (the experts' sum, the new residual)."""

    def __init__(self, hidden=2880, inter=2880, experts=32, k=4, x_format="e4m3", device="cuda"):
        self.hidden, self.inter, self.experts, self.k, self.x_format = hidden, inter, experts, k, x_format
        self.device = torch.device(device)

        def weight(*shape):
            return (torch.randn(*shape, device=self.device) * shape[-1] ** -0.5).bfloat16()

        def packed(w):
            return skg.mxfp4_pack(*skg.quant_mx(w, "e2m1"))

        self.wo = packed(weight(hidden, hidden))
        self.gain = (1 + 0.1 * torch.randn(hidden, device=self.device)).bfloat16()
        self.router = weight(experts, hidden)
        self.w13 = packed(weight(experts, 2 * inter, hidden))
        self.w2 = packed(weight(experts, hidden, inter))

    def reserve(self, max_tokens, stream):
        """Workspace for graphs captured on `stream`."""
        skg.reserve(max_tokens, max(self.experts, 1), self.hidden, 64, stream=stream)
        skg.reserve_moe(max_M=max_tokens, max_K=self.hidden, max_T=max_tokens, k=self.k, H=self.hidden,
                        I=self.inter, E=self.experts, stream=stream)

    def forward(self, a, residual):
        o = skg.gemm_mxfp4(a, self.wo, x_format=self.x_format)
        n = skg.rmsnorm(o, self.gain, residual=residual)
        weights, ids = skg.route(skg.gemm_bf16_f32(n.y, self.router), self.k)
        return skg.moe_mxfp4(n.y, ids, weights, self.w13, self.w2, x_format=self.x_format), n.residual

    def capture(self, a, residual):
        """(graph, its outputs): replay() recomputes them from a's and residual's memory."""
        stream = torch.cuda.Stream(self.device)
        self.reserve(a.shape[0], stream)
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
            out = self.forward(a, residual)
        return graph, out


def timed(f, n=200):
    for _ in range(10):
        f()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        f()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / n * 1e6


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, nargs="+", default=[1, 8, 64])
    p.add_argument("--hidden", type=int, default=2880)
    p.add_argument("--inter", type=int, default=2880)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("-k", type=int, default=4)
    p.add_argument("--x-format", choices=("e4m3", "e2m1"), default="e4m3")
    o = p.parse_args(argv)
    torch.manual_seed(0)
    block = MoeBlock(o.hidden, o.inter, o.experts, o.k, o.x_format)
    for T in o.tokens:
        a, r = (torch.randn(T, o.hidden, device=block.device).bfloat16() for _ in range(2))
        eager = timed(lambda: block.forward(a, r))
        graph, out = block.capture(a, r)
        replayed = timed(graph.replay)
        same = all(torch.equal(x, y) for x, y in zip(out, block.forward(a, r)))
        print(f"{T:4d} tokens: {eager:8.1f} us step by step, {replayed:8.1f} us as a graph"
              f"{'' if same else ', THE TWO DIFFER'}", flush=True)


if __name__ == "__main__":
    main()
