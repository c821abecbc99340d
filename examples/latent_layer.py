"""An attention block over a latent cache on the library's operators, with random
weights: prompts in the expanded form, then single tokens in the absorbed form,
the cache, keys and values of all heads being one row of 576 values a token.

    x  -> latents and queries          gemm_bf16
       -> norm, rotation, cache        latent_append
    prompts:
       -> keys and values of the heads heads_gemm
       -> attention                    latent_attention_expanded
    single tokens:
       -> queries against latents      heads_gemm
       -> attention                    latent_attention
       -> values of the heads          heads_gemm
       -> output projection            gemm_bf16

    python examples/latent_layer.py --sequences 1 8 64 --length 4000

prints, for each number of sequences, the time of a single token's step called
step by step and replayed as a HIP graph, and whether the two agree.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import latency_skinny_gemm_amd as skg  # noqa: E402

NOPE, ROPE, V, LATENT = 128, 64, 128, 512


class LatentBlock:
    """Weights of one block and its cache, float8_e4m3fn or bf16."""

    def __init__(self, hidden=2048, heads=16, pages=1024, page_size=64, width=128, e4m3=False, device="cuda"):
        self.hidden, self.heads, self.width = hidden, heads, width
        self.device = torch.device(device)
        self.softmax_scale = (NOPE + ROPE) ** -0.5

        def weight(*shape):
            return (torch.randn(*shape, device=self.device) * shape[-1] ** -0.5).bfloat16()

        self.wq, self.wkv = weight(heads * (NOPE + ROPE), hidden), weight(LATENT + ROPE, hidden)
        self.gain = (1 + 0.1 * torch.randn(LATENT, device=self.device)).bfloat16()
        self.up = weight(heads, NOPE + V, LATENT)                        # latents -> a head's keys and values
        self.absorb = self.up[:, :NOPE].transpose(1, 2).contiguous()     # queries -> against latents
        self.values = self.up[:, NOPE:].contiguous()                     # sums of latents -> sums of values
        self.wo = weight(hidden, heads * V)
        self.scale = torch.full((1,), 0.03, device=self.device) if e4m3 else None
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.cache = torch.zeros(pages, page_size, LATENT + ROPE, dtype=dtype, device=self.device)
        rows = torch.arange(width * page_size, dtype=torch.float64)[:, None]
        angle = rows * 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)
        self.rotations = torch.cat((angle.cos(), angle.sin()), 1).float().to(self.device)

    def prompt(self, x, q_starts, table, kv_lens):
        """Whole prompts, x [T, hidden]; kv_lens are their lengths."""
        T = x.shape[0]
        q = skg.gemm_bf16(x, self.wq).view(T, self.heads, NOPE + ROPE)
        new = skg.latent_append(skg.gemm_bf16(x, self.wkv), self.cache, table, kv_lens, self.rotations, q_starts=q_starts,
                                weight=self.gain, scale=self.scale, q_rope=q[..., NOPE:], q_rope_out=q[..., NOPE:], latent=True)
        latent = new.latent
        kv = skg.heads_gemm(latent[:, None, :LATENT].expand(T, self.heads, LATENT), self.up)
        o = skg.latent_attention_expanded(q, kv, latent[:, LATENT:], q_starts, self.softmax_scale)
        return skg.gemm_bf16(o.view(T, self.heads * V), self.wo)

    def step(self, x, table, kv_lens):
        """One token of each sequence, x [B, hidden]; kv_lens count it."""
        B = x.shape[0]
        q = skg.gemm_bf16(x, self.wq).view(B, self.heads, NOPE + ROPE)
        absorbed = torch.empty(B, self.heads, LATENT + ROPE, dtype=torch.bfloat16, device=x.device)
        skg.latent_append(skg.gemm_bf16(x, self.wkv), self.cache, table, kv_lens, self.rotations, weight=self.gain,
                          scale=self.scale, q_rope=q[..., NOPE:], q_rope_out=absorbed[..., LATENT:])
        skg.heads_gemm(q[..., :NOPE], self.absorb, out=absorbed[..., :LATENT])
        o = skg.latent_attention(absorbed, self.cache, table, kv_lens, self.softmax_scale, scale=self.scale)
        return skg.gemm_bf16(skg.heads_gemm(o, self.values).view(B, self.heads * V), self.wo)

    def reserve(self, max_tokens, stream):
        """Workspace for graphs captured on `stream`."""
        skg.reserve(max_tokens, max(self.heads * (NOPE + ROPE), self.hidden), max(self.hidden, self.heads * V), 64, stream=stream)
        skg.reserve_latent(self.heads, stream=stream)

    def capture(self, x, table, kv_lens):
        """(graph, its output): replay() makes a step of what x, table and kv_lens hold then."""
        stream = torch.cuda.Stream(self.device)
        self.reserve(x.shape[0], stream)
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
            out = self.step(x, table, kv_lens)
        return graph, out


def timed(f, n=100):
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
    p.add_argument("--sequences", type=int, nargs="+", default=[1, 8, 64])
    p.add_argument("--length", type=int, default=4000)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--heads", type=int, default=16)
    p.add_argument("--e4m3", action="store_true")
    o = p.parse_args(argv)
    torch.manual_seed(0)
    width = -(-o.length // 64)
    block = LatentBlock(o.hidden, o.heads, max(o.sequences) * width, 64, width, o.e4m3)
    block.cache.copy_(torch.randn(block.cache.shape, device=block.device, dtype=torch.bfloat16).to(block.cache.dtype))
    for B in o.sequences:
        x = torch.randn(B, o.hidden, device=block.device).bfloat16()
        table = torch.randperm(B * width, device=block.device).view(B, width).to(torch.int32)
        kv_lens = torch.full((B,), o.length, dtype=torch.int32, device=block.device)
        eager = timed(lambda: block.step(x, table, kv_lens))
        graph, out = block.capture(x, table, kv_lens)
        replayed = timed(graph.replay)
        same = torch.equal(out, block.step(x, table, kv_lens))
        print(f"{B:4d} sequences of {o.length}: {eager:8.1f} us step by step, {replayed:8.1f} us as a graph"
              f"{'' if same else ', THE TWO DIFFER'}", flush=True)


if __name__ == "__main__":
    main()
