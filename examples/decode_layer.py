"""One decode layer of a mixture-of-experts model from the library's calls:

    norm (+ residual) -> q, k, v matvecs on its 8-bit output -> append to the
    8-bit cache -> page selection -> attention over the selected pages ->
    output matvec + residual -> norm -> router -> experts

run for a batch of sequences with random weights, first eagerly on a prompt,
then as a captured CUDA graph that is replayed while the sequences grow.

    python examples/decode_layer.py [--steps 16] [--seqs 8] [--prompt 700]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from moe_matvec_gb300 import api  # noqa: E402


class Layer:
    """Weights, cache and buffers of one layer for a fixed batch size (at most
    64 sequences, the matvecs' limit)."""

    def __init__(self, hidden=2048, heads=16, kv_heads=4, head_dim=128, experts=16, top_k=4, ffn=512, seqs=8,
                 page=64, pages_per_seq=16, select=8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weights(fmt, rows, cols):
            return api.quantize_weights(fmt, torch.randn(rows, cols, generator=g, device="cuda") * 0.02)

        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, head_dim
        self.experts, self.top_k, self.select, self.seqs, self.page = experts, top_k, select, seqs, page
        self.rows = (heads + 2 * kv_heads) * head_dim
        self.norm1 = 1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")
        self.norm2 = 1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")
        self.w_qkv = weights(api.Q8_0, self.rows, hidden)
        self.w_out = weights(api.Q8_0, hidden, heads * head_dim)
        self.w_router = weights(api.Q8_0, experts, hidden)
        gate_up = torch.stack([weights(api.Q4_K, 2 * ffn, hidden) for _ in range(experts)])
        down = torch.stack([weights(api.Q4_K, hidden, ffn) for _ in range(experts)])
        self.moe = api.moe_experts(experts, hidden, ffn, api.Q4_K, api.Q4_K, gate_up, down)
        self.cache = api.kv_cache(kv_heads, head_dim, page, seqs * pages_per_seq, bounds=True)
        perm = torch.randperm(seqs * pages_per_seq, generator=g, device="cuda").to(torch.int32)
        self.table = perm.reshape(seqs, pages_per_seq).contiguous()
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")

    def qkv(self, n, x8):
        """The fused projection of n tokens, split into views of q, k and v."""
        y = api.run_q8(api.Q8_0, self.w_qkv, *x8, self.rows, self.hidden)
        y = y.view(n, self.heads + 2 * self.kv_heads, self.dim)
        return y.split((self.heads, self.kv_heads, self.kv_heads), 1)

    def prompt(self, x, starts):
        """Put prompts (x [n_tok][hidden], ragged by starts) into the cache."""
        n = x.shape[0]
        parts = [self.qkv(min(64, n - i), api.rms_norm(x[i:i + 64], self.norm1, want="q8")[1])
                 for i in range(0, n, 64)]
        k, v = (torch.cat([p[j] for p in parts]) for j in (1, 2))
        self.lens += starts[1:] - starts[:-1]
        api.kv_append(self.cache, k, v, self.table, self.lens, starts)

    def step(self, x, residual):
        """One token per sequence: x and residual [seqs][hidden] -> (experts'
        output, residual), the next layer's inputs."""
        self.lens += 1
        _, x8, residual = api.rms_norm(x, self.norm1, r=residual, want="q8")
        q, k, v = self.qkv(self.seqs, x8)
        api.kv_append(self.cache, k, v, self.table, self.lens)
        pages = api.kv_select(self.cache, q, self.table, self.lens, self.select)
        o = api.kv_attend(self.cache, q, self.table, self.lens, pages=pages)
        o = o.reshape(self.seqs, self.heads * self.dim)
        h = api.run_residual(api.Q8_0, self.w_out, o, residual, self.hidden, self.heads * self.dim)
        y = api.rms_norm(h, self.norm2)[0]
        ids, gates, _ = api.route_run(api.Q8_0, self.w_router, y, self.experts, self.hidden, self.top_k)
        return api.moe_run(self.moe, ids, gates, y), h


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700, help="tokens of the longest prompt")
    a = ap.parse_args()
    torch.manual_seed(0)
    layer = Layer(seqs=a.seqs, pages_per_seq=-(-(a.prompt + a.steps + 8) // 64))
    lens = torch.randint(1, a.prompt + 1, (a.seqs,))
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).cuda()
    layer.prompt(torch.randn(int(lens.sum()), layer.hidden, device="cuda"), starts)
    x, r = torch.randn(a.seqs, layer.hidden, device="cuda"), torch.randn(a.seqs, layer.hidden, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, r)  # first launches configure the kernels
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y, h = layer.step(x, r)
        side.synchronize()
        t = time.perf_counter()
        for _ in range(a.steps):
            graph.replay()
            x.copy_(y)
            r.copy_(h)
        side.synchronize()
        t = (time.perf_counter() - t) / a.steps
    err = api.get_device_error()
    print(f"{a.seqs} sequences of {int(layer.lens.min())} to {int(layer.lens.max())} tokens: {1e6 * t:.1f} us a layer "
          f"and step, output rms {float(y.square().mean().sqrt()):.3f}, device errors {err:#x}")
    return err


if __name__ == "__main__":
    sys.exit(main())
