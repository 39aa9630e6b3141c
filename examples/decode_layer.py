"""One decode layer of a mixture-of-experts model from the library's calls:

    norm (+ residual) -> q, k, v matvecs on its 8-bit output -> append to the
    8-bit cache -> page selection -> attention over the selected pages ->
    output matvec + residual -> norm -> router -> experts

run for a batch of sequences with random weights, first eagerly on a prompt,
then as a captured CUDA graph that is replayed while the sequences grow.  With
--whole also what stands between them: each sequence's low-rank adapter on the q,
k, v projection, the norm and rotation of the heads, expert selection with a balance
bias and groups, and after the layer a head with the log probabilities of the
tokens.

    python examples/decode_layer.py [--steps 16] [--seqs 8] [--prompt 700] [--whole]
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
                 page=64, pages_per_seq=16, select=8, seed=0, whole=False, adapters=4, rank=16, vocab=4096):
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
        self.whole = whole
        if not whole:
            return

        def randn(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.rope = api.rope(head_dim, torch.exp(torch.arange(head_dim // 2, device="cuda") * (-2 * 9.21 / head_dim)))
        self.q_norm, self.k_norm = 1 + 0.1 * randn(head_dim), 1 + 0.1 * randn(head_dim)
        # a pool of adapters; each sequence has one, or none (-1)
        self.lora = api.lora((randn(adapters, rank, hidden) / hidden ** 0.5).bfloat16(),
                             (0.1 * randn(adapters, self.rows, rank)).bfloat16())
        self.adapter = (torch.arange(seqs, device="cuda") % (adapters + 1) - 1).to(torch.int32)
        self.groups = 4 if experts % 4 == 0 and 2 * (experts // 4) >= top_k else 1
        self.balance = 0.05 * randn(experts)
        self.vocab, self.w_head = vocab, weights(api.Q8_0, vocab, hidden)

    def qkv(self, x8, x, lens, starts=None, seq=None):
        """The fused projection of the tokens x (x8 in the 8-bit layout), q and k of it normed
        and turned in place, split into views of q, k and v.  The tokens are the last ones
        of sequences of these lens; seq: each token's sequence (None: token i of sequence i)."""
        n = x8[0].shape[0]
        y = api.run_q8(api.Q8_0, self.w_qkv, *x8, self.rows, self.hidden)
        if self.whole:
            y = api.lora_run(self.lora, self.adapter if seq is None else self.adapter[seq], x, y, out=y)
        y = y.view(n, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = y.split((self.heads, self.kv_heads, self.kv_heads), 1)
        if self.whole:
            api.norm_rope(self.rope, q, k, self.q_norm, self.k_norm, lens=lens, starts=starts, q_out=q, k_out=k)
        return q, k, v

    def prompt(self, x, starts):
        """Put prompts (x [n_tok][hidden], ragged by starts) into the cache."""
        n = x.shape[0]
        first = self.lens.clone()
        self.lens += starts[1:] - starts[:-1]
        seq = torch.repeat_interleave(torch.arange(self.seqs, device="cuda"), starts.diff(), output_size=n)
        parts = []
        for i in range(0, n, 64):  # (the matvecs' limit)
            m = min(64, n - i)
            # what of each sequence this piece holds, and how long that makes it
            part = (starts - i).clamp(0, m).to(torch.int32)
            lens = first + ((starts[1:] - i).clamp(max=m) + i - starts[:-1]).clamp(min=0).to(torch.int32)
            y, x8, _ = api.rms_norm(x[i:i + 64], self.norm1, want="both" if self.whole else "q8")
            parts.append(self.qkv(x8, y, lens, part, seq[i:i + m]))
        k, v = (torch.cat([p[j] for p in parts]) for j in (1, 2))
        api.kv_append(self.cache, k, v, self.table, self.lens, starts)

    def step(self, x, residual):
        """One token per sequence: x and residual [seqs][hidden] -> (experts'
        output, residual), the next layer's inputs."""
        self.lens += 1
        y, x8, residual = api.rms_norm(x, self.norm1, r=residual, want="both" if self.whole else "q8")
        q, k, v = self.qkv(x8, y, self.lens)
        api.kv_append(self.cache, k, v, self.table, self.lens)
        pages = api.kv_select(self.cache, q, self.table, self.lens, self.select)
        o = api.kv_attend(self.cache, q, self.table, self.lens, pages=pages)
        o = o.reshape(self.seqs, self.heads * self.dim)
        h = api.run_residual(api.Q8_0, self.w_out, o, residual, self.hidden, self.heads * self.dim)
        y = api.rms_norm(h, self.norm2)[0]
        if self.whole:
            logits = api.run(api.Q8_0, self.w_router, y, self.experts, self.hidden)
            ids, gates = api.route_select(logits, self.top_k, api.GATING_SIGMOID, bias=self.balance, groups=self.groups,
                                          keep=max(1, self.groups // 2), scale=2.5)
        else:
            ids, gates, _ = api.route_run(api.Q8_0, self.w_router, y, self.experts, self.hidden, self.top_k)
        return api.moe_run(self.moe, ids, gates, y), h

    def score(self, x, residual, tokens, n_top=5):
        """Log probabilities of the tokens (int32 [seqs][n]) after the layer's outputs, the
        entropy and the n_top likeliest tokens with theirs."""
        _, x8, _ = api.rms_norm(x, self.norm2, r=residual, want="q8")
        logits = api.run_q8(api.Q8_0, self.w_head, *x8, self.vocab, self.hidden)
        logp, _, entropy, ids, top = api.logprobs(logits, tokens, n_top)
        return logp, entropy, ids, top


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700, help="tokens of the longest prompt")
    ap.add_argument("--whole", action="store_true", help="with adapters, rotation, grouped routing and log probabilities")
    a = ap.parse_args()
    torch.manual_seed(0)
    layer = Layer(seqs=a.seqs, pages_per_seq=-(-(a.prompt + a.steps + 8) // 64), whole=a.whole)
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
    if a.whole:
        logp, entropy, ids, top = layer.score(x, r, torch.zeros(a.seqs, 1, dtype=torch.int32, device="cuda"))
        print(f"entropy {float(entropy.mean()):.3f}, log probability of token 0 {float(logp.mean()):.3f}, "
              f"of the likeliest {float(top[:, 0].mean()):.3f}")
    err = api.get_device_error()
    print(f"{a.seqs} sequences of {int(layer.lens.min())} to {int(layer.lens.max())} tokens: {1e6 * t:.1f} us a layer "
          f"and step, output rms {float(y.square().mean().sqrt()):.3f}, device errors {err:#x}")
    return err


if __name__ == "__main__":
    sys.exit(main())
