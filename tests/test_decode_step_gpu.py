"""The whole decode step of examples/decode_layer.py (adapters, head norm and
rotation, grouped routing, log probabilities beside the calls that were there): each
new call of a step against 64 bits on what the step hands it, prompts against the
same tokens step by step, and the captured graph against the eager step."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import step_ref
from tests.test_decode_layer_gpu import example  # noqa: F401

pytestmark = pytest.mark.gpu


def fresh(example, seed=1, seqs=3, prompt=(100, 1, 37)):  # noqa: F811
    layer = example.Layer(hidden=512, heads=4, kv_heads=2, head_dim=64, experts=8, top_k=2, ffn=256, seqs=seqs, page=16,
                          pages_per_seq=12, select=4, seed=seed, whole=True, adapters=3, rank=8, vocab=1000)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(int(sum(prompt)), 512, generator=g).cuda()
    starts = torch.tensor(np.concatenate([[0], np.cumsum(prompt)]), dtype=torch.int32).cuda()
    layer.prompt(x, starts)
    return layer, torch.randn(seqs, 512, generator=g).cuda(), torch.randn(seqs, 512, generator=g).cuda(), (x, starts)


def f64(t):
    return t.double().cpu().numpy()


def test_each_call_of_a_step_is_its_definition(lib, example, monkeypatch):  # noqa: F811
    layer, x, r, _ = fresh(example)
    seen = {}

    def spy(name):
        real = getattr(api, name)

        def call(*a, **k):
            # (the inputs as they are before the call, which may write to them)
            seen[name] = ([t.clone() if isinstance(t, torch.Tensor) else t for t in a], dict(k))
            out = real(*a, **k)
            seen[name] += ([t.clone() if isinstance(t, torch.Tensor) else t for t in (out if isinstance(out, tuple) else (out,))],)
            return out
        monkeypatch.setattr(api, name, call)

    for name in ("lora_run", "norm_rope", "route_select", "logprobs"):
        spy(name)
    for _ in range(3):
        x, r = layer.step(x, r)
        # tolerances: tests/test_lora_gpu.py, test_norm_rope_gpu.py, test_route_select_gpu.py
        (_, ids, xin, res), _, (y,) = seen["lora_run"]
        A, B, _, _ = layer.lora._tensors
        want, mag = step_ref.lora(f64(A), f64(B), ids.tolist(), f64(xin), f64(res), None, None)
        assert (np.abs(f64(y) - want) <= 2.0 ** -24 * (43 * mag + np.abs(want)) + 1e-37).all()
        (_, q, k, qw, kw), kw_args, (qo, ko) = seen["norm_rope"]
        pos = [[int(t) - 1] for t in layer.lens]
        assert torch.equal(kw_args["lens"], layer.lens)
        freq = f64(layer.rope._tensors[0])
        for a, w, o in ((q, qw, qo), (k, kw, ko)):
            want, mag = step_ref.norm_rope(f64(a), f64(w), 1e-6, pos, [0] * 32, freq, False, 1.0)
            assert (np.abs(f64(o) - want) <= 2.0 ** -19 * mag + 2.0 ** -24 * np.abs(want) + 1e-37).all()
        (logits, top_k, gating), args, (picks, gates) = seen["route_select"]
        want, g, below = step_ref.route(f64(logits), top_k, True, f64(args["bias"]), args["groups"], args["keep"], 2, True,
                                        args["scale"])
        assert np.array_equal(picks.cpu().numpy(), want)
        assert (np.abs(f64(gates) - g) <= 2.0 ** -24 * (48 + 2 * below) * g).all()
    logp, entropy, ids, top = layer.score(x, r, torch.tensor([[5, -1], [999, 0], [1, 1]], dtype=torch.int32).cuda())
    (logits, tokens, n_top), _, _ = seen["logprobs"]
    wp, _, wh, wi, wt, rest = step_ref.logprobs(f64(logits), tokens.cpu().numpy(), n_top, 1.0)
    N = 1000 / 512 + 94 + 4
    log_s = np.log1p(rest)
    assert np.array_equal(ids.cpu().numpy(), wi)
    assert (np.abs(f64(logp) - wp) <= 2.0 ** -24 * N * (log_s[:, None] + np.abs(wp))).all()
    assert (np.abs(f64(top) - wt) <= 2.0 ** -24 * N * (log_s[:, None] + np.abs(wt))).all()
    assert (np.abs(f64(entropy) - wh) <= 2.0 ** -24 * 2 * N * wh).all()
    assert api.get_device_error() == 0


def test_a_prompt_in_pieces_is_rotated_like_one_token_at_a_time(lib, example, monkeypatch):  # noqa: F811
    layer, _, _, (x, starts) = fresh(example)
    got = api.kv_read(layer.cache, layer.table, layer.lens, starts, x.shape[0])
    # the keys that went in: every token's by itself, at its position
    seq = torch.repeat_interleave(torch.arange(3), starts.cpu().diff())
    pos = (torch.arange(x.shape[0]) - starts.cpu()[seq]).to(torch.int32)
    keys = torch.empty(x.shape[0], 2, 64, device="cuda")
    for t in range(x.shape[0]):
        y, x8, _ = api.rms_norm(x[t:t + 1], layer.norm1, want="both")
        p = api.run_q8(api.Q8_0, layer.w_qkv, *x8, layer.rows, layer.hidden)
        p = api.lora_run(layer.lora, layer.adapter[seq[t]:seq[t] + 1].clone(), y, p)
        k = p.view(1, 8, 64)[:, 4:6].contiguous()
        keys[t] = api.norm_rope(layer.rope, k, None, layer.k_norm, pos=pos[t:t + 1, None].cuda())[0][0]
    # a code is off by at most half a step and a step more for each rescaling of its page; scales are amax / 127
    step = keys.abs().amax() / 127
    assert (got[0] - keys).abs().max() <= 3 * step
    assert api.get_device_error() == 0


def test_a_captured_step_replays_like_the_eager_one(lib, example):  # noqa: F811
    a, x, r, _ = fresh(example)
    b, _, _, _ = fresh(example)
    tokens = torch.tensor([[1], [2], [3]], dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ya, ha = a.step(x, r)
        a.score(ya, ha, tokens)
        graph = torch.cuda.CUDAGraph()
        gx, gr = ya.clone(), ha.clone()
        with torch.cuda.graph(graph, stream=side):
            gy, gh = a.step(gx, gr)
            got = a.score(gy, gh, tokens)
        side.synchronize()
        y, h = b.step(x, r)
        for i in range(20):  # across page borders
            if i == 10:  # adapters change between replays
                for layer in (a, b):
                    layer.adapter.copy_(torch.tensor([2, 2, -1], dtype=torch.int32))
            graph.replay()
            y, h = b.step(y, h)
            want = b.score(y, h, tokens)
            assert torch.equal(gy, y) and torch.equal(gh, h)
            assert all(torch.equal(p, q) for p, q in zip(got, want))
            gx.copy_(gy)
            gr.copy_(gh)
        side.synchronize()
    assert torch.equal(a.lens, b.lens) and api.get_device_error() == 0


def test_the_example_runs(lib, example, monkeypatch, capsys):  # noqa: F811
    monkeypatch.setattr("sys.argv", ["decode_layer.py", "--steps", "3", "--seqs", "4", "--prompt", "90", "--whole"])
    assert example.main() == 0
    assert "log probability" in capsys.readouterr().out
