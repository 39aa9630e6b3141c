"""The decode layer of examples/decode_layer.py: its attention against 64 bits
on what the layer's own calls put into the cache, and the captured graph
against the eager step."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import kv_ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def fresh(example, seed=1):
    layer = example.Layer(hidden=512, heads=4, kv_heads=2, head_dim=64, experts=8, top_k=2, ffn=256, seqs=3, page=16,
                          pages_per_seq=12, select=4, seed=seed)
    lens = torch.tensor([100, 1, 37])
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).cuda()
    g = torch.Generator().manual_seed(seed)
    layer.prompt(torch.randn(138, 512, generator=g).cuda(), starts)
    return layer, torch.randn(3, 512, generator=g).cuda(), torch.randn(3, 512, generator=g).cuda()


def test_the_steps_attention_is_the_definitions(lib, example):
    layer, x, r = fresh(example)
    for _ in range(3):
        seen = {}
        attend, select = api.kv_attend, api.kv_select
        try:
            api.kv_select = lambda c, q, *a, **k: seen.setdefault("ids", select(c, q, *a, **k))
            api.kv_attend = lambda c, q, *a, **k: (seen.setdefault("q", q), seen.setdefault("out", attend(c, q, *a, **k)))[1]
            x, r = layer.step(x, r)
        finally:
            api.kv_attend, api.kv_select = attend, select
        ref = kv_ref.Cache(2, 64, 16, 36)
        ref.pages[:] = layer.cache.page_tensor.cpu().numpy()
        ref.bounds[:] = layer.cache.bounds_tensor.cpu().numpy()
        q, table, lens = seen["q"].cpu().numpy(), layer.table.cpu().numpy(), layer.lens.tolist()
        ids = kv_ref.select(ref, q, table, lens, np.arange(4), 4)
        assert np.array_equal(seen["ids"].cpu().numpy(), ids)
        want, mag, arg = kv_ref.attend(ref, q, table, lens, np.arange(4), 64 ** -0.5, pages=ids)
        # (tolerance: tests/test_kv_attend_gpu.py)
        err = np.abs(seen["out"].double().cpu().numpy() - want)
        assert (err <= (2.0 ** -17 * arg + 2.0 ** -16) * mag).all()
    assert torch.isfinite(x).all() and api.get_device_error() == 0


def test_a_captured_step_replays_like_the_eager_one(lib, example):
    a, x, r = fresh(example)
    b, _, _ = fresh(example)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ya, ha = a.step(x, r)
        graph = torch.cuda.CUDAGraph()
        gx, gr = ya.clone(), ha.clone()
        with torch.cuda.graph(graph, stream=side):
            gy, gh = a.step(gx, gr)
        side.synchronize()
        y, h = b.step(x, r)
        for _ in range(20):  # across page borders
            graph.replay()
            y, h = b.step(y, h)
            assert torch.equal(gy, y) and torch.equal(gh, h)
            gx.copy_(gy)
            gr.copy_(gh)
        side.synchronize()
    assert torch.equal(a.lens, b.lens) and api.get_device_error() == 0
