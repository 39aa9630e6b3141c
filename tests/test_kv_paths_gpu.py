"""The ways a batch can be divided, each through the tests of memory bounds,
given buffers, streams and graphs: attention in equal shares of the GPU with a
second kernel (a table of room for many tokens), in clusters of several CTAs (a
table of a few thousand), in clusters of one (a table as wide as the data), and
selection with its keys in the workspace (more than 8192 pages)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests.test_canary_gpu import Guarded
from tests.test_debug_gpu import both, same_bits
from tests.test_kv_attend_gpu import check, filled
from tests.test_kv_cache_gpu import Pair, dev32, randn, tables

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]
ROOM = {"shares": 100000, "clusters": 2500, "single": 0}


def roomy(table, P, way):
    """The same pages in a table of room for that many tokens."""
    more = max(ROOM[way] // P - table.shape[1], 0)
    return np.concatenate([table, np.full((len(table), more), -1, table.dtype)], 1)


@pytest.fixture(scope="module")
def dbg(lib):
    return api.load_debug()


@pytest.mark.parametrize("way", list(ROOM))
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P,G", [(64, 16, 2), (64, 32, 12), (128, 64, 6), (128, 32, 16), (192, 32, 3), (256, 64, 9)])
def test_range_checked_build(lib, dbg, way, dtype, D, P, G):
    rng = np.random.default_rng(D + P + G)
    lens, news = [700, 1, 40, 0, 129], [3, 1, 9, 0, 1]
    st = np.concatenate([[0], np.cumsum(news)])
    pair, table = filled(rng, 2, D, P, lens)
    td, ld, sd = dev32(roomy(table, P, way)), dev32(lens), dev32(st)
    one, q = randn(rng, 5, 2 * G, D, dtype=dtype), randn(rng, st[-1], 2 * G, D, dtype=dtype)

    def run():
        ids = api.kv_select(pair.dev, q, td, ld, 3, sd)
        return [ids, api.kv_attend(pair.dev, one, td, ld), api.kv_attend(pair.dev, one, td, ld, window=100),
                api.kv_attend(pair.dev, q, td, ld, sd), api.kv_attend(pair.dev, q, td, ld, sd, causal=False),
                api.kv_attend(pair.dev, q, td, ld, sd, window=70), api.kv_attend(pair.dev, q, td, ld, sd, pages=ids)]

    rel, d, err = both(dbg, run)
    assert err == 0
    assert all(same_bits(a, b) for a, b in zip(rel, d))
    check(pair, one, table, lens, None, rel[1])
    check(pair, q, table, lens, st, rel[3])


@pytest.mark.parametrize("way", list(ROOM))
@pytest.mark.parametrize("last", [16, 200])  # tokens of the last sequence: one tile, and several that are joined
def test_the_checks_are_live(lib, dbg, way, last):
    # the result's extent handed to the checks eight elements short: those stores are skipped and flagged
    rng = np.random.default_rng(last)
    lens = [300, 1, 33, last]
    pair, table = filled(rng, 2, 128, 16, lens)
    td, ld, q = dev32(roomy(table, 16, way)), dev32(lens), randn(rng, 4, 12, 128)
    want = api.kv_attend(pair.dev, q, td, ld)
    got = torch.full_like(q, 7)
    with api.using(dbg):
        api.get_device_error()
        api.debug_shrink_outputs(8)
        try:
            api.kv_attend(pair.dev, q, td, ld, out=got)
        finally:
            err = api.get_device_error()
            api.debug_shrink_outputs(0)
        assert err == api.DEVERR_RANGE
        assert torch.equal(got.flatten()[:-8], want.flatten()[:-8]) and (got.flatten()[-8:] == 7).all()
        api.kv_attend(pair.dev, q, td, ld, out=got)
        assert api.get_device_error() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("way", list(ROOM))
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P,H,G", [(64, 16, 1, 1), (64, 64, 2, 20), (128, 64, 3, 5), (128, 16, 1, 20), (192, 32, 2, 9),
                                     (256, 16, 2, 3)])
def test_guard_bands(lib, way, dtype, D, P, H, G):
    rng = np.random.default_rng(D + P)
    lens, news = [P + 3, 1, 400, 2 * P - 1], [P + 3, 1, 2, P]
    st = np.concatenate([[0], np.cumsum(news)])
    pair, table = filled(rng, H, D, P, lens)
    td, ld, sd, n = dev32(roomy(table, P, way)), dev32(lens), dev32(st), int(st[-1])
    q = randn(rng, n, H * G, D, dtype=dtype)
    ids = api.kv_select(pair.dev, q, td, ld, 3, sd)
    for pages in (None, ids):
        want = api.kv_attend(pair.dev, q, td, ld, sd, pages=pages)
        out, ws = Guarded((n, H * G, D), dtype, 1), Guarded((api.kv_attend_workspace_bytes(pair.dev, H * G, n, 4),), torch.uint8, 2)
        api.kv_attend(pair.dev, q, td, ld, sd, pages=pages, ws=ws.t, out=out.t)
        out.check_guards("out"), ws.check_guards("ws")
        assert same_bits(out.t, want)
        check(pair, q, table, lens, st, out.t, pages=None if pages is None else ids.cpu().numpy())
    got, ws = Guarded((n, H, 3), torch.int32, 3), Guarded((api.kv_select_workspace_bytes(pair.dev, n, td.shape[1]),), torch.uint8, 4)
    api.kv_select(pair.dev, q, td, ld, 3, sd, ws=ws.t, ids=got.t)
    got.check_guards("ids"), ws.check_guards("ws of selection")
    assert torch.equal(got.t, ids)


@pytest.mark.parametrize("way", list(ROOM))
def test_strided_queries_and_a_dirty_workspace(lib, way):
    rng = np.random.default_rng(33)
    lens = [1000, 77]
    pair, table = filled(rng, 2, 128, 32, lens)
    q = randn(rng, 2, 12, 128)[:, 2:10]
    td = dev32(roomy(table, 32, way))
    for fill in (0xFF, 0x00, 0x7F):
        ws = torch.full((api.kv_attend_workspace_bytes(pair.dev, 8, 2, 2),), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((2, 8, 128), float("nan"), device="cuda")
        assert api.kv_attend(pair.dev, q, td, dev32(lens), ws=ws, out=out) is out
        check(pair, q, table, lens, None, out)
        assert (way == "shares") == (not (ws == fill).all())  # this way alone writes its workspace


def test_workspaces_in_use_on_another_stream(lib):
    # both calls write the workspace that they make and drop: nobody may have its memory before the work is done
    rng = np.random.default_rng(37)
    H, D, P, n = 1, 64, 16, 8400 * 16 - 5
    cache = api.kv_cache(H, D, P, 8403, bounds=True)
    table = tables(rng, [n], P, 8403)
    for a in range(0, n, 60000):
        b = min(n, a + 60000)
        api.kv_append(cache, randn(rng, b - a, H, D), randn(rng, b - a, H, D), dev32(table), dev32([b]), dev32([0, b - a]))
    q, td, ld = randn(rng, 1, 4, D), dev32(table), dev32([n])
    want, picks = api.kv_attend(cache, q, td, ld), api.kv_select(cache, q, td, ld, 300)
    sizes = [api.kv_attend_workspace_bytes(cache, 4, 1, 1)] * 2 + [api.kv_select_workspace_bytes(cache, 1, td.shape[1])] * 2
    used = [torch.zeros(sizes[i], dtype=torch.uint8, device="cuda") for i in (0, 2)]
    api.kv_attend(cache, q, td, ld, ws=used[0]), api.kv_select(cache, q, td, ld, 300, ws=used[1])
    assert all(u.any() for u in used)  # (both are written)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # the work below starts some 10 ms later
    out = api.kv_attend(cache, q, td, ld, stream=side)
    ids = api.kv_select(cache, q, td, ld, 300, stream=side)
    other = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in sizes]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(ids, picks)
    assert not any(t.any() for t in other)
    assert api.get_device_error() == 0


@pytest.mark.parametrize("way", list(ROOM))
def test_graph_replays_as_lengths_grow(lib, way):
    rng = np.random.default_rng(36)
    H, D, P, first = 2, 128, 64, [100, 510]
    pair = Pair(H, D, P, 14)
    table = tables(rng, [300, 560], P, 14)
    lens = dev32(first)
    n = sum(first)
    pair.append(randn(rng, n, H, D), randn(rng, n, H, D), table, first, [0, first[0], n])
    k, v, q = randn(rng, 2, H, D), randn(rng, 2, H, D), randn(rng, 2, 8, D)
    td = dev32(roomy(table, P, way))
    ws = torch.empty(api.kv_attend_workspace_bytes(pair.dev, 8, 2, 2), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 8, D, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.kv_attend(pair.dev, q, td, lens, ws=ws, out=out)  # first launches configure the kernel
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            lens.add_(1)
            api.kv_append(pair.dev, k, v, td, lens)
            api.kv_attend(pair.dev, q, td, lens, ws=ws, out=out)
    torch.cuda.synchronize()
    for step in range(1, 40):  # one sequence passes 128 and the other 512 and 544: more tiles than were captured
        k.copy_(randn(rng, 2, H, D))
        v.copy_(randn(rng, 2, H, D))
        g.replay()
        torch.cuda.synchronize()
        now = [f + step for f in first]
        pair.ref.append(k.cpu().numpy(), v.cpu().numpy(), table, now, [0, 1, 2])
        if step % 6 == 0 or step < 4:
            check(pair, q, table, now, None, out)
    assert np.array_equal(pair.dev.page_tensor.cpu().numpy(), pair.ref.pages)


def test_a_captured_layer_on_a_table_for_long_contexts(lib):
    # as tests/test_decode_layer_gpu.py, in a table whose width rules the clusters out
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)

    def layer():
        x = example.Layer(hidden=512, heads=4, kv_heads=2, head_dim=64, experts=8, top_k=2, ffn=256, seqs=3, page=16,
                          pages_per_seq=3000, select=200, seed=1)
        g = torch.Generator().manual_seed(1)
        x.prompt(torch.randn(938, 512, generator=g).cuda(), dev32([0, 900, 901, 938]))
        return x, torch.randn(3, 512, generator=g).cuda(), torch.randn(3, 512, generator=g).cuda()

    (a, x, r), (b, _, _) = layer(), layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gx, gr = a.step(x, r)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gy, gh = a.step(gx, gr)
        side.synchronize()
        y, h = b.step(x, r)
        for _ in range(20):
            graph.replay()
            y, h = b.step(y, h)
            assert torch.equal(gy, y) and torch.equal(gh, h)
            gx.copy_(gy), gr.copy_(gh)
        side.synchronize()
    assert torch.equal(a.lens, b.lens) and api.get_device_error() == 0
