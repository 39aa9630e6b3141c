"""Memory bounds of the norm, cache, attention and selection kernels, without a
device memory checker: guard bands around every result, workspace and cache
(as tests/test_canary_gpu.py), and the range-checked build of the library
(as tests/test_debug_gpu.py): the same bits, no failed check, and checks that
are shown to be live."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests.test_canary_gpu import Guarded
from tests.test_debug_gpu import both, same_bits
from tests.test_kv_cache_gpu import dev32, randn, tables

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def dbg(lib):
    return api.load_debug()


# ------------------------------------------------------------ guard bands
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,K", [(1, 1), (1, 256), (3, 512), (5, 33), (70, 256), (2, 5120), (700, 2304), (1, 8193), (2, 32768)])
def test_norm_stays_in_its_buffers(lib, dtype, n, K):
    rng = np.random.default_rng(n + K)
    x, r, w = randn(rng, n, K, dtype=dtype), randn(rng, n, K, dtype=dtype), randn(rng, K)
    q8 = K % 256 == 0
    want = api.rms_norm(x, w, r=r, want="both" if q8 else "float")
    y, res = Guarded((n, K), dtype, 1), Guarded((n, K), dtype, 2)
    gs = [Guarded((n, K), torch.int8, 3), Guarded((n, K // 32), torch.float32, 4), Guarded((n, K // 32), torch.int32, 5)] \
        if q8 else []
    keep = [t.clone() for t in (x, r, w)]
    got = api.rms_norm(x, w, r=r, want="both" if q8 else "float", y=y.t, res=res.t, q8=tuple(g.t for g in gs) or None)
    for g in [y, res] + gs:
        g.check_guards("rms_norm")
    assert same_bits(got[0], want[0]) and same_bits(got[2], want[2])
    assert all(same_bits(a, b) for a, b in zip(keep, (x, r, w)))
    if q8:
        assert all(same_bits(a, b) for a, b in zip(got[1], want[1]))
        back = Guarded((n, K), dtype, 6)
        api.dequantize_act(gs[0].t, gs[1].t, out=back.t)
        back.check_guards("dequantize_act")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P,H,G", [(64, 16, 1, 1), (128, 64, 3, 5), (192, 32, 2, 9), (256, 16, 2, 3), (128, 16, 1, 20)])
def test_cache_calls_stay_in_their_buffers(lib, dtype, D, P, H, G):
    rng = np.random.default_rng(D + P)
    lens = [P + 3, 1, 5 * P, 2 * P - 1]
    news = [P + 3, 1, 2, P]
    st = np.concatenate([[0], np.cumsum(news)])
    first = [t - c for t, c in zip(lens, news)]
    n_pages = sum(-(-t // P) for t in lens)  # every page of the pool is used
    table = tables(rng, lens, P, n_pages)
    pages = Guarded((n_pages, H, 16 + 2 * P * D), torch.uint8, 7)
    bounds = Guarded((n_pages, H, 16 + 2 * D), torch.uint8, 8)
    c = api.kv_cache(H, D, P, n_pages, pages=pages.t, bounds=bounds.t)
    args = dev32(table), dev32(lens)
    f0 = np.concatenate([[0], np.cumsum(first)])
    k0, v0 = randn(rng, f0[-1], H, D, dtype=dtype), randn(rng, f0[-1], H, D, dtype=dtype)
    api.kv_append(c, k0, v0, dev32(table), dev32(first), dev32(f0))
    k, v = randn(rng, st[-1], H, D, dtype=dtype), randn(rng, st[-1], H, D, dtype=dtype, scale=2)
    api.kv_append(c, k, v, *args, dev32(st))
    api.kv_append(c, k[:4].contiguous(), v[:4].contiguous(), *args)  # the last tokens again, one a sequence
    q = randn(rng, st[-1], H * G, D, dtype=dtype)
    want = api.kv_attend(c, q, *args, dev32(st)), api.kv_select(c, q, *args, 3, dev32(st)), api.kv_read(c, *args, dev32(st), int(st[-1]), dtype)
    n = int(st[-1])
    out, ids = Guarded((n, H * G, D), dtype, 9), Guarded((n, H, 3), torch.int32, 10)
    ws = Guarded((api.kv_attend_workspace_bytes(c, H * G, n, 4),), torch.uint8, 11)
    ws2 = Guarded((api.kv_select_workspace_bytes(c, n, table.shape[1]),), torch.uint8, 12)
    ko, vo = Guarded((n, H, D), dtype, 13), Guarded((n, H, D), dtype, 14)
    api.kv_attend(c, q, *args, dev32(st), ws=ws.t, out=out.t)
    api.kv_select(c, q, *args, 3, dev32(st), ws=ws2.t, ids=ids.t)
    api.kv_read(c, *args, dev32(st), n, k=ko.t, v=vo.t)
    for g, what in ((pages, "pages"), (bounds, "bounds"), (out, "out"), (ids, "ids"), (ws, "ws"), (ws2, "ws2"), (ko, "k"), (vo, "v")):
        g.check_guards(what)
    assert same_bits(out.t, want[0]) and same_bits(ids.t, want[1]) and same_bits(ko.t, want[2][0]) and same_bits(vo.t, want[2][1])
    sel = Guarded((n, H * G, D), dtype, 15)
    ws3 = Guarded((api.kv_attend_workspace_bytes(c, H * G, n, 4),), torch.uint8, 16)
    api.kv_attend(c, q, *args, dev32(st), pages=ids.t, ws=ws3.t, out=sel.t)
    sel.check_guards("out of selected pages")
    ws3.check_guards("ws of selected pages")
    assert api.get_device_error() == 0


# ------------------------------------------------------ range-checked build
def state(D=128, P=16, H=2, dtype=torch.float32, seed=0):
    rng = np.random.default_rng(seed)
    lens = [70, 1, 33, 16]
    table = tables(rng, lens, P, 20)
    c = api.kv_cache(H, D, P, 20, pages=torch.full((20, H, 16 + 2 * P * D), 0xFF, dtype=torch.uint8, device="cuda"),
                     bounds=torch.full((20, H, 16 + 2 * D), 0xFF, dtype=torch.uint8, device="cuda"))
    st = np.concatenate([[0], np.cumsum(lens)])
    k, v = randn(rng, st[-1], H, D, dtype=dtype), randn(rng, st[-1], H, D, dtype=dtype)
    return c, dev32(table), dev32(lens), dev32(st), k, v, randn(rng, 4, 6 * H, D, dtype=dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (192, 32), (256, 64)])
def test_range_checked_build_gives_the_same_bits(dbg, dtype, D, P):
    c, table, lens, st, k, v, q = state(D, P, dtype=dtype)

    def run():
        c.page_tensor.fill_(0xFF)
        c.bounds_tensor.fill_(0xFF)
        api.kv_append(c, k, v, table, lens, st)
        api.kv_append(c, k[:4].contiguous() * 2, v[:4].contiguous(), table, lens)
        ids = api.kv_select(c, q, table, lens, 2)
        many = api.kv_attend(c, k.repeat(1, 3, 1)[:, :2 * c.n_kv_heads].contiguous(), table, lens, st)
        return [c.page_tensor.clone(), c.bounds_tensor.clone(), ids, api.kv_attend(c, q, table, lens), many,
                api.kv_attend(c, q, table, lens, pages=ids), *api.kv_read(c, table, lens, st, int(st[-1]), dtype)]

    rel, d, err = both(dbg, run)
    assert err == 0
    assert all(same_bits(a, b) for a, b in zip(rel, d))


@pytest.mark.parametrize("dtype", DT)
def test_range_checked_norm(dbg, dtype):
    rng = np.random.default_rng(3)
    for n, K in ((1, 7), (3, 256), (300, 512), (2, 8448)):
        x, w = randn(rng, n, K, dtype=dtype), randn(rng, K)
        rel, d, err = both(dbg, lambda: [t for t in api.rms_norm(x, w, r=x, want="float")[::2]])
        assert err == 0 and all(same_bits(a, b) for a, b in zip(rel, d))
        if K % 256 == 0:
            rel, d, err = both(dbg, lambda: list(api.rms_norm(x, w, want="q8")[1]))
            assert err == 0 and all(same_bits(a, b) for a, b in zip(rel, d))


def test_the_checks_are_live(dbg):
    # results' extents handed to the checks eight elements short: those stores
    # are skipped and flagged, the others made; the next call is clean again
    c, table, lens, st, k, v, q = state()
    api.kv_append(c, k, v, table, lens, st)
    x, w = randn(np.random.default_rng(4), 3, 512), torch.ones(512, device="cuda")
    n = int(st[-1])
    calls = {
        "norm": lambda o: api.rms_norm(x, w, y=o), "attend": lambda o: api.kv_attend(c, q, table, lens, out=o),
        "select": lambda o: api.kv_select(c, q, table, lens, 5, ids=o),
        "read": lambda o: api.kv_read(c, table, lens, st, n, k=o, v=torch.empty_like(o)),
    }
    shapes = {"norm": (3, 512), "attend": tuple(q.shape), "select": (4, 2, 5), "read": (n, 2, 128)}
    for name, call in calls.items():
        dt = torch.int32 if name == "select" else torch.float32
        want = torch.full(shapes[name], 7, dtype=dt, device="cuda")
        call(want)
        got = torch.full(shapes[name], 7, dtype=dt, device="cuda")
        with api.using(dbg):
            api.get_device_error()
            api.debug_shrink_outputs(8)
            try:
                call(got)
            finally:
                err = api.get_device_error()
                api.debug_shrink_outputs(0)
            assert err == api.DEVERR_RANGE, name
            flat, ref = got.flatten(), want.flatten()
            assert torch.equal(flat[:-16], ref[:-16]) and (flat[-8:] == 7).all(), name
            call(got)
            assert api.get_device_error() == 0 and torch.equal(got, want), name
