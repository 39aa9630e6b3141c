"""lens and starts that contradict the call's sizes or each other: attention,
selection and read-back stay inside their buffers (guard bands, and no failed
check in the range-checked build, which goes first), flag what they use of them,
and the next call is right again.  (Append's bytes: tests/test_kv_cache_gpu.py.)"""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests.test_canary_gpu import Guarded
from tests.test_kv_attend_gpu import check, filled, wide
from tests.test_kv_cache_gpu import dev32, randn

pytestmark = pytest.mark.gpu

LENS, STARTS, N = [150, 40, 5], [0, 5, 7, 8], 8
BIG = 2 ** 31 - 1
BAD = {
    "longer than the table": ([10 ** 9, 40, BIG], STARTS),
    "negative lengths": ([-1, -BIG - 1, 5], STARTS),
    "past the tokens": (LENS, [0, 5, 9, 9]),
    "far past the tokens": (LENS, [0, BIG, BIG, BIG]),
    "negative starts": (LENS, [-5, 3, 6, 8]),
    "the most negative starts": (LENS, [-BIG - 1, -BIG - 1, 2, 8]),
    "descending": (LENS, [8, 5, 2, 0]),
    "the same tokens twice": (LENS, [0, 8, 0, 8]),
}


@pytest.fixture(scope="module")
def dbg(lib):
    return api.load_debug()


@pytest.mark.parametrize("what", list(BAD))
@pytest.mark.parametrize("D,P,G,dtype", [(64, 16, 3, torch.float32), (128, 64, 12, torch.bfloat16), (256, 32, 2, torch.float32)])
def test_contradictions_stay_inside(lib, dbg, what, D, P, G, dtype):
    rng = np.random.default_rng(D)
    pair, table = filled(rng, 2, D, P, LENS)
    lens, starts = (dev32(x) for x in BAD[what])
    q = randn(rng, N, 2 * G, D, dtype=dtype)
    allowed = api.DEVERR_BATCH | api.DEVERR_PAGE  # (a clamped length reaches entries of the table that are no page)
    for build in (dbg, api.load()):
        with api.using(build):
            for t in (table, wide(table, P)):
                td = dev32(t)
                for causal, window in ((True, 0), (False, 0), (True, 30)):
                    out, ws = Guarded(q.shape, dtype, 1), Guarded((api.kv_attend_workspace_bytes(pair.dev, 2 * G, N, 3),), torch.uint8, 2)
                    api.kv_attend(pair.dev, q, td, lens, starts, causal=causal, window=window, ws=ws.t, out=out.t)
                    err = api.get_device_error()
                    assert err & ~allowed == 0
                    if t is not table:  # equal shares look at every sequence
                        assert err & api.DEVERR_BATCH
                    out.check_guards("out"), ws.check_guards("ws")
                ids, ws = Guarded((N, 2, 3), torch.int32, 3), Guarded((api.kv_select_workspace_bytes(pair.dev, N, t.shape[1]),), torch.uint8, 4)
                ids.t.fill_(1)
                api.kv_select(pair.dev, q, td, lens, 3, starts, ws=ws.t, ids=ids.t)
                assert api.get_device_error() & ~allowed == 0
                ids.check_guards("ids"), ws.check_guards("ws of selection")
                out, ws = Guarded(q.shape, dtype, 5), Guarded((api.kv_attend_workspace_bytes(pair.dev, 2 * G, N, 3),), torch.uint8, 6)
                api.kv_attend(pair.dev, q, td, lens, starts, pages=ids.t, ws=ws.t, out=out.t)
                assert api.get_device_error() & ~allowed == 0
                out.check_guards("out of pages"), ws.check_guards("ws of pages")
                k, v = Guarded((N, 2, D), dtype, 7), Guarded((N, 2, D), dtype, 8)
                api.kv_read(pair.dev, td, lens, starts, N, k=k.t, v=v.t)
                assert api.get_device_error() & ~allowed == 0
                k.check_guards("k"), v.check_guards("v")
                good = api.kv_attend(pair.dev, q, td, dev32(LENS), dev32(STARTS))
                check(pair, q, table, LENS, STARTS, good)


def test_what_append_flags(lib):
    rng = np.random.default_rng(1)
    c = api.kv_cache(1, 64, 16, 8)
    k = randn(rng, 4, 1, 64)

    def call(lens, starts):
        api.kv_append(c, k, k, dev32([[0, 1], [2, 3]]), dev32(lens), dev32(starts))
        return api.get_device_error()

    assert call([4, 4], [3, 1, 2]) == api.DEVERR_BATCH      # descending
    assert call([4, 4], [0, 2, 5]) == api.DEVERR_BATCH      # past n_tok
    assert call([4, 1], [0, 2, 4]) == api.DEVERR_BATCH      # two tokens of one
    assert call([4, 0], [0, 2, 4]) == 0                     # an empty slot
    assert call([4, 4], [1, 2, 3]) == 0                     # padding at both ends


def test_more_new_tokens_than_the_sequence_holds(lib):
    # three of four tokens lie before the sequence's first: zeros (flagged by the read-back), no picks, nothing seen
    rng = np.random.default_rng(2)
    lens, starts = [1, 33], [0, 4, 6]
    pair, table = filled(rng, 2, 64, 16, lens)
    q = randn(rng, 6, 4, 64)
    args = dev32(lens), dev32(starts)
    for t in (table, wide(table, 16)):
        out = api.kv_attend(pair.dev, q, dev32(t), *args)
        ids = api.kv_select(pair.dev, q, dev32(t), args[0], 2, args[1])
        assert api.get_device_error() == 0
        assert (out[:3] == 0).all() and (ids[:3] == -1).all()
        check(pair, q, table, lens, starts, out)
        k, v = api.kv_read(pair.dev, dev32(t), *args, 6)
        assert api.get_device_error() == api.DEVERR_BATCH
        assert (k[:3] == 0).all() and (v[:3] == 0).all()


def test_padding_at_both_ends_is_left_alone(lib):
    rng = np.random.default_rng(3)
    lens, starts = [90, 20], [1, 4, 5]
    pair, table = filled(rng, 2, 64, 16, lens)
    q = randn(rng, 7, 4, 64)
    for t in (table, wide(table, 16)):
        td, args = dev32(t), (dev32(lens), dev32(starts))
        out, k, v = torch.full_like(q, 7), *(torch.full((7, 2, 64), 7.0, device="cuda") for _ in range(2))
        ids = torch.full((7, 2, 3), 7, dtype=torch.int32, device="cuda")
        api.kv_attend(pair.dev, q, td, *args, out=out)
        api.kv_select(pair.dev, q, td, args[0], 3, args[1], ids=ids)
        api.kv_read(pair.dev, td, *args, 7, k=k, v=v)
        assert api.get_device_error() == 0
        for x in (out, ids, k, v):
            assert (x[[0, 5, 6]] == 7).all()
        check(pair, q[1:5], table, lens, [0, 3, 4], out[1:5])
