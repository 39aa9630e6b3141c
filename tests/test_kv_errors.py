"""Host-side argument checking of the norm, cache, attention and selection
entry points: every call here is refused before a device is touched."""
import ctypes

import pytest
import torch

from moe_matvec_gb300 import api

A, MIS = 0x10000, 0x10004  # an aligned and a misaligned address, never dereferenced
R = ctypes.byref


@pytest.fixture(scope="module")
def L():
    return api.load()


def cache(H=8, D=128, P=64, n=10, pages=A, bounds=A):
    return api.KvCache(H, D, P, n, pages, bounds)


def batch(table=A, lens=A, starts=None, n_seq=4, max_pages=16, n_tok=4):
    return api.KvBatch(table, lens, starts, n_seq, max_pages, n_tok, 0)


def test_norm_rejects_bad_arguments(L):
    def norm(dt=0, x=A, ldx=512, r=None, w=A, eps=1e-6, rows=2, K=512, res=None, y=A, q=None, d=None, s=None):
        return L.qmv_rms_norm(dt, x, ldx, r, w, eps, rows, K, res, y, q, d, s, None)

    assert norm(dt=3) == -1 and norm(dt=-1) == -1
    assert norm(K=0) == -2 and norm(K=32769, ldx=40000) == -2 and norm(ldx=511) == -2 and norm(rows=0) == -2
    assert norm(eps=-1.0) == -2 and norm(eps=float("nan")) == -2 and norm(eps=float("inf")) == -2
    assert norm(K=500, q=A, d=A, s=A) == -2                                  # Q8 output needs K % 256
    assert norm(x=None) == -4 and norm(w=None) == -4 and norm(y=None) == -4  # nothing wanted
    assert norm(q=A, d=A) == -4 and norm(d=A) == -4
    assert norm(x=MIS) == -5 and norm(r=MIS) == -5 and norm(res=MIS) == -5 and norm(q=MIS, d=A, s=A) == -5
    assert norm(ldx=513, q=A, d=A, s=A) == -5                                # rows not 16-byte aligned
    assert L.qmv_dequantize_act(4, A, A, 1, 256, A, None) == -1
    assert L.qmv_dequantize_act(0, A, A, 1, 100, A, None) == -2
    assert L.qmv_dequantize_act(0, A, None, 1, 256, A, None) == -4
    assert L.qmv_dequantize_act(0, A, A, 1, 256, MIS, None) == -5


def test_cache_shapes(L):
    assert L.qmv_kv_page_bytes(128, 64) == 16 + 2 * 64 * 128 and L.qmv_kv_bounds_bytes(192) == 16 + 384
    for D, P in ((96, 64), (0, 64), (512, 64), (128, 8), (128, 128), (128, 0)):
        assert L.qmv_kv_page_bytes(D, P) == -2
    assert L.qmv_kv_bounds_bytes(100) == -2
    assert L.qmv_kv_attend_workspace_bytes(R(cache()), 12, 4, 4) == 0              # 12 heads on 8
    assert L.qmv_kv_attend_workspace_bytes(R(cache()), 32, 4, 4) > 0
    assert L.qmv_kv_select_workspace_bytes(R(cache()), R(batch())) == 4 * 8 * 16 * 4


CALLS = {
    "append": lambda L, c, b, dt=0, x=A, st=1024: L.qmv_kv_append(c, b, dt, x, st, A, 1024, None),
    "append_v": lambda L, c, b, dt=0, x=A, st=1024: L.qmv_kv_append(c, b, dt, A, 1024, x, st, None),
    "attend": lambda L, c, b, dt=0, x=A, st=4096: L.qmv_kv_attend(c, b, dt, x, st, A, 32, 0.1, 1, 0, None, 0, A, 1 << 30,
                                                                 None),
    "select": lambda L, c, b, dt=0, x=A, st=4096: L.qmv_kv_select(c, b, dt, x, st, 32, A, 4, A, 1 << 30, None),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_batched_calls_reject_bad_arguments(L, name):
    call = CALLS[name]
    assert call(L, R(cache()), R(batch()), dt=7) == -1
    assert call(L, R(cache(D=96)), R(batch())) == -2 and call(L, R(cache(P=48)), R(batch())) == -2
    assert call(L, R(cache(H=0)), R(batch())) == -2 and call(L, R(cache(n=0)), R(batch())) == -2
    assert call(L, R(cache()), R(batch(n_seq=0))) == -2 and call(L, R(cache()), R(batch(n_seq=1025, n_tok=1025))) == -2
    assert call(L, R(cache()), R(batch(max_pages=0))) == -2 and call(L, R(cache()), R(batch(max_pages=(1 << 20) + 1))) == -2
    assert call(L, R(cache()), R(batch(n_tok=0))) == -3 and call(L, R(cache()), R(batch(n_tok=5))) == -3
    assert call(L, R(cache()), R(batch(starts=A, n_tok=65536))) == -3
    assert call(L, None, R(batch())) == -4 and call(L, R(cache()), None) == -4
    assert call(L, R(cache(pages=None)), R(batch())) == -4
    assert call(L, R(cache()), R(batch(table=None))) == -4 and call(L, R(cache()), R(batch(lens=None))) == -4
    assert call(L, R(cache()), R(batch()), x=None) == -4
    assert call(L, R(cache(pages=MIS)), R(batch())) == -5 and call(L, R(cache(bounds=MIS)), R(batch())) == -5
    assert call(L, R(cache()), R(batch(lens=MIS))) == -5 and call(L, R(cache()), R(batch(starts=MIS))) == -5
    assert call(L, R(cache()), R(batch()), x=MIS) == -5
    assert call(L, R(cache()), R(batch()), st=1000) == -2                    # tokens overlap
    assert call(L, R(cache()), R(batch()), st=4097) == -5                    # tokens not 16-byte aligned


def test_attend_and_select_reject_bad_arguments(L):
    def attend(heads=32, scale=0.1, window=0, pages=None, n_sel=0, out=A, ws=A, wsb=1 << 30):
        return L.qmv_kv_attend(R(cache()), R(batch()), 0, A, 1 << 20, out, heads, scale, 1, window, pages, n_sel, ws, wsb,
                               None)

    assert attend(heads=0) == -2 and attend(heads=12) == -2 and attend(heads=32768) == -2
    assert attend(scale=float("nan")) == -2 and attend(scale=float("inf")) == -2 and attend(window=-1) == -2
    assert attend(pages=A, n_sel=0) == -2
    assert attend(out=None) == -4 and attend(ws=None) == -4
    assert attend(out=MIS) == -5 and attend(ws=MIS) == -5 and attend(pages=MIS, n_sel=4) == -5
    need = L.qmv_kv_attend_workspace_bytes(R(cache()), 32, 4, 4)
    assert attend(wsb=need - 1) == -6

    def select(c=None, heads=32, n_sel=4, ids=A, ws=A, wsb=1 << 30):
        return L.qmv_kv_select(R(c or cache()), R(batch()), 0, A, 1 << 21, heads, ids, n_sel, ws, wsb, None)

    assert select(heads=9) == -2 and select(n_sel=0) == -2 and select(heads=8 * 257) == -2
    assert select(c=cache(bounds=None)) == -4 and select(ids=None) == -4 and select(ws=None) == -4
    assert select(ids=MIS) == -5
    assert select(wsb=4 * 8 * 16 * 4 - 1) == -6
    assert L.qmv_kv_read(R(cache()), R(batch()), 0, None, A, None) == -4
    assert L.qmv_kv_read(R(cache()), R(batch()), 9, A, A, None) == -1


def test_binding_refuses_mismatched_tensors():
    x = torch.zeros(2, 512)
    with pytest.raises(ValueError):
        api.rms_norm(x.to(torch.int32), torch.zeros(512))
    with pytest.raises(ValueError):
        api.rms_norm(x, torch.zeros(512))                # not on a device
    with pytest.raises(ValueError):
        api.rms_norm(x, torch.zeros(512), want="int8")
    c = cache()
    t, lens = torch.zeros(4, 16, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.kv_append(c, torch.zeros(4, 7, 128), torch.zeros(4, 7, 128), t, lens)
    with pytest.raises(ValueError):
        api.kv_attend(c, torch.zeros(4, 32, 64), t, lens)
    with pytest.raises(ValueError):
        api.kv_read(c, t, lens, lens)                    # n_tok missing
    with pytest.raises(api.QmvError):
        api.kv_page_bytes(100, 64)
    with pytest.raises(api.QmvError):
        api.kv_cache(0, 128, 64, 4)
