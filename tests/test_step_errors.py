"""Host-side argument checking of the rotation, adapter, expert selection and log
probability entry points: every call here is refused before a device is touched."""
import ctypes

import pytest
import torch

from moe_matvec_gb300 import api

A, MIS = 0x10000, 0x10004  # an aligned and a misaligned address, never dereferenced
R = ctypes.byref
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return api.load()


def test_norm_rope(L):
    def call(D=128, R_=128, axes=1, rscale=1.0, freq=A, axis=None, dt=0, q=A, qs=512, qo=2 * A, qos=512, H=4, qw=A, k=A, ks=128,
             ko=2 * A, kos=128, Hk=1, kw=A, eps=1e-6, pos=None, lens=A, starts=None, n_seq=3, n=3, rope=True):
        r = api.Rope(D, R_, 0, axes, rscale, 0, freq, axis)
        return L.qmv_norm_rope(R(r) if rope else None, dt, q, qs, qo, qos, H, qw, k, ks, ko, kos, Hk, kw, eps, pos, lens,
                               starts, n_seq, n, None)

    assert call(rope=False) == -4
    assert call(dt=3) == -1 and call(dt=-1) == -1
    assert call(D=0) == -2 and call(D=127) == -2 and call(D=258, qs=2000, qos=2000) == -2 and call(R_=0) == -2
    assert call(R_=130) == -2 and call(R_=63) == -2 and call(axes=0) == -2 and call(axes=5) == -2
    assert call(rscale=NAN) == -2 and call(eps=-1.0) == -2 and call(eps=NAN) == -2 and call(eps=INF) == -2
    assert call(n=0) == -3 and call(n=65536) == -3
    assert call(freq=None) == -4 and call(freq=MIS) == -5 and call(axis=MIS) == -5
    for x, s, o, os, h in (("q", "qs", "qo", "qos", "H"), ("k", "ks", "ko", "kos", "Hk")):
        assert call(**{h: 16385}) == -2 and call(**{x: None}) == -4 and call(**{o: None}) == -4
        assert call(**{s: 100}) == -2 and call(**{os: 100}) == -2
        assert call(**{x: MIS}) == -5 and call(**{o: MIS}) == -5 and call(**{s: 1001}) == -5 and call(**{os: 1001}) == -5
        assert call(**{s: 1024, o: A}) == -2                # in place with two strides
    assert call(H=0) == -2 and call(Hk=0) == -2             # keys without heads
    assert call(k=None, ko=None, Hk=2) == -4
    assert call(qw=MIS) == -5 and call(kw=MIS) == -5
    assert call(lens=None) == -4 and call(pos=A) == -2 and call(pos=MIS, lens=None) == -5 and call(lens=MIS) == -5
    assert call(starts=MIS) == -5 and call(n_seq=2) == -3   # one token a sequence
    assert call(starts=A, n_seq=0) == -2 and call(starts=A, n_seq=1025) == -2
    assert call(dt=1, qs=516, qo=A + 64) == -5              # 16-bit tokens not 16-byte aligned


def test_lora(L):
    def pool(n=3, r=8, dt=2, a=A, b=A, ranks=None, scales=None):
        return api.Lora(n, r, dt, 0, a, b, ranks, scales)

    def call(l=None, ids=A, x=A, res=A, y=A, K=64, M=100, n=4, ws=A, wsb=1 << 20):
        return L.qmv_lora_run(R(l if l is not None else pool()), ids, x, res, y, K, M, n, ws, wsb, None)

    assert L.qmv_lora_run(None, A, A, A, A, 64, 100, 4, A, 1 << 20, None) == -4
    assert call(pool(dt=3)) == -1
    assert call(pool(n=0)) == -2 and call(pool(n=(1 << 20) + 1)) == -2
    for r in (0, 2, 6, 132):
        assert call(pool(r=r)) == -2
    assert call(K=0) == -2 and call(K=60) == -2 and call(K=(1 << 20) + 8) == -2 and call(M=0) == -2
    assert call(M=(1 << 30) + 1) == -2
    assert call(n=0) == -3 and call(n=65) == -3
    for name in ("ids", "x", "res", "y", "ws"):
        assert call(**{name: None}) == -4 and call(**{name: MIS}) == -5
    assert call(pool(a=None)) == -4 and call(pool(b=None)) == -4 and call(pool(a=MIS)) == -5 and call(pool(b=MIS)) == -5
    assert call(pool(ranks=MIS)) == -5 and call(pool(scales=MIS)) == -5
    # y over x (256 * 4 bytes), or over a part of res (400 * 4 bytes)
    assert call() == -2 and call(x=A + 1584) == -2 and call(x=A - 1008) == -2
    assert call(x=4 * A, y=A + 16) == -2 and call(x=4 * A, res=A + 1584) == -2
    need = L.qmv_lora_workspace_bytes(R(pool()), 64, 4)
    assert need == 4 * 8 * 4 and call(wsb=need - 1) == -6
    assert L.qmv_lora_workspace_bytes(R(pool(r=6)), 64, 4) == 0 and L.qmv_lora_workspace_bytes(None, 64, 4) == 0


def test_route_select(L):
    def call(dt=0, logits=A, ld=64, bias=A, E=64, n=4, k=8, gating=1, groups=8, keep=4, top=2, scale=1.0, ids=A, gates=A):
        return L.moe_route_select(dt, logits, ld, bias, E, n, k, gating, groups, keep, top, 1, scale, ids, gates, None)

    assert call(dt=9) == -1
    assert call(E=0) == -2 and call(E=520, ld=520) == -2 and call(groups=0) == -2 and call(groups=7) == -2
    assert call(groups=64, keep=8, top=1) == -2 and call(keep=0) == -2 and call(keep=9) == -2
    assert call(top=0) == -2 and call(top=3) == -2 and call(E=8, ld=8, top=2, k=1) == -2 and call(ld=63) == -2
    assert call(gating=2) == -2 and call(gating=-1) == -2 and call(scale=NAN) == -2 and call(scale=INF) == -2
    assert call(k=0) == -3 and call(k=9) == -3 and call(n=0) == -3 and call(n=16385) == -3
    assert call(E=8, ld=8, keep=4, top=1, k=5) == -2
    assert call(logits=None) == -4 and call(ids=None) == -4 and call(gates=None) == -4
    assert call(logits=MIS) == -5 and call(bias=MIS) == -5 and call(ids=MIS) == -5 and call(gates=MIS) == -5


def test_logprobs(L):
    def call(dt=0, logits=A, ld=100, rows=2, V=100, scale=1.0, tokens=A, given=1, logp=A, lse=A, entropy=A, n_top=2, ids=A,
             top=A):
        return L.qmv_logprobs(dt, logits, ld, rows, V, scale, tokens, given, logp, lse, entropy, n_top, ids, top, None)

    assert call(dt=3) == -1
    assert call(rows=0) == -2 and call(rows=(1 << 24) + 1) == -2 and call(V=0) == -2 and call(ld=99) == -2
    assert call(V=(1 << 28) + 1, ld=1 << 29) == -2
    assert call(given=-1) == -2 and call(given=65) == -2 and call(n_top=-1) == -2 and call(n_top=33) == -2
    for s in (0.0, -1.0, NAN, INF, 1e38, 1e-38):
        assert call(scale=s) == -2
    assert call(logits=None) == -4 and call(tokens=None) == -4 and call(logp=None) == -4
    assert call(ids=None) == -4 and call(top=None) == -4
    assert call(given=0, n_top=0, lse=None, entropy=None) == -4
    for name in ("tokens", "logp", "lse", "entropy", "ids", "top"):
        assert call(**{name: MIS}) == -5
    assert call(logits=A + 2) == -5 and call(logits=A + 1, dt=1) == -5  # their type's alignment is enough


def test_binding_refuses_mismatched_tensors():
    f = torch.ones(32)
    with pytest.raises(ValueError):
        api.rope(64, f)                                     # not on a device
    with pytest.raises(ValueError):
        api.rope(64, f.double())
    with pytest.raises(ValueError):
        api.rope(64, f, axis=torch.zeros(32))
    with pytest.raises(ValueError):
        api.lora(torch.zeros(2, 8, 64), torch.zeros(2, 10, 4))
    with pytest.raises(ValueError):
        api.lora(torch.zeros(2, 8, 64), torch.zeros(2, 10, 8).half())
    with pytest.raises(ValueError):
        api.lora(torch.zeros(2, 8, 64), torch.zeros(2, 10, 8), ranks=torch.zeros(2))
    r = api.Rope(64, 64, 0, 1, 1.0, 0, A, None)
    x = torch.zeros(3, 4, 64)
    with pytest.raises(ValueError):
        api.norm_rope(r, x, lens=torch.ones(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        api.route_select(torch.zeros(3, 64), 4)
    with pytest.raises(ValueError):
        api.route_select(torch.zeros(3, 64, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        api.logprobs(torch.zeros(3, 64))
    d = api.Lora(2, 8, 2, 0, A, A, None, None)
    d.K, d.M = 64, 10
    with pytest.raises(ValueError):
        api.lora_run(d, torch.zeros(3, dtype=torch.int32), torch.zeros(3, 63), torch.zeros(3, 10))
    with pytest.raises(ValueError):
        api.lora_run(d, torch.zeros(3, dtype=torch.int32), torch.zeros(3, 64), torch.zeros(3, 10))
    with pytest.raises(TypeError):
        api.logprobs(None)
    assert api.lora_workspace_bytes(d, 3) == 3 * 8 * 4
