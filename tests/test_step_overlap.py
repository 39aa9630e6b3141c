"""Results of the rotation and the adapters that overlap what other warps still read
are refused; results among the rows of one buffer that lie apart are not."""
import ctypes
import random

import pytest
import torch

from moe_matvec_gb300 import api

A = 0x100000  # an address, never dereferenced: what is refused reaches no device
SHAPE = -2
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass every check")


@pytest.fixture(scope="module")
def L():
    return api.load()


def norm_rope(L, n, q, qs, H, qo, qos, k=None, ks=0, Hk=0, ko=None, kos=0, dt=0, D=8):
    """Addresses in units of 16 bytes, strides likewise."""
    e = 4 if dt == 0 else 2
    at = lambda a: None if a is None else A + 16 * a  # noqa: E731
    r = api.Rope(D, D, 0, 1, 1.0, 0, A, None)
    return L.qmv_norm_rope(ctypes.byref(r), dt, at(q), qs * 16 // e, at(qo), qos * 16 // e, H, None, at(k), ks * 16 // e, at(ko),
                           kos * 16 // e, Hk, None, 1e-6, A, None, None, 0, n, None)


def test_overlapping_results_of_the_rotation(L):
    # heads of 8 fp32 (2 units); tokens of 6 q heads, 2 k heads, 2 v heads: 20 units
    fused = dict(q=0, qs=20, H=6, k=12, ks=20, Hk=2)
    for n in (1, 2, 5):
        assert norm_rope(L, n, 0, 20, 6, 2, 20) == SHAPE                         # a head on
        assert norm_rope(L, n, 2, 20, 6, 0, 20) == SHAPE                         # a head back
        assert norm_rope(L, n, 0, 20, 6, 11, 20) == SHAPE                        # the last 16 bytes
        assert norm_rope(L, n, qo=0, qos=20, ko=0, kos=20, **fused) == SHAPE     # both results in one place
        assert norm_rope(L, n, qo=100 * n, qos=20, ko=100 * n + 10, kos=20, **fused) == SHAPE
        assert norm_rope(L, n, qo=0, qos=20, ko=10, kos=20, **fused) == SHAPE    # keys moved on to a part of q
        assert norm_rope(L, n, qo=4, qos=20, ko=500, kos=20, **fused) == SHAPE   # queries over the keys
        # one input, in place for one of two results
        assert norm_rope(L, n, 0, 20, 2, 0, 20, 0, 20, 2, 500, 20) == SHAPE
    for n in (2, 5):
        assert norm_rope(L, n, 0, 12, 6, 12, 12) == SHAPE                        # a token on
        assert norm_rope(L, n, 12, 12, 6, 0, 12) == SHAPE
        assert norm_rope(L, n, 0, 20, 6, 10, 20) == SHAPE                        # round into the next token
        assert norm_rope(L, n, 0, 20, 6, 12, 12) == SHAPE                        # another stride
        assert norm_rope(L, n, qo=0, qos=20, ko=14, kos=16, **fused) == SHAPE    # keys closed up within the buffer


def rows(at, step, length, n):
    return [(at + i * step, at + i * step + length) for i in range(n)]


def meet(a, b):
    return any(x0 < y1 and y0 < x1 for x0, x1 in a for y0, y1 in b)


@no_device
def test_what_is_refused_is_what_overlaps(L):
    rng = random.Random(3)
    got = {True: 0, False: 0}
    for _ in range(20000):
        n, H, Hk, D = rng.choice([1, 2, 3, 7]), rng.randint(1, 3), rng.randint(0, 2), 8
        dt = rng.choice([0, 1])
        head = 2 if dt == 0 else 1
        s = [rng.choice([0, 0, rng.randint(0, 9)]) for _ in range(4)]
        base = rng.choice([0, head * (H + Hk)])
        qs, qos = (max(head * H, base) + x for x in s[:2])
        ks, kos = (max(head * Hk, base) + x for x in s[2:])
        place = lambda: rng.randint(0, rng.choice([12, 60]))  # noqa: E731
        q, k, ko = place(), place(), place()
        qo = q if rng.random() < 0.3 else place()
        if rng.random() < 0.3:
            ko = k
        if (q == qo and qs != qos and n > 1) or (Hk and k == ko and ks != kos and n > 1):
            continue  # refused for that
        Q, QO = rows(q, qs, head * H, n), rows(qo, qos, head * H, n)
        K, KO = (rows(a, b, head * Hk, n) if Hk else [] for a, b in ((k, ks), (ko, kos)))
        bad = (q != qo and meet(Q, QO)) or (k != ko and meet(K, KO)) or meet(K, QO) or meet(Q, KO) or meet(QO, KO)
        rc = norm_rope(L, n, q, qs, H, qo, qos, *((k, ks, Hk, ko, kos) if Hk else ()), dt=dt, D=D)
        assert (rc == SHAPE) == bad and (bad or rc in (-7, -8)), (n, H, Hk, dt, q, qs, qo, qos, k, ks, ko, kos)
        got[bad] += 1
    assert min(got.values()) > 2000


def lora(L, x, res, y, ws, wsb=1 << 20, K=64, M=100, n=4, rank=8):
    """Addresses in units of 16 bytes: x 64 units, res and y 100, the workspace 8 (one split)."""
    at = lambda a: A + 16 * a  # noqa: E731
    d = api.Lora(3, rank, 2, 0, A, A, None, None)
    return L.qmv_lora_run(ctypes.byref(d), A, at(x), at(res), at(y), K, M, n, at(ws), wsb, None)


def test_an_adapters_workspace_that_overlaps(L):
    x, res, y = 0, 1000, 2000
    for ws in (x, x - 7, x + 63, res, res - 7, res + 99, y, y - 7, y + 99):
        assert lora(L, x, res, y, ws) == SHAPE and lora(L, x, res, y, ws, wsb=8 * 16) == SHAPE
        assert lora(L, x, res, res, ws if ws < y - 7 else ws - 1000) == SHAPE   # in place
    # rank 128 and 40000 columns: 20 splits of 4 x 128 sums, 2560 units
    for ws in (6001 - 2560, 6000 + 99):
        assert lora(L, 100000, 6000, 9000, ws, K=40000, rank=128) == SHAPE
    d = api.Lora(3, 128, 2, 0, A, A, None, None)
    assert L.qmv_lora_workspace_bytes(ctypes.byref(d), 40000, 4) == 2560 * 16


@no_device
def test_a_workspace_beside_the_tensors(L):
    for ws in (64, 1000 - 8, 1100, 2000 - 8, 2100):
        assert lora(L, 0, 1000, 2000, ws) in (-7, -8)  # (a larger buffer's unused rest may be anything)
    assert lora(L, 0, 1000, 1000, 2000) in (-7, -8)
    assert lora(L, 100000, 6000, 9000, 6000 - 2560, K=40000, rank=128) in (-7, -8)


@no_device
def test_far_rows(L):
    # tokens 2^20 elements apart (2^18 units of fp32), 65535 of them: extents of 2^38 bytes
    far = 1 << 18
    assert norm_rope(L, 65535, 0, far, 6, 12, far) in (-7, -8)
    assert norm_rope(L, 65535, 0, far, 6, 12 + far, far) in (-7, -8)
    assert norm_rope(L, 65535, 0, far, 6, 11 + 65534 * far, far) == SHAPE
    assert norm_rope(L, 65535, 0, far, 6, 12 + 65534 * far, far) in (-7, -8)
    # a step of one unit more each token: away from the row before, the next one 262044 tokens on
    assert norm_rope(L, 65535, 0, far, 6, 100, far + 1) in (-7, -8)
    assert norm_rope(L, 65535, 0, far, 6, 100, far - 1) == SHAPE      # towards it
    # (the last token is 65534 units nearer: it meets the row's 12 units from 65534 + 11 on down)
    assert norm_rope(L, 65535, 0, far, 6, 65535 + 11, far - 1) in (-7, -8)
    assert norm_rope(L, 65535, 0, far, 6, 65534 + 11, far - 1) == SHAPE
    assert norm_rope(L, 65535, 0, far, 6, 100, 2 * far) in (-7, -8)


@pytest.mark.gpu
def test_results_among_the_rows_of_one_buffer(lib):
    n, D = 37, 64
    r = api.rope(D, torch.exp(-0.2 * torch.arange(D // 2)).cuda())
    pos = torch.arange(n, dtype=torch.int32).cuda()[:, None].contiguous()
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.randn(n, 12, D, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
        before = buf.clone()
        want = api.norm_rope(r, buf[:, :4], buf[:, 4:6], pos=pos)
        # queries to heads 6 to 9, keys in place
        api.norm_rope(r, buf[:, :4], buf[:, 4:6], pos=pos, q_out=buf[:, 6:10], k_out=buf[:, 4:6])
        assert torch.equal(buf[:, 6:10], want[0]) and torch.equal(buf[:, 4:6], want[1])
        assert torch.equal(buf[:, :4], before[:, :4]) and torch.equal(buf[:, 10:], before[:, 10:])
        # every other row of a buffer: results with another stride among the inputs
        wide = before.clone().view(n * 12, 1, D)
        x, y = wide[:n:1].clone(), wide.as_strided((n, 1, D), (4 * D, D, 1), D)
        src = wide.as_strided((n, 1, D), (2 * D, D, 1))
        src.copy_(x)
        keep = wide.clone()
        one = api.norm_rope(r, src, pos=pos)[0]
        api.norm_rope(r, src, pos=pos, q_out=y)
        assert torch.equal(y, one) and torch.equal(wide[::2], keep[::2])
        for out in (buf[:, 1:5], buf[:, 3:7], buf[:, 2:6]):
            with pytest.raises(api.QmvError):
                api.norm_rope(r, buf[:, :4], buf[:, 4:6], pos=pos, q_out=out)
