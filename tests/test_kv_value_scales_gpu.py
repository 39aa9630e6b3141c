"""Attention where a page of values far larger than the others is loaded but
says nothing, or next to nothing, about a row: later than the row's token, out
of its window, or of negligible weight.  Such a row has to be as exact as it
would be without that page.

Tolerance: that of tests/test_kv_attend_gpu.py, (2^-17 A + 2^-16) sum p |v| and half
a unit of the output's type, relative to what the row itself sees.  A row that
does see the large page loses what lies far below it: the products of weight and
value scale enter the second product with an error of 2^-31 of the row's largest
where they are small, which n tokens of up to 127 scales make n 2^-31 T, T the
largest p 127 scale of a token that the row sees.  (Nothing beside 2^-16 sum p |v|
for the rows that do not see the page: their T is that of the small pages.)"""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests.test_kv_attend_gpu import UNIT, wide
from tests.test_kv_cache_gpu import Pair, dev32, randn, tables

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]
SHAPES = [(64, 16), (64, 64), (128, 32), (192, 64), (256, 16)]
BIG = [1e4, 1e6, 1e8]
BASE = 1e-4  # of the other values: the large ones still fit f16


def exact(ref, q, row, length, news, window):
    """One sequence's (out, its bound without the output's rounding) in 64 bits."""
    H, P, D = ref.H, ref.P, q.shape[2]
    G = q.shape[1] // H
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    see = np.arange(length)
    for h in range(H):
        k, v = ref.values(row, h, length)
        dv = np.array([ref.scales(row[j // P], h)[1] for j in see], np.float64)
        for i in range(news):
            pos = length - news + i
            keep = (see <= pos) & ((see > pos - window) | (window == 0))
            for g in range(h * G, h * G + G):
                x = q[i, g].astype(np.float64)
                z = k[keep] @ x / np.sqrt(D)
                p = np.exp(z - z.max())
                p /= p.sum()
                out[i, g] = p @ v[keep]
                arg = np.abs(x).max() * np.abs(k[keep]).sum(1).max() / np.sqrt(D)
                bound[i, g] = (2.0 ** -17 * arg + 2.0 ** -16) * (p @ np.abs(v[keep])) + \
                    keep.sum() * 2.0 ** -31 * (p * dv[keep]).max() * 127
    return out, bound


def attend_both(pair, q, table, lens, starts, P, window=0):
    """A cluster per item (a table as wide as the data), and equal shares (a wide one)."""
    want, bound = exact(pair.ref, q.float().cpu().numpy(), table[0], lens[0], len(q), window)
    for t in (table, wide(table, P)):
        out = api.kv_attend(pair.dev, q, dev32(t), dev32(lens), None if starts is None else dev32(starts), window=window)
        got = out.double().cpu().numpy()
        most = bound + UNIT[out.dtype] * np.abs(want) + (2.0 ** -25 if out.dtype == torch.float16 else 1e-38)
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= most).all(), f"worst {np.max(np.abs(got - want) / most)} of the bound"
        assert api.get_device_error() == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P", SHAPES)
@pytest.mark.parametrize("big", BIG)
def test_a_large_page_after_the_token(lib, dtype, D, P, big):
    # eight new tokens, the last four on a page of large values that the first four do not see
    rng = np.random.default_rng(D + P)
    n = 3 * P + 4
    pair = Pair(2, D, P, 6)
    table = tables(rng, [n], P, 6)
    k, v = randn(rng, n, 2, D), randn(rng, n, 2, D, scale=BASE)
    v[3 * P:] *= big
    pair.append(k, v, table, [n], [0, n])
    for G in (1, 3):
        attend_both(pair, randn(rng, 8, 2 * G, D, dtype=dtype), table, [n], [0, 8], P)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P", SHAPES)
@pytest.mark.parametrize("big", BIG)
def test_a_large_page_before_the_window(lib, dtype, D, P, big):
    # eight new tokens; the window of the last four begins after a page of large values
    rng = np.random.default_rng(D + P + 1)
    n = 3 * P + 15
    pair = Pair(2, D, P, 6)
    table = tables(rng, [n], P, 6)
    k, v = randn(rng, n, 2, D), randn(rng, n, 2, D, scale=BASE)
    v[2 * P:3 * P] *= big
    pair.append(k, v, table, [n], [0, n])
    for G in (1, 3):
        attend_both(pair, randn(rng, 8, 2 * G, D, dtype=dtype), table, [n], [0, 8], P, window=11)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P", SHAPES)
@pytest.mark.parametrize("big", BIG)
@pytest.mark.parametrize("at", [0, 2, 39])
def test_a_large_page_of_little_weight(lib, dtype, D, P, big, at):
    # the keys of the page with the large values lie 30 below the others' logits
    rng = np.random.default_rng(D + P + at)
    n = 40 * P - 3
    pair = Pair(1, D, P, 42)
    table = tables(rng, [n], P, 42)
    k, v = randn(rng, n, 1, D, scale=0.3), randn(rng, n, 1, D, scale=BASE)
    k[at * P:at * P + P] = -30 / (1.3 * D ** 0.5)
    v[at * P:at * P + P] *= big
    pair.append(k, v, table, [n], [0, n])
    for G in (4, 12):
        q = (randn(rng, 1, G, D).abs() + 0.5).to(dtype)
        attend_both(pair, q, table, [n], None, P)


def test_a_tokens_output_does_not_depend_on_later_pages(lib):
    # the same four tokens with and without a page of large values after them, bit for bit
    rng = np.random.default_rng(5)
    D, P, n = 128, 16, 52
    k, v, q = randn(rng, n, 1, D), randn(rng, n, 1, D), randn(rng, 8, 3, D)  # (items of 8 rows mix tokens)
    outs = []
    for big in (1, 1e7):
        pair = Pair(1, D, P, 4)
        v2 = v.clone()
        v2[48:] *= big
        pair.append(k, v2, np.array([[2, 0, 3, 1]]), [n], [0, n])
        outs.append(api.kv_attend(pair.dev, q, dev32([[2, 0, 3, 1]]), dev32([n]), dev32([0, 8]))[:4])
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", DT)
def test_tiny_huge_and_zero_values(lib, dtype):
    # value scales at both ends of fp32 (1 / scale overflows, scale^2 too), and none at all
    rng = np.random.default_rng(6)
    D, P, n = 64, 16, 100
    for scale in (0.0, 1e-42, 1e-37, 1e-30, 1e30, 1e34):
        if dtype == torch.float16 and scale > 1:
            continue  # the results would be infinite
        pair = Pair(1, D, P, 8)
        table = tables(rng, [n], P, 8)
        k, v = randn(rng, n, 1, D), randn(rng, n, 1, D) * scale
        pair.append(k, v, table, [n], [0, n])
        for G in (2, 12):
            q = randn(rng, 1, G, D, dtype=dtype)
            for t in (table, wide(table, P)):
                out = api.kv_attend(pair.dev, q, dev32(t), dev32([n]))
                assert torch.isfinite(out).all()
                if scale == 0 or dtype == torch.float16:
                    assert (out == 0).all()
                elif scale >= 1e-30:
                    attend_both(pair, q, table, [n], None, P)
                else:
                    assert (out.abs() <= 8 * scale).all()
        assert api.get_device_error() == 0
