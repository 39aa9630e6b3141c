"""Append to the paged 8-bit cache and reading it back: every byte against the
restatement in kv_ref (scales and codes are defined by fp32 operations whose
order is fixed, so nothing is tolerated)."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import kv_ref

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]


def dev32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def tables(rng, lens, P, n_pages, spare=2):
    """A random page table with -1 past each sequence's pages."""
    need = [-(-n // P) for n in lens]
    perm = rng.permutation(n_pages)[:sum(need)]
    t = np.full((len(lens), max(need + [1]) + spare), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        t[s, :n] = perm[at:at + n]
        at += n
    return t


class Pair:
    """The library's cache and the restatement's, byte for byte alike at the start."""

    def __init__(self, H, D, P, n_pages, fill=0xFF):
        self.ref = kv_ref.Cache(H, D, P, n_pages, fill)
        self.dev = api.kv_cache(H, D, P, n_pages, pages=torch.from_numpy(self.ref.pages.copy()).cuda(),
                                bounds=torch.from_numpy(self.ref.bounds.copy()).cuda())

    def append(self, k, v, table, lens, starts):
        ragged = starts is not None
        starts = np.arange(len(lens) + 1) if starts is None else np.asarray(starts)
        self.ref.append(k.float().cpu().numpy(), v.float().cpu().numpy(), table, lens, starts)
        api.kv_append(self.dev, k, v, dev32(table), dev32(lens), dev32(starts) if ragged else None)

    def check(self):
        assert np.array_equal(self.dev.page_tensor.cpu().numpy(), self.ref.pages)
        assert np.array_equal(self.dev.bounds_tensor.cpu().numpy(), self.ref.bounds)
        assert api.get_device_error() == 0


def randn(rng, *shape, dtype=torch.float32, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("P", [16, 32, 64])
def test_prompts_then_single_tokens(lib, dtype, D, P):
    rng = np.random.default_rng(D + P)
    H, first = 2, [1, P - 1, P, P + 1, 3 * P + 5]
    n = len(first)
    pair = Pair(H, D, P, 64)
    final = [f + 4 for f in first]
    table = tables(rng, final, P, 64)
    starts = np.concatenate([[0], np.cumsum(first)])
    pair.append(randn(rng, starts[-1], H, D, dtype=dtype), randn(rng, starts[-1], H, D, dtype=dtype, scale=0.1), table,
                first, starts)
    pair.check()
    for step in range(1, 5):  # growing magnitudes: most steps rescale the page's old codes
        lens = [f + step for f in first]
        pair.append(randn(rng, n, H, D, dtype=dtype, scale=step), randn(rng, n, H, D, dtype=dtype, scale=1 / step),
                    table, lens, None)
        pair.check()


def test_several_tokens_across_a_page_border_and_appending_again(lib):
    rng = np.random.default_rng(5)
    H, D, P = 3, 128, 16
    pair = Pair(H, D, P, 40)
    table = tables(rng, [40, 60, 33], P, 40)
    pair.append(randn(rng, 53, H, D), randn(rng, 53, H, D), table, [10, 30, 13], [0, 10, 40, 53])
    # ragged: no new token at all in the middle sequence
    k, v = randn(rng, 27, H, D, scale=2), randn(rng, 27, H, D)
    pair.append(k, v, table, [17, 30, 33], [0, 7, 7, 27])
    pair.check()
    # the same call again leaves every byte (the scales are already large enough)
    pair.append(k, v, table, [17, 30, 33], [0, 7, 7, 27])
    pair.check()
    # a rejected draft: lens go back and other tokens take the place
    pair.append(randn(rng, 3, H, D), randn(rng, 3, H, D), table, [12, 29, 30], None)
    pair.check()


def test_zero_tiny_and_tied_values(lib):
    rng = np.random.default_rng(6)
    H, D, P = 1, 64, 16
    pair = Pair(H, D, P, 8)
    table = tables(rng, [9], P, 8)
    x = torch.zeros(1, H, D, device="cuda")
    pair.append(x, x, table, [1], None)                       # all zero: scale 0
    pair.append(x + 1e-39, x + 1e-38, table, [2], None)       # subnormal scale, 1 / d overflows
    pair.append(x + 1e-30, x, table, [3], None)
    ties = (torch.arange(64, device="cuda").float() + 0.5).reshape(1, 1, 64)
    ties[..., 0] = 127.0                                      # d = 1: every other value is a tie
    pair.append(ties, -ties, table, [4], None)
    pair.append(2 * ties, -ties, table, [5], None)            # ratio 1/2: old codes tie too
    pair.check()


def test_strided_tokens_and_no_bounds(lib):
    rng = np.random.default_rng(7)
    H, D, P = 4, 128, 32
    pair = Pair(H, D, P, 30)
    table = tables(rng, [70, 5], P, 30)
    fused = randn(rng, 75, 3 * H, D)  # q, k, v of a token side by side
    k, v = fused[:, H:2 * H], fused[:, 2 * H:]
    pair.append(k, v, table, [70, 5], [0, 70, 75])
    pair.check()
    plain = api.kv_cache(H, D, P, 30)
    assert plain.bounds is None
    api.kv_append(plain, k, v, dev32(table), dev32([70, 5]), dev32([0, 70, 75]))
    a, b = api.kv_read(plain, dev32(table), dev32([70, 5]), dev32([0, 70, 75]), 75)
    c, d = api.kv_read(pair.dev, dev32(table), dev32([70, 5]), dev32([0, 70, 75]), 75)
    assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (192, 32), (256, 16)])
def test_read_gives_the_codes_values(lib, dtype, D, P):
    rng = np.random.default_rng(8)
    H, lens = 2, [1, 2 * P, 0, 3 * P - 7]
    pair = Pair(H, D, P, 20)
    table = tables(rng, lens, P, 20)
    starts = np.concatenate([[0], np.cumsum(lens)])
    pair.append(randn(rng, starts[-1], H, D), randn(rng, starts[-1], H, D), table, lens, starts)
    pair.check()
    back = [min(n, P + 3) for n in lens]  # the last tokens only
    st = np.concatenate([[0], np.cumsum(back)])
    k, v = api.kv_read(pair.dev, dev32(table), dev32(lens), dev32(st), int(st[-1]), dtype)
    for s, n in enumerate(lens):
        for h in range(H):
            kk, vv = (a[n - back[s]:n].astype(np.float32) for a in pair.ref.values(table[s], h, n))
            assert np.array_equal(k[st[s]:st[s + 1], h].float().cpu().numpy(), torch.from_numpy(kk).to(dtype).float().numpy())
            assert np.array_equal(v[st[s]:st[s + 1], h].float().cpu().numpy(), torch.from_numpy(vv).to(dtype).float().numpy())
    # an empty slot of a decode batch reads as zeros and is no error
    k, v = api.kv_read(pair.dev, dev32(table), dev32(lens))
    assert (k[2] == 0).all() and (v[2] == 0).all() and api.get_device_error() == 0


def test_quantization_error_is_at_most_half_a_step(lib):
    # written at once, |x - value| <= scale / 2 (+ fp32 roundings of x / d and c d)
    rng = np.random.default_rng(9)
    H, D, P, n = 2, 128, 64, 200
    cache = api.kv_cache(H, D, P, 4)
    x, y = randn(rng, n, H, D), randn(rng, n, H, D, scale=30)
    t, lens, st = dev32([[2, 0, 3, 1]]), dev32([n]), dev32([0, n])
    api.kv_append(cache, x, y, t, lens, st)
    k, v = api.kv_read(cache, t, lens, st, n)
    for a, b in ((x, k), (y, v)):
        for p0 in range(0, n, P):
            for h in range(H):
                u, w = a[p0:p0 + P, h], b[p0:p0 + P, h]
                d = u.abs().max() / 127
                assert ((u - w).abs() <= d * (0.5 + 127 * 2.0 ** -22)).all()


def test_contradictions_are_flagged_and_nothing_else_is_touched(lib):
    rng = np.random.default_rng(10)
    H, D, P = 2, 64, 16
    pair = Pair(H, D, P, 10)
    k = randn(rng, 4, H, D)

    def call(table, lens, starts=None, n=4):
        api.kv_append(pair.dev, k[:n], k[:n], dev32(table), dev32(lens), None if starts is None else dev32(starts))
        return api.get_device_error()

    assert call([[10], [-1], [0], [1]], [1, 1, 1, 1]) == api.DEVERR_PAGE       # no such pages
    pair.ref.append(k[2:4].cpu().numpy(), k[2:4].cpu().numpy(), np.array([[0], [1]]), [1, 1], [0, 1, 2])
    pair.check()
    assert call([[2]], [3], [0, 4]) == api.DEVERR_BATCH                        # four tokens of three
    pair.ref.append(k[1:4].cpu().numpy(), k[1:4].cpu().numpy(), np.array([[2]]), [3], [0, 3])
    pair.check()
    assert call([[3]], [17], [0, 4]) == api.DEVERR_BATCH                       # longer than its table
    assert call([[3], [4]], [2, 2], [0, 2, 9]) == api.DEVERR_BATCH             # past n_tok
    assert call([[5], [6]], [1, 1], [3, 1, 2]) & ~api.DEVERR_BATCH == 0        # not ascending
    assert call([[7]] * 4, [0, 0, 0, 0]) == 0                                  # empty slots are no error


def test_pages_past_four_gigabytes(lib):
    H, D, P = 8, 256, 64
    n_pages = (1 << 33) // (H * kv_ref_bytes(D, P)) + 9  # over 8 GB
    cache = api.kv_cache(H, D, P, n_pages, bounds=True)
    assert cache.page_tensor.numel() > 1 << 33
    rng = np.random.default_rng(11)
    pages = [n_pages - 1, n_pages // 2 + 1, 0]
    n = 2 * P + 5
    k, v = randn(rng, n, H, D), randn(rng, n, H, D)
    small = Pair(H, D, P, 3)
    api.kv_append(cache, k, v, dev32([pages]), dev32([n]), dev32([0, n]))
    small.append(k, v, np.array([[0, 1, 2]]), [n], [0, n])
    small.check()
    t = torch.tensor(pages, device="cuda")
    for p0, p1 in zip(pages, range(3)):
        a, b = cache.page_tensor[p0], small.dev.page_tensor[p1]
        if p1 < 2:
            assert torch.equal(a[:, 16:], b[:, 16:]) and torch.equal(a[:, :8], b[:, :8])
    big, ref = (api.kv_read(c, tt, dev32([n]), dev32([0, n]), n)
                for c, tt in ((cache, dev32([pages])), (small.dev, dev32([[0, 1, 2]]))))
    assert torch.equal(big[0], ref[0]) and torch.equal(big[1], ref[1])
    q = randn(rng, 1, 2 * H, D)
    for sel in (None, dev32(np.broadcast_to([[[0, 2]]], (1, H, 2)).copy())):
        a = api.kv_attend(cache, q, dev32([pages]), dev32([n]), pages=sel)
        b = api.kv_attend(small.dev, q, dev32([[0, 1, 2]]), dev32([n]), pages=sel)
        assert torch.equal(a, b)
    a = api.kv_select(cache, q, dev32([pages]), dev32([n]), 2)
    assert torch.equal(a, api.kv_select(small.dev, q, dev32([[0, 1, 2]]), dev32([n]), 2))
    assert t.numel() == 3 and api.get_device_error() == 0


def kv_ref_bytes(D, P):
    return 16 + 2 * P * D
