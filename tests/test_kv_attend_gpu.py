"""Attention over the paged 8-bit cache, and page selection, against 64 bits.

Tolerance of an fp32 output: with A the largest |scale| max|q| sum|k| of the
row, a logit is off by at most 2^-23 A from q's two f16 parts, 16 * 2^-23 A from
the products' fp32 sums and 2^-22 A from the scaling; the softmax weight by
twice that (its own and the maximum's share of the sum).  Weights and their
f16 parts add 2^-21, and sums of up to a few hundred fp32 terms 2^-17 of
sum p |v|.  In all |out - out64| <= (2^-17 A + 2^-16) sum p |v|, plus half a unit
of the output's type.  Picks are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import kv_ref
from tests.test_kv_cache_gpu import Pair, dev32, randn, tables

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
DT = list(UNIT)


def filled(rng, H, D, P, lens, n_pages=None, scale=1.0):
    """A cache holding lens[s] random tokens per sequence; unused pages and slots hold 0xFF (scales NaN)."""
    n_pages = n_pages or sum(-(-n // P) for n in lens) + 3
    pair = Pair(H, D, P, n_pages)
    table = tables(rng, lens, P, n_pages)
    starts = np.concatenate([[0], np.cumsum(lens)])
    if starts[-1]:
        step = 16384
        assert starts[-1] <= step
        k, v = randn(rng, starts[-1], H, D, scale=scale), randn(rng, starts[-1], H, D)
        pair.append(k, v, table, lens, starts)
        pair.check()
    return pair, table


def check(pair, q, table, lens, starts, out, scale=None, **kw):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    st = np.arange(len(lens) + 1) if starts is None else np.asarray(starts)
    want, mag, arg = kv_ref.attend(pair.ref, q.float().cpu().numpy(), table, lens, st, scale, **kw)
    got = out.double().cpu().numpy()
    bound = (2.0 ** -17 * arg + 2.0 ** -16) * mag + UNIT[out.dtype] * np.abs(want) + (2.0 ** -25 if out.dtype == torch.float16 else 1e-38)
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= bound).all(), f"worst {np.max(err / bound)} of the bound"
    assert api.get_device_error() == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("P", [16, 32, 64])
def test_single_tokens_ragged_lengths(lib, dtype, D, P):
    rng = np.random.default_rng(D * P)
    lens = [1, 0, P - 1, P, P + 1, 63, 64, 65, 127, 200, 777]
    pair, table = filled(rng, 2, D, P, lens)
    q = randn(rng, len(lens), 6, D, dtype=dtype, scale=2)
    out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens))
    assert (out[1] == 0).all()
    check(pair, q, table, lens, None, out)


@pytest.mark.parametrize("H,G", [(1, 1), (2, 3), (1, 7), (3, 8), (1, 9), (2, 16), (1, 33), (8, 1)])
def test_head_groups(lib, H, G):
    rng = np.random.default_rng(H * 100 + G)
    lens = [130, 5, 300]
    pair, table = filled(rng, H, 128, 32, lens)
    q = randn(rng, 3, H * G, 128)
    check(pair, q, table, lens, None, api.kv_attend(pair.dev, q, dev32(table), dev32(lens)))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 17, 64, 100])
def test_several_tokens_masks_and_windows(lib, causal, window):
    rng = np.random.default_rng(window + causal)
    lens, news = [150, 9, 40, 0, 300], [5, 9, 1, 0, 21]
    st = np.concatenate([[0], np.cumsum(news)])
    for D, P, G in ((64, 16, 4), (128, 64, 3)):
        pair, table = filled(rng, 2, D, P, lens)
        q = randn(rng, st[-1], 2 * G, D, scale=1.5)
        out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), dev32(st), causal=causal, window=window)
        check(pair, q, table, lens, st, out, causal=causal, window=window)


def test_the_largest_window(lib):
    # with more tokens in the call than the sequence holds, and none at all
    rng = np.random.default_rng(29)
    lens, news = [1, 0, 90], [4, 3, 2]
    st = np.concatenate([[0], np.cumsum(news)])
    pair, table = filled(rng, 1, 64, 16, lens)
    q = randn(rng, st[-1], 2, 64)
    out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), dev32(st), window=2 ** 31 - 1)
    check(pair, q, table, lens, st, out)
    assert torch.equal(out, api.kv_attend(pair.dev, q, dev32(table), dev32(lens), dev32(st)))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P,G", [(64, 16, 3), (64, 64, 12), (128, 64, 4), (128, 32, 16), (192, 16, 5), (256, 64, 9)])
def test_one_token_a_sequence_with_and_without_starts(lib, dtype, D, P, G):
    # the same batch as items known beforehand (a cluster each) and as equal shares of the GPU
    rng = np.random.default_rng(D + P + G)
    lens = [1, 700, 0, 64, 333, 1500]
    pair, table = filled(rng, 2, D, P, lens)
    q = randn(rng, len(lens), 2 * G, D).to(dtype)
    st = list(range(len(lens) + 1))
    for window in (0, 70):
        for starts in (None, dev32(st)):
            out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), starts, window=window)
            check(pair, q, table, lens, st, out, window=window)


def wide(table, P):
    """The same pages in a table of room for 100000 tokens."""
    return np.concatenate([table, np.full((len(table), 100000 // P - table.shape[1]), -1, table.dtype)], 1)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P,G", [(64, 16, 3), (64, 64, 12), (128, 64, 4), (128, 32, 16), (192, 16, 5), (256, 64, 9)])
def test_narrow_and_wide_tables(lib, dtype, D, P, G):
    # few tiles by the table (a cluster per item) and possibly many (equal shares of the GPU)
    rng = np.random.default_rng(D + P + G + 1)
    for lens, news in (([1, 700, 0, 64, 333], [1, 5, 0, 2, 1]), ([0, 90, 200], [1, 1, 1]), ([40], [40])):
        st = np.concatenate([[0], np.cumsum(news)])
        pair, table = filled(rng, 2, D, P, lens)
        q = randn(rng, st[-1], 2 * G, D).to(dtype)
        for window, causal in ((0, True), (0, False), (70, True)):
            for t in (table, wide(table, P)):
                out = api.kv_attend(pair.dev, q, dev32(t), dev32(lens), dev32(st), causal=causal, window=window)
                check(pair, q, table, lens, st, out, causal=causal, window=window)
    ids = np.array([[[0, 1], [0, -1]]] * 40, np.int32)
    out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), dev32(st), pages=dev32(ids))
    check(pair, q, table, lens, st, out, pages=ids)


def test_rows_that_are_no_numbers_stay_so(lib):
    rng = np.random.default_rng(28)
    lens = [300, 50]
    pair, table = filled(rng, 1, 128, 64, lens)
    q = randn(rng, 2, 4, 128)
    q[0, 1, 5] = float("nan")
    for t in (table, wide(table, 64)):
        out = api.kv_attend(pair.dev, q, dev32(t), dev32(lens))
        assert out[0, 1].isnan().all()
        assert not out[0, [0, 2, 3]].isnan().any() and not out[1].isnan().any()


def test_a_whole_prompt(lib):
    rng = np.random.default_rng(30)
    lens = [260, 33]
    st = [0, 260, 293]
    pair, table = filled(rng, 2, 64, 64, lens)
    q = randn(rng, 293, 8, 64)
    check(pair, q, table, lens, st, api.kv_attend(pair.dev, q, dev32(table), dev32(lens), dev32(st)))


@pytest.mark.parametrize("n_seq,length", [(1, 9000), (3, 5000), (70, 150), (300, 40)])
def test_long_and_many_sequences(lib, n_seq, length):
    rng = np.random.default_rng(n_seq)
    lens = [int(v) for v in rng.integers(1, length, n_seq)]
    lens[0] = length
    pair, table = filled(rng, 1, 128, 64, lens)
    q = randn(rng, n_seq, 4, 128, scale=3)
    out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens))
    check(pair, q, table, lens, None, out)
    # bitwise reproducible
    assert torch.equal(out, api.kv_attend(pair.dev, q, dev32(table), dev32(lens)))


def test_peaked_and_extreme_logits(lib):
    rng = np.random.default_rng(31)
    lens = [500, 500, 500]
    pair, table = filled(rng, 1, 128, 64, lens, scale=8)
    q = randn(rng, 3, 8, 128)
    q[0] *= 100     # one token takes all the weight
    q[1] = 0        # uniform weights
    q[2] *= 1e-20
    for scale in (None, 0.0, -0.3, 5.0):
        out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), scale=scale)
        check(pair, q, table, lens, None, out, scale=scale)


def test_pages_of_very_different_scales(lib):
    # an outlier page a thousand times larger than its neighbours
    rng = np.random.default_rng(32)
    H, D, P = 1, 128, 16
    pair = Pair(H, D, P, 20)
    table = tables(rng, [200], P, 20)
    k, v = randn(rng, 200, H, D), randn(rng, 200, H, D)
    v[48:64] *= 1000
    v[64:80] *= 1e-3
    k[80:96] = 0
    v[96:112] = 0
    pair.append(k, v, table, [200], [0, 200])
    q = randn(rng, 1, 5, D)
    check(pair, q, table, [200], None, api.kv_attend(pair.dev, q, dev32(table), dev32([200])))


def test_strided_queries_and_given_buffers(lib):
    rng = np.random.default_rng(33)
    lens = [100, 77]
    pair, table = filled(rng, 2, 128, 32, lens)
    fused = randn(rng, 2, 12, 128)
    q = fused[:, 2:10]
    ws = torch.full((api.kv_attend_workspace_bytes(pair.dev, 8, 2, 2),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((2, 8, 128), float("nan"), device="cuda")
    r = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), ws=ws, out=out)
    assert r is out
    check(pair, q, table, lens, None, out)


def test_non_finite_rows_stay_their_own(lib):
    rng = np.random.default_rng(34)
    lens = [90, 70]
    pair, table = filled(rng, 1, 64, 16, lens)
    q = randn(rng, 2, 4, 64)
    bad = q.clone()
    bad[0, 1, 3] = float("nan")
    a = api.kv_attend(pair.dev, q, dev32(table), dev32(lens))
    b = api.kv_attend(pair.dev, bad, dev32(table), dev32(lens))
    keep = torch.ones(2, 4, dtype=torch.bool)
    keep[0, 1] = False
    assert torch.equal(a[keep.cuda()], b[keep.cuda()]) and b[0, 1].isnan().all()


def test_missing_pages_are_left_out_and_flagged(lib):
    rng = np.random.default_rng(35)
    pair, table = filled(rng, 1, 64, 16, [80, 20])
    q = randn(rng, 2, 2, 64)
    bad = table.copy()
    bad[0, 2] = -1
    bad[0, 3] = 1000
    out = api.kv_attend(pair.dev, q, dev32(bad), dev32([80, 20]))
    assert api.get_device_error() == api.DEVERR_PAGE
    only = dev32(np.array([[[0, 1, 4]], [[0, 1, -1]]]))
    assert torch.equal(out, api.kv_attend(pair.dev, q, dev32(table), dev32([80, 20]), pages=only)) or torch.allclose(
        out, api.kv_attend(pair.dev, q, dev32(table), dev32([80, 20]), pages=only), rtol=1e-5, atol=1e-6)
    assert api.get_device_error() == 0


def test_graph_replays_as_lengths_grow(lib):
    rng = np.random.default_rng(36)
    H, D, P = 2, 128, 64
    pair = Pair(H, D, P, 12)
    table = tables(rng, [200, 300], P, 12)
    lens = dev32([100, 130])
    pair.append(randn(rng, 230, H, D), randn(rng, 230, H, D), table, [100, 130], [0, 100, 230])
    k, v, q = randn(rng, 2, H, D), randn(rng, 2, H, D), randn(rng, 2, 8, D)
    td = dev32(table)
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
    for step in range(1, 6):
        k.copy_(randn(rng, 2, H, D))
        v.copy_(randn(rng, 2, H, D, scale=step))
        g.replay()
        torch.cuda.synchronize()
        now = [100 + step, 130 + step]
        pair.ref.append(k.cpu().numpy(), v.cpu().numpy(), table, now, [0, 1, 2])
        assert np.array_equal(pair.dev.page_tensor.cpu().numpy(), pair.ref.pages)
        check(pair, q, table, now, None, out)


def test_a_stream_that_is_not_the_current_one(lib):
    # the workspace is dropped when the call returns: nobody may have its memory before the work is done
    rng = np.random.default_rng(37)
    pair, table = filled(rng, 2, 128, 64, [900, 1200])
    q, td, lens = randn(rng, 2, 8, 128), dev32(table), dev32([900, 1200])
    want = api.kv_attend(pair.dev, q, td, lens)
    picks = api.kv_select(pair.dev, q, td, lens, 5)
    size = api.kv_attend_workspace_bytes(pair.dev, 8, 2, 2)
    small = api.kv_select_workspace_bytes(pair.dev, 2, td.shape[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # the work below starts some 10 ms later
    out = api.kv_attend(pair.dev, q, td, lens, stream=side)
    ids = api.kv_select(pair.dev, q, td, lens, 5, stream=side)
    other = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (size, size, small, small)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(ids, picks)
    assert not any(t.any() for t in other)


# ---------------------------------------------------------------- selection
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,P,G", [(64, 16, 1), (128, 32, 4), (192, 16, 3), (256, 64, 8)])
def test_picks_are_the_definitions(lib, dtype, D, P, G):
    rng = np.random.default_rng(D + G)
    lens = [1, P, 12 * P + 3, 40 * P - 1, 0]
    pair, table = filled(rng, 2, D, P, lens)
    q = randn(rng, len(lens), 2 * G, D, dtype=dtype)
    for n_sel in (1, 2, 5, 12, 13, 39, 64):
        ids = api.kv_select(pair.dev, q, dev32(table), dev32(lens), n_sel).cpu().numpy()
        want = kv_ref.select(pair.ref, q.float().cpu().numpy(), table, lens, np.arange(len(lens) + 1), n_sel)
        assert np.array_equal(ids, want)
        out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), pages=dev32(ids))
        check(pair, q, table, lens, None, out, pages=ids)


def test_ties_go_to_the_lower_page(lib):
    rng = np.random.default_rng(41)
    H, D, P = 1, 64, 16
    pair = Pair(H, D, P, 700)
    n = 690 * P
    table = tables(rng, [n], P, 700)
    few = randn(rng, 5 * P, H, D)
    k = few.repeat(138, 1, 1)  # every page has 137 twins
    pair.append(k, k, table, [n], [0, n])
    for q in (randn(rng, 1, 3, D), torch.zeros(1, 3, D, device="cuda")):
        for n_sel in (2, 100, 139, 400):
            ids = api.kv_select(pair.dev, q, dev32(table), dev32([n]), n_sel).cpu().numpy()
            assert np.array_equal(ids, kv_ref.select(pair.ref, q.cpu().numpy(), table, [n], [0, 1], n_sel))


def test_more_pages_than_shared_memory_holds_scores_of(lib):
    rng = np.random.default_rng(49)
    H, D, P, n = 1, 64, 16, 8400 * 16 - 5
    pair = Pair(H, D, P, 8403)
    table = tables(rng, [n], P, 8403)
    for at in range(0, n, 16000):
        m = min(16000, n - at)
        pair.append(randn(rng, m, H, D), randn(rng, m, H, D), table, [at + m], [0, m])
    for heads in (1, 5):
        q = randn(rng, 1, heads, D)
        for n_sel in (2, 300, 8400):
            ids = api.kv_select(pair.dev, q, dev32(table), dev32([n]), n_sel).cpu().numpy()
            assert np.array_equal(ids, kv_ref.select(pair.ref, q.cpu().numpy(), table, [n], [0, 1], n_sel))


def test_picks_of_several_tokens(lib):
    rng = np.random.default_rng(42)
    H, D, P = 2, 128, 16
    lens, news = [130, 47, 300], [3, 20, 1]
    st = np.concatenate([[0], np.cumsum(news)])
    pair, table = filled(rng, H, D, P, lens)
    q = randn(rng, st[-1], 4, D)
    ids = api.kv_select(pair.dev, q, dev32(table), dev32(lens), 3, dev32(st)).cpu().numpy()
    assert np.array_equal(ids, kv_ref.select(pair.ref, q.cpu().numpy(), table, lens, st, 3))
    for window in (0, 20):
        out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), dev32(st), window=window, pages=dev32(ids))
        check(pair, q, table, lens, st, out, window=window, pages=ids)


def test_bounds_are_upper_bounds_of_the_quantized_logits(lib):
    # score(page) >= max over the page's tokens and the group's heads of d_h dk (codes . codes)
    rng = np.random.default_rng(43)
    H, D, P, n = 1, 128, 32, 400
    pair, table = filled(rng, H, D, P, [n])
    q = randn(rng, 1, 4, D)
    ids = api.kv_select(pair.dev, q, dev32(table), dev32([n]), 4).cpu().numpy()[0, 0]
    best = np.full(-(-n // P), -np.inf)
    bound = np.full(-(-n // P), -np.inf)
    for g in range(4):
        x = q[0, g].cpu().numpy()
        d = np.abs(x).max() / np.float32(127)
        c = kv_ref.rule(x, d)
        for pg in range(-(-n // P)):
            k, _ = pair.ref.codes(table[0, pg], 0)
            dk, low, top = pair.ref.extremes(table[0, pg], 0)
            m = min(P, n - pg * P)
            best[pg] = max(best[pg], (k[:m] @ c).max() * float(d) * float(dk))
            bound[pg] = max(bound[pg], np.maximum(c * low, c * top).sum() * float(d) * float(dk))
    assert (best <= bound * (1 + 1e-6) + 1e-6).all()
    assert ids[-1] == (n - 1) // P and len(set(ids)) == 4


def test_pages_listed_by_the_caller(lib):
    rng = np.random.default_rng(44)
    lens = [200, 90]
    pair, table = filled(rng, 2, 64, 16, lens)
    q = randn(rng, 2, 6, 64)
    # unordered, with gaps, past the sequence, none at all
    ids = np.array([[[5, -1, 2, 11], [-1, -1, -1, -1]], [[0, 1, -1, 12], [3, -1, -1, 4]]], np.int32)
    out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), pages=dev32(ids))
    check(pair, q, table, lens, None, out, pages=ids)
    assert (out[0, 3:] == 0).all()
    far = ids.copy()
    far[0, 0, 0] = 10_000_000  # no page of the table
    api.kv_attend(pair.dev, q, dev32(table), dev32(lens), pages=dev32(far))
    assert api.get_device_error() == api.DEVERR_PAGE


@pytest.mark.parametrize("D,P,H,n_seq,length", [(128, 64, 4, 40, 9000), (64, 16, 8, 40, 6000), (256, 32, 2, 24, 6000)])
def test_shares_of_many_tiles(lib, D, P, H, n_seq, length):
    # a hundred tiles and more per SM: every stage, plan and barrier is used again and again
    g = torch.Generator().manual_seed(D)
    rng = np.random.default_rng(D)
    lens = [int(v) for v in rng.integers(length // 2, length, n_seq)]
    pages = [-(-n // P) for n in lens]
    cache = api.kv_cache(H, D, P, sum(pages))
    table = tables(rng, lens, P, sum(pages))
    td, ld = dev32(table), dev32(lens)
    for s in range(n_seq):
        k, v = (torch.randn(lens[s], H, D, generator=g).cuda() for _ in range(2))
        api.kv_append(cache, k, v, td[s:s + 1].clone(), dev32(lens[s:s + 1]), dev32([0, lens[s]]))
    q = torch.randn(n_seq, 4 * H, D, generator=g).cuda()
    first = api.kv_attend(cache, q, td, ld)
    for _ in range(10):
        assert torch.equal(first, api.kv_attend(cache, q, td, ld))
    for s in range(0, n_seq, 7):
        k, v = (t.double() for t in api.kv_read(cache, td[s:s + 1].clone(), dev32(lens[s:s + 1]), dev32([0, lens[s]]), lens[s]))
        for h in range(H):
            x = q[s, 4 * h:4 * h + 4].double()
            p = torch.softmax(x @ k[:, h].T / D ** 0.5, -1)
            want, mag = p @ v[:, h], p @ v[:, h].abs()
            arg = (x.abs().amax(1) * k[:, h].abs().sum(1).max() / D ** 0.5)[:, None]
            assert ((first[s, 4 * h:4 * h + 4] - want).abs() <= (2.0 ** -17 * arg + 2.0 ** -16) * mag).all()
    assert api.get_device_error() == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("G,news", [(3, [7, 1, 20]), (8, [2, 5, 1]), (16, [1, 1, 3]), (33, [1, 2, 1])])
def test_rows_per_kv_head(lib, dtype, D, G, news):
    # row counts around the kernels' 8, 16 and 32 rows of an item
    rng = np.random.default_rng(D + G)
    lens = [90, 31, 260]
    st = np.concatenate([[0], np.cumsum(news)])
    pair, table = filled(rng, 2, D, 32, lens)
    q = randn(rng, st[-1], 2 * G, D, dtype=dtype, scale=1.5)
    for kw in ({}, {"window": 40}, {"causal": False}):
        out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), dev32(st), **kw)
        check(pair, q, table, lens, st, out, **kw)


@pytest.mark.parametrize("dtype", DT)
def test_outlier_pages_in_every_type(lib, dtype):
    # values of one page a thousand or a million times larger than its
    # neighbours', which still count in full in the sum of the weights
    rng = np.random.default_rng(52)
    H, D, P = 2, 64, 16
    for big in (1e3, 1e6):
        pair = Pair(H, D, P, 20)
        table = tables(rng, [250], P, 20)
        k, v = randn(rng, 250, H, D), randn(rng, 250, H, D) * 0.01
        v[32:48] *= big
        pair.append(k, v, table, [250], [0, 250])
        q = randn(rng, 1, 6, D, dtype=dtype)
        if dtype == torch.float16 and big > 1e3:
            q *= 0  # (the values' mean still fits f16)
        check(pair, q, table, [250], None, api.kv_attend(pair.dev, q, dev32(table), dev32([250])))
        # the big page under a mask: the others must be as exact as without it
        sel = np.array([[[p for p in range(16) if p != 2]] * H], np.int32)
        check(pair, q, table, [250], None, api.kv_attend(pair.dev, q, dev32(table), dev32([250]), pages=dev32(sel)), pages=sel)


def by_device(cache):
    """A restatement cache holding what the device's holds."""
    ref = kv_ref.Cache(cache.n_kv_heads, cache.head_dim, cache.page_tokens, cache.n_pages)
    ref.pages[:] = cache.page_tensor.cpu().numpy()
    ref.bounds[:] = cache.bounds_tensor.cpu().numpy()
    return ref


@pytest.mark.parametrize("pages_held", [2500, 12000])
def test_picks_among_thousands_of_pages(lib, pages_held):
    # more pages than a block brings in at once, and than it keeps keys of
    rng = np.random.default_rng(60)
    H, D, P, n = 1, 64, 16, pages_held * 16 - 5
    cache = api.kv_cache(H, D, P, pages_held + 1, bounds=True)
    table = tables(rng, [n], P, pages_held + 1)
    for a in range(0, n, 60000):
        b = min(n, a + 60000)
        api.kv_append(cache, randn(rng, b - a, H, D), randn(rng, b - a, H, D), dev32(table), dev32([b]), dev32([0, b - a]))
    ref = by_device(cache)
    q = randn(rng, 1, 3, D)
    for n_sel in (2, 64, 2049, pages_held - 3):
        ids = api.kv_select(cache, q, dev32(table), dev32([n]), n_sel).cpu().numpy()
        assert np.array_equal(ids, kv_ref.select(ref, q.cpu().numpy(), table, [n], [0, 1], n_sel))
    assert api.get_device_error() == 0


def test_picks_for_many_query_heads(lib):
    rng = np.random.default_rng(61)
    pair, table = filled(rng, 1, 256, 16, [400])
    q = randn(rng, 1, 200, 256)
    ids = api.kv_select(pair.dev, q, dev32(table), dev32([400]), 7).cpu().numpy()
    assert np.array_equal(ids, kv_ref.select(pair.ref, q.cpu().numpy(), table, [400], [0, 1], 7))
    out = api.kv_attend(pair.dev, q, dev32(table), dev32([400]), pages=dev32(ids))
    check(pair, q, table, [400], None, out, pages=ids)


@pytest.mark.parametrize("D,dtype", [(64, torch.float32), (128, torch.bfloat16), (256, torch.float32)])
def test_as_many_sequences_as_a_call_takes(lib, D, dtype):
    rng = np.random.default_rng(62)
    lens = [int(v) for v in rng.integers(0, 12, 1024)]
    pair, table = filled(rng, 1, D, 16, lens)
    q = randn(rng, 1024, 3, D, dtype=dtype)
    check(pair, q, table, lens, None, api.kv_attend(pair.dev, q, dev32(table), dev32(lens)))
    ids = api.kv_select(pair.dev, q, dev32(table), dev32(lens), 1).cpu().numpy()
    assert np.array_equal(ids[:, 0, 0], [0 if n else -1 for n in lens])
    starts = np.concatenate([[0], np.cumsum([min(n, 2) for n in lens])])
    q = randn(rng, starts[-1], 12, D, dtype=dtype)
    out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), dev32(starts))
    check(pair, q, table, lens, starts, out)
