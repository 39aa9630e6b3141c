"""Positions that the rotation takes from lens and starts where these contradict the
call: as the cache calls clamp them, with the same error bits."""
import pytest
import torch

from moe_matvec_gb300 import api

pytestmark = pytest.mark.gpu

BATCH = api.DEVERR_BATCH


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def stored(lens, starts, k):
    """The slots of a fresh cache that kv_append writes (values 1 and up): {token: (sequence, position)}, and the error word."""
    n_seq, P, pages = len(lens), 16, 4
    cache = api.kv_cache(k.shape[1], 64, P, n_seq * pages)
    table = torch.arange(n_seq * pages, dtype=torch.int32).view(n_seq, pages).cuda()
    zero = torch.zeros(n_seq * P * pages, k.shape[1], 64, device="cuda")
    full = ints([P * pages] * n_seq)
    every = ints([i * P * pages for i in range(n_seq + 1)])
    api.kv_append(cache, zero, zero, table, full, every)
    assert api.get_device_error() == 0
    api.kv_append(cache, k, k, table, ints(lens), None if starts is None else ints(starts))
    err = api.get_device_error()
    got = api.kv_read(cache, table, full, every, n_seq * P * pages)[0][:, 0, 0].view(n_seq, P * pages)
    at = {}
    for s in range(n_seq):
        for i in range(P * pages):
            v = int(round(float(got[s, i])))
            if v:
                at[v - 1] = (s, i)
    return at, err


# lens, starts, tokens, position of each token (None: not covered)
CASES = [
    ([5], [0, 9], 3, [2, 3, 4]),                 # the last start past the call's tokens
    ([9, 4], [0, 2, 9], 4, [7, 8, 2, 3]),
    ([4], [-7, 3], 3, [1, 2, 3]),
    ([4], [5, 1], 3, [None, None, None]),        # descending
    ([2], [0, 3], 3, [-1, 0, 1]),                # fewer than the call brings
    ([7, 1], [0, 1, 4], 4, [6, -2, -1, 0]),
    ([-4, 3], [0, 1, 2], 2, [-1, 2]),            # negative: as 0
    ([3, 2], None, 2, [2, 1]),
    ([3, -2], None, 2, [2, -1]),
]


@pytest.mark.parametrize("lens,starts,n,pos", CASES)
def test_contradictions_are_clamped_as_by_the_cache(lib, lens, starts, n, pos):
    k = (torch.arange(1, n + 1, device="cuda").float()[:, None, None] * torch.ones(1, 2, 64, device="cuda")).contiguous()
    at, kv_err = stored(lens, starts, k)
    held, there = {t: p for t, (_, p) in at.items()}, {t: p for t, p in enumerate(pos) if p is not None and p >= 0}
    if starts is not None and starts[0] < 0:
        assert held.items() <= there.items()  # (the cache leaves some out)
    else:
        assert held == there
    r = api.rope(64, torch.exp(-0.2 * torch.arange(32)).cuda())
    x = torch.randn(n, 2, 64, generator=torch.Generator().manual_seed(n)).cuda()
    out = torch.full_like(x, 7.0)
    api.norm_rope(r, x, lens=ints(lens), starts=None if starts is None else ints(starts), q_out=out)
    err = api.get_device_error()
    assert err == kv_err
    want = api.norm_rope(r, x, pos=ints([[p or 0] for p in pos]))[0]
    for t, p in enumerate(pos):
        assert torch.equal(out[t], torch.full_like(out[t], 7.0) if p is None else want[t]), t
    assert api.get_device_error() == 0


def test_what_is_flagged(lib):
    r = api.rope(64, torch.exp(-0.2 * torch.arange(32)).cuda())
    x = torch.randn(3, 2, 64, device="cuda")
    for lens, starts, flagged in (([2], [0, 3], True), ([3], [0, 3], False), ([0], [0, 3], False), ([9, 1], [0, 1, 3], True),
                                  ([1, 0, 4], None, False), ([1, -1, 4], None, True), ([5], [0, 4], True), ([5], [1, 2], False)):
        api.norm_rope(r, x, lens=ints(lens), starts=None if starts is None else ints(starts))
        assert api.get_device_error() == (BATCH if flagged else 0), (lens, starts)


def test_an_axis_that_is_none_is_flagged_either_way(lib):
    freq = torch.exp(-0.2 * torch.arange(32)).cuda()
    axis = torch.zeros(32, dtype=torch.uint8)
    axis[31] = 2
    good, bad = api.rope(64, freq), api.rope(64, freq, axis=axis.cuda(), n_axes=2)
    x = torch.randn(3, 2, 64, device="cuda")
    for at in (dict(lens=ints([4, 5, 6])), dict(lens=ints([9]), starts=ints([0, 3]))):
        want = api.norm_rope(good, x, **at)[0]
        assert api.get_device_error() == 0
        assert torch.equal(api.norm_rope(bad, x, **at)[0], want)
        assert api.get_device_error() == BATCH
