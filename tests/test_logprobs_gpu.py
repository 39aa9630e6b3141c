"""Log probabilities against 64 bits.

With s the sum over the row but for its largest term, in units of 2^-24: a term of
s and of the entropy's sum is off by its exponent's three roundings (3 |d|, of which
what counts is weighed by the term: at most 3 ln V on average over a sum) and ex2 (4); a
thread adds them in two chains of at most V / 512 (256 threads a row), and some 30
more join the sums.  So s is off by N = V / 512 + 3 * 18 + 40 units of itself, the log-sum-exp's log1p(s) by as much
of itself (and 2 for log1pf), the entropy by twice that of itself, a log probability by
that and 3 units of the difference to the largest."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import step_ref

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]
UNIT = 2.0 ** -24


def check(logits, tokens, n_top, scale=1.0):
    got = api.logprobs(logits, None if tokens is None else tokens.cuda(), n_top, scale)
    l = logits.double().cpu().numpy()
    *want, rest = step_ref.logprobs(l, None if tokens is None else tokens.numpy(), n_top, scale)
    if n_top:
        assert np.array_equal(got[3].cpu().numpy(), want[3])
    else:
        assert got[3] is None and got[4] is None
    N = l.shape[1] / 512 + 3 * 18 + 40
    log_s = np.log1p(rest)
    for i in (0, 1, 2, 4):
        if got[i] is None:
            assert want[i] is None or i == 4
            continue
        g, w = got[i].double().cpu().numpy(), want[i]
        fine = np.isfinite(w)
        assert np.array_equal(np.isnan(g), np.isnan(w)) and np.array_equal(g[~fine & ~np.isnan(w)], w[~fine & ~np.isnan(w)])
        of = log_s if i in (1, 2) else log_s[:, None]
        if i == 1:
            bound = UNIT * ((N + 2) * of + 2 * np.abs(w) + 1e-30)
        elif i == 2:
            bound = UNIT * 2 * (N + 4) * np.abs(w) + 1e-37
        else:
            bound = UNIT * ((N + 2) * of + 4 * np.abs(w) + 1e-30)
        err = np.abs(g - w)
        bound = np.broadcast_to(bound, w.shape)
        assert (err[fine] <= bound[fine]).all(), (i, (err[fine] / bound[fine]).max())
    return got


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [1, 2, 7, 33, 500, 1000, 4097, 32000, 151936])
@pytest.mark.parametrize("n,given,n_top", [(1, 1, 20), (3, 2, 5), (2, 0, 32), (2, 3, 0), (170, 1, 1)])
def test_against_64_bits(lib, dtype, V, n, given, n_top):
    if n > 100 and V > 5000:
        V = 5001
    g = torch.Generator().manual_seed(V + n)
    logits = (3 * torch.randn(n, V, generator=g)).to(dtype).cuda()
    tokens = torch.randint(0, V, (n, given), generator=g, dtype=torch.int32) if given else None
    check(logits, tokens, n_top)
    check(logits, tokens, n_top, 0.6)
    assert lib.get_device_error() == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [1, 40, 200])
def test_nearly_certain_rows(lib, dtype, n):
    """The largest logit well ahead: log probabilities and entropies near 0 keep their digits."""
    g = torch.Generator().manual_seed(n)
    V = 20011
    logits = (2 * torch.randn(n, V, generator=g)).to(dtype)
    at = torch.randint(0, V, (n,), generator=g)
    ahead = torch.linspace(9, 60, n)
    logits[torch.arange(n), at] = ahead.to(dtype)
    tokens = torch.stack([at, (at + 1) % V], 1).to(torch.int32)
    logp, lse, entropy, ids, top = check(logits.cuda(), tokens, 3)
    assert torch.equal(ids[:, 0].cpu(), at.to(torch.int32)) and (logp[:, 0] < 0).all() and (entropy > 0).all()


@pytest.mark.parametrize("dtype", DT)
def test_ties_and_orders(lib, dtype):
    V = 9001
    t = torch.zeros(8, V)
    t[1] = torch.arange(V) / 64            # rising: the list lies in one place
    t[2] = -torch.arange(V) / 64
    t[3, 4000:4100] = 5                    # more equal ones than the list takes
    t[4, ::3] = 1
    t[5, 8999] = -0.0                      # equal to 0
    t[6] = torch.arange(V) % 2 * 1.0
    t[7] = -7.5
    t = t.to(dtype).cuda()
    for k in (1, 5, 32):
        got = check(t, None, k)
        assert got[3][0].tolist() == list(range(k)) and got[3][3].tolist() == list(range(4000, 4000 + k))
    big = torch.zeros(2, 151936, dtype=dtype, device="cuda")  # shared memory does not hold the candidates
    big[1, 100000:] = 2
    got = check(big, None, 20)
    assert got[3].tolist() == [list(range(20)), list(range(100000, 100020))]


@pytest.mark.parametrize("dtype", DT)
def test_masks_and_odd_values(lib, dtype):
    inf, V = float("inf"), 3001
    low = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(3)
    t = torch.randn(12, V, generator=g)
    t[0] = -inf                         # nothing left
    t[1, 7:] = -inf                     # fewer than the list takes
    t[2, :2990] = -inf
    t[3] = low                          # all of the type's lowest value: uniform
    t[4, 5:] = low
    t[5, 100] = float("nan")
    t[6] = float("nan")
    t[7, 100] = inf
    t[8] = -inf
    t[8, 2000] = float("nan")           # a NaN among masks
    t[9] = -inf
    t[9, 3000] = 4.0                    # one token left
    t[10] = torch.finfo(dtype).max
    t[11, ::2] = -inf
    t = t.to(dtype).cuda()
    tokens = torch.tensor([[0, 3000, -1]] * 12, dtype=torch.int32)
    for k in (0, 4, 32):
        got = check(t, tokens, k)
        assert got[2][0] == 0 and got[2][9] == 0 and got[0][9, 1] == 0 and (got[0][:, 2] == 0).all()
    assert lib.get_device_error() == 0
    api.logprobs(t, torch.full((12, 1), V, dtype=torch.int32).cuda())
    assert lib.get_device_error() == api.DEVERR_TOKEN


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V,ld,off", [(1003, 1003, 0), (1003, 1009, 0), (5000, 5001, 8), (151937, 151939, 0), (700, 705, 3), (40, 40, 1)])
def test_rows_of_any_alignment(lib, dtype, V, ld, off):
    g = torch.Generator().manual_seed(V)
    buf = torch.full((off + 9 * ld,), float("nan"), dtype=dtype, device="cuda")  # what lies between rows is not looked at
    view = buf[off:off + 9 * ld].view(9, ld)[:, :V] if ld > V else buf[off:].view(9, ld)
    view.copy_((2 * torch.randn(9, V, generator=g)).to(dtype))
    tokens = torch.randint(0, V, (9, 2), generator=g, dtype=torch.int32)
    check(view, tokens, 7)


@pytest.mark.parametrize("n", [1, 2, 19, 38, 76, 153, 305])
def test_every_division_of_a_row_gives_the_definition(lib, n):
    """One to eight CTAs a row, by the number of rows; the same row in each call agrees within the tolerance."""
    g = torch.Generator().manual_seed(9)
    row = 3 * torch.randn(1, 50000, generator=g)
    logits = row.repeat(n, 1).cuda()
    logp, lse, entropy, ids, top = api.logprobs(logits, torch.full((n, 1), 77, dtype=torch.int32).cuda(), 32)
    for t in (logp, lse, entropy, ids, top):
        assert torch.equal(t, t[:1].expand_as(t))
    check(logits[:1], torch.tensor([[77]], dtype=torch.int32), 32)
    again = api.logprobs(logits, torch.full((n, 1), 77, dtype=torch.int32).cuda(), 32)
    assert all(torch.equal(a, b) for a, b in zip((logp, lse, entropy, ids, top), again))


def test_extreme_scales(lib):
    t = torch.tensor([[0.0, 1e-30, -5.0, 3e38, -3e38], [1.0, 1.0, 1.0, 0.5, 1.0]], device="cuda")
    tokens = torch.tensor([[0, 3], [3, 1]], dtype=torch.int32)
    for scale in (1e-30, 1e-6, 1e20, 8e37):
        got = api.logprobs(t, tokens.cuda(), 2, scale)
        want = step_ref.logprobs(t.double().cpu().numpy(), tokens.numpy(), 2, float(np.float32(scale)))
        assert np.array_equal(got[3].cpu().numpy(), want[3])
        for g, w in zip(got[:3], want[:3]):
            w = np.where(np.abs(w) > 3.4028235e38, np.sign(w) * np.inf, w)  # (fp32 has no more)
            assert np.allclose(g.double().cpu().numpy(), w, rtol=1e-5, atol=1e-30)


def test_only_what_is_asked_for(lib):
    t = torch.randn(3, 100, device="cuda")
    logp, lse, entropy, ids, top = api.logprobs(t)
    assert logp is None and ids is None and top is None and lse.shape == entropy.shape == (3,)
    outs = dict(lse=torch.empty(3, device="cuda"), entropy=torch.empty(3, device="cuda"),
                ids=torch.empty(3, 2, dtype=torch.int32, device="cuda"), top=torch.empty(3, 2, device="cuda"))
    got = api.logprobs(t, n_top=2, **outs)
    assert got[1].data_ptr() == outs["lse"].data_ptr() and torch.equal(got[1], lse) and torch.equal(got[2], entropy)
    assert got[3].data_ptr() == outs["ids"].data_ptr() and got[4].data_ptr() == outs["top"].data_ptr()


def test_offsets_past_32_bits(lib):
    V, n = 200000, 12000  # 2.4e9 values
    logits = torch.zeros(n, V, dtype=torch.float16, device="cuda")
    logits[-1, 199999] = 12.0
    logp, lse, entropy, ids, top = api.logprobs(logits, torch.full((n, 1), 199999, dtype=torch.int32).cuda(), 2)
    assert ids[-1].tolist() == [199999, 0] and ids[0].tolist() == [0, 1]
    check(logits[-1:], torch.tensor([[199999]], dtype=torch.int32), 2)
    want = -np.log(V)
    assert (logp[:-1].double() - want).abs().max() <= 2.0 ** -24 * 300 * abs(want)
