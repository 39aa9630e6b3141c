"""Sums of long rows, every division of a row, and extreme scales, against 64 bits.

Tolerance, with s the sum over the row but for its largest term, in units of 2^-24 of
s: a chain of at most min(V / 512, 512) additions before it is joined in 64 bits; a
term's exponent d (in powers of 2) is rounded three times and ex2 is 2 ulp off,
3 |d| + 4, which over the rows here is at most 16 on average; a sum that is rescaled
takes as much as a term, less each time by the factor (22 in all); the joins of lanes,
warps and CTAs 30: N = min(V / 512, 512) + 70.  log1p(s) is off by N s / (1 + s) and 2 ulp
of itself, the mean of |d| by 2 N of itself and by the part of s that it is relative
to (2 N s / (1 + s)), a log probability by the former and 2 units of its difference to the
largest; each has its own rounding."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import step_ref

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]
UNIT = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def within(what, got, want, bound):
    err = np.abs(got - want)
    assert (err <= bound).all(), (what, (err / bound).max(), np.argmax(err / bound))


def compare(V, logp, lse, entropy, diff, top, s, mean, more=0):
    """diff: the given tokens' distances from the largest logit (0 or less), top the largest
    (times the scale), s as above, mean: of the distances' magnitude; one entry a row."""
    N = min(V / 512, 512) + 70 + more
    log_s, part = np.log1p(s), s / (1 + s)
    sums = N * part + 2 * log_s
    want = top + log_s
    within("lse", f64(lse), want, UNIT * (sums + 2 * np.abs(want) + np.abs(top)))
    want = diff - log_s[:, None]
    within("logp", f64(logp), want, UNIT * (sums[:, None] + 2 * np.abs(diff) + np.abs(want)))
    want = log_s + mean
    within("entropy", f64(entropy), want, UNIT * (sums + 2 * N * (mean + part) + 10 * mean + 2 * want))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,log_v", [(1, 24), (1, 28), (100, 22), (160, 20), (160, 22), (160, 24)])
def test_long_rows_of_equal_terms(lib, dtype, rows, log_v):
    """One likely token, all others alike, another value in each row: equal terms, whose sum's
    roundings all go one way.  The likely one first, last or in between."""
    if rows == 1 and dtype is torch.float16:
        rows = 2
    V = 1 << log_v
    logits = torch.empty(rows, V, dtype=dtype, device="cuda")
    for seed in range(8 if rows <= 2 else 1):
        other = -((torch.arange(rows) + 5 * seed) % 32 + 1) / 16.0
        logits[:] = other.to(dtype)[:, None].cuda()
        at = torch.tensor([0, V - 1, V // 2 + 1, V // 3])[(torch.arange(rows) + seed) % 4]
        logits[torch.arange(rows), at] = 0.5
        tokens = torch.stack([at, (at + 1) % V], 1).to(torch.int32)
        logp, lse, entropy, ids, _ = api.logprobs(logits, tokens.cuda(), 1 if log_v <= 22 else 0)
        d = other.double().numpy() - 0.5
        s = (V - 1) * np.exp(d)
        compare(V, logp, lse, entropy, np.stack([np.zeros(rows), d], 1), np.full(rows, 0.5), s, -d * s / (1 + s))
        if ids is not None:
            assert torch.equal(ids[:, 0].cpu(), at.to(torch.int32))
    assert lib.get_device_error() == 0


@pytest.mark.parametrize("rows", [1, 160])
def test_rows_that_rise_slowly(lib, rows):
    """The largest logit so far grows at every step of the sums: ex2, 4 units, for each of
    the 64 rescalings (of 8 terms a step) before a sum is joined in 64 bits."""
    V, levels = 1 << 24, 4096
    step = torch.arange(1, rows + 1, dtype=torch.float32) * 2.0 ** -18
    logits = (torch.arange(levels, dtype=torch.float32).cuda()[None] * step.cuda()[:, None]).repeat_interleave(V // levels, 1)
    tokens = torch.tensor([[0, V - 1]] * rows, dtype=torch.int32)
    logp, lse, entropy, _, _ = api.logprobs(logits, tokens.cuda())
    d = (np.arange(levels) - levels + 1.0)[None] * step.double().numpy()[:, None]
    n = np.full(levels, V // levels)
    n[-1] -= 1
    s, t = (n * np.exp(d)).sum(1), (n * np.exp(d) * -d).sum(1)
    compare(V, logp, lse, entropy, d[:, [0, -1]], (levels - 1) * step.double().numpy(), s, t / (1 + s), 4 * 64)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [1, 2, 19, 38, 76, 153, 305])
def test_every_division_of_a_row(lib, n, dtype):
    """One to eight CTAs a row, by the number of rows: what each of them gives."""
    V, k = 50000, 32
    g = torch.Generator().manual_seed(9)
    row = (3 * torch.randn(1, V, generator=g)).to(dtype)
    tokens = torch.tensor([[77, V - 1, 0]], dtype=torch.int32)
    logp, lse, entropy, ids, top = api.logprobs(row.repeat(n, 1).cuda(), tokens.repeat(n, 1).cuda(), k)
    for t in (logp, lse, entropy, ids, top):
        assert torch.equal(t, t[:1].expand_as(t))
    _, _, want_h, want_ids, want_top, s = step_ref.logprobs(f64(row), tokens.numpy(), k, 1.0)
    assert np.array_equal(ids[:1].cpu().numpy(), want_ids)
    l, order = f64(row)[0], np.concatenate([tokens.numpy()[0], want_ids[0]])
    log_s = np.log1p(s)
    compare(V, torch.cat([logp, top], 1)[:1], lse[:1], entropy[:1], (l[order] - l.max())[None], l.max(), s, want_h - log_s)


def test_the_top_list_at_extreme_scales(lib):
    t = torch.tensor([[0.0, 1e-30, -5.0, 3e38, -3e38], [1.0, 1.0, 1.0, 0.5, 1.0], [-3e38, 3e38, 3e38, -1.0, 2.0]], device="cuda")
    for scale in (1e-30, 1e-6, 1.0, 1e20, 8e37):
        _, _, _, ids, top = api.logprobs(t, n_top=5, scale=scale)
        want = step_ref.logprobs(f64(t), None, 5, float(np.float32(scale)))
        assert np.array_equal(ids.cpu().numpy(), want[3])
        w = want[4]
        w = np.where(np.abs(w) > 3.4028235e38, np.sign(w) * np.inf, w)  # (fp32 has no more)
        assert np.allclose(f64(top), w, rtol=1e-5, atol=1e-30), scale
