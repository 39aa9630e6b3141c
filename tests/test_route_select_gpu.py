"""Expert selection against 64 bits: picks equal; gates, in units of 2^-24 of the
gate: exp 2 ulp (4), the distance from the row's largest logit (its rounding, twice
as long as the sum is of such terms), the sum over 512 experts (16 + 5), reciprocal,
product, sum of 8 picks, division and scale (12), as bounds of every step: 48 + 2 |l - top|.
A score below 2^-126 may be 0, and the sum that divides it is at least 2^-60 (smaller
ones are formed in 64 bits): 2^-66 of the scale."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import step_ref

pytestmark = pytest.mark.gpu


def check(logits, top_k, gating, bias=None, groups=1, keep=1, group_top=2, renorm=True, scale=1.0):
    ids, gates = api.route_select(logits, top_k, gating, bias=bias, groups=groups, keep=keep, group_top=group_top,
                                  renorm=renorm, scale=scale)
    want, g, below = step_ref.route(logits.double().cpu().numpy(), top_k, gating == api.GATING_SIGMOID,
                                    None if bias is None else bias.double().cpu().numpy(), groups, keep, group_top, renorm,
                                    scale)
    assert ids.dtype is torch.int32 and gates.dtype is torch.float32
    assert np.array_equal(ids.cpu().numpy(), want)
    err = np.abs(gates.double().cpu().numpy() - g)
    bound = 2.0 ** -24 * (48 + 2 * below) * np.abs(g) + 2.0 ** -66 * abs(scale)
    assert (err <= bound).all(), (err / bound).max()
    return ids, gates


SHAPES = [(1, 1, 1, 1, 1), (8, 8, 1, 1, 1), (37, 3, 1, 1, 1), (128, 8, 1, 1, 1), (512, 8, 1, 1, 1), (256, 8, 8, 4, 2),
          (256, 6, 8, 3, 1), (160, 6, 8, 3, 2), (60, 4, 4, 1, 2), (100, 8, 5, 2, 2), (512, 8, 32, 5, 2), (72, 8, 9, 8, 2),
          (510, 8, 17, 2, 1), (34, 2, 17, 2, 2), (32, 4, 32, 4, 1), (510, 5, 3, 2, 2), (96, 8, 1, 1, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gating", [0, 1])
@pytest.mark.parametrize("E,k,G,keep,top", SHAPES)
def test_against_64_bits(lib, dtype, gating, E, k, G, keep, top):
    g = torch.Generator().manual_seed(E + k)
    logits = (2 * torch.randn(67, E, generator=g)).to(dtype).cuda()
    bias = (0.3 * torch.randn(E, generator=g)).cuda()
    check(logits, k, gating, bias, G, keep, top, True, 2.5)
    check(logits, k, gating, None, G, keep, top, False, 1.0)
    assert lib.get_device_error() == 0


@pytest.mark.parametrize("n", [1, 3, 4, 5, 16384])
def test_token_counts(lib, n):
    g = torch.Generator().manual_seed(n)
    logits = torch.randn(min(n, 700), 64, generator=g).repeat(-(-n // 700), 1)[:n].contiguous().cuda()
    bias = (0.1 * torch.randn(64, generator=g)).cuda()
    few = api.route_select(logits[:700], 6, 1, bias=bias, groups=4, keep=2)
    all_ = api.route_select(logits, 6, 1, bias=bias, groups=4, keep=2)
    check(logits[:700], 6, 1, bias, 4, 2)
    for a, b in zip(few, all_):
        assert torch.equal(a, b[:700])
        assert torch.equal(b[-1], b[(n - 1) % 700])
    with pytest.raises(api.QmvError):
        api.route_select(logits[:1].expand(16385, 64), 6)


@pytest.mark.parametrize("gating", [0, 1])
def test_scores_that_fp32_cannot_tell_apart(lib, gating):
    """Logits and biases whose scores differ by about 2^-30 at every border."""
    rng = np.random.default_rng(5)
    n, E = 300, 64
    l = rng.integers(-8, 8, (n, E)) / 4.0
    base = 1 / (1 + np.exp(-l[0])) if gating else np.exp(l[0] - l[0].max()) / np.exp(l[0] - l[0].max()).sum()
    logits = np.tile(l[0], (n, 1)).astype(np.float32)
    # biases that bring every score of row 0 to 0.75 but for a few ulp
    bias = (0.75 - base).astype(np.float32)
    logits += (rng.integers(-2, 3, (n, E)) * 2.0 ** -22).astype(np.float32)
    t, b = torch.from_numpy(logits).cuda(), torch.from_numpy(bias).cuda()
    check(t, 8, gating, b)
    check(t, 8, gating, b, 8, 3, 2)
    check(t, 8, gating, b, 8, 3, 1)
    check(t, 8, gating, None, 8, 3, 2)


@pytest.mark.parametrize("gating", [0, 1])
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
def test_ties_go_to_the_lower_index(lib, gating, bias):
    b = None if bias is None else torch.full((96,), bias).cuda()
    t = torch.zeros(5, 96, device="cuda")
    t[1, 90:] = 1
    t[2] = -0.0
    t[2, 40] = 0.0
    ids, gates = check(t, 8, gating, b)
    assert ids[0].tolist() == list(range(8)) and ids[1].tolist() == [90, 91, 92, 93, 94, 95, 0, 1]
    assert ids[2].tolist() == list(range(8)) and (gates[0] == 1 / 8).all()
    ids, _ = check(t, 8, gating, b, 12, 2)
    assert ids[0].tolist() == list(range(8))


@pytest.mark.parametrize("gating", [0, 1])
def test_masked_and_odd_logits(lib, gating):
    inf = float("inf")
    g = torch.Generator().manual_seed(gating)
    t = torch.randn(8, 32, generator=g).cuda()
    t[0] = -inf                      # nothing left: gates 0, distinct picks
    t[1, 3:] = -inf                  # fewer than top_k left
    t[2, 5] = float("nan")
    t[3] = float("nan")
    t[4, 7] = inf
    t[5] = torch.finfo(torch.float32).min
    t[6, ::2] = torch.finfo(torch.float32).min
    t[7] = torch.linspace(-90, 90, 32)
    wide = torch.arange(32) * 1.0  # picks whose scores are next to nothing
    for b in (None, torch.zeros(32).cuda(), torch.randn(32, generator=g).cuda(), wide.cuda(), -wide.cuda()):
        ids, gates = check(t, 5, gating, b)
        assert torch.isfinite(gates).all() and (gates[0] == 0).all() and (gates[3] == 0).all()
        check(t, 5, gating, b, 4, 2, 2)
        check(t, 5, gating, b, 4, 2, 1, False, 3.0)
    out = torch.zeros(32, device="cuda")
    out[4:] = -inf                   # experts behind all others
    out[9] = float("nan")
    ids, _ = check(t[7:], 6, gating, out)
    assert ids[0].tolist()[:4] == [3, 2, 1, 0]
    check(t, 8, gating, out, 8, 3, 2)
    # experts out of use by a low bias: in whole groups, and all but one of a group
    for low in (-inf, -1e9, torch.finfo(torch.float32).min):
        some = 0.1 * torch.randn(32, generator=g).cuda()
        some[12:] = low
        for one in (None, 13):
            if one:
                some[one] = 0.2
            for keep, top in ((3, 2), (4, 2), (4, 1), (5, 2)):
                ids, _ = check(t, 8, gating, some, 8, keep, top)
            check(t, 8, gating, some)


@pytest.mark.parametrize("gating", [0, 1])
@pytest.mark.parametrize("E,G,keep,top", [(64, 8, 3, 2), (64, 8, 3, 1), (512, 1, 1, 1), (510, 17, 5, 2), (300, 2, 1, 2)])
def test_large_biases(lib, gating, E, G, keep, top):
    # up to 2^30: scores count for nothing beside some, for all beside others, and pairs cancel
    g = torch.Generator().manual_seed(E + G + gating)
    logits = (2 * torch.randn(200, E, generator=g)).cuda()
    bias = (2.0 ** torch.randint(-4, 31, (E,), generator=g)) * (torch.randint(0, 2, (E,), generator=g) * 2 - 1)
    check(logits, 8, gating, bias.cuda(), G, keep, top)
    check(logits, 8, gating, (bias / 2.0 ** 20).cuda(), G, keep, top)
    check(logits, 8, gating, bias.sign().cuda() * 2.0 ** 22, G, keep, top)


def test_strided_rows_and_given_results(lib):
    big = torch.randn(20, 300, device="cuda")
    view = big[:, 4:4 + 129]
    ids, gates = torch.empty(20, 4, dtype=torch.int32, device="cuda"), torch.empty(20, 4, device="cuda")
    got = api.route_select(view, 4, 1, ids=ids, gates=gates)
    assert got[0].data_ptr() == ids.data_ptr() and got[1].data_ptr() == gates.data_ptr()
    want = api.route_select(view.contiguous(), 4, 1)
    assert torch.equal(ids, want[0]) and torch.equal(gates, want[1])


def test_it_agrees_with_the_router_and_feeds_the_experts(lib):
    E, H, F, n, k = 16, 512, 256, 12, 4
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    Wr = api.quantize_weights(api.Q8_0, rnd(E, H) * 0.05)
    x = rnd(n, H)
    for gating in (0, 1):
        ids, gates, logits = api.route_run(api.Q8_0, Wr, x, E, H, k, gating)
        mine = api.route_select(logits, k, gating)
        assert torch.equal(ids, mine[0])
        assert ((gates - mine[1]).abs() <= 2.0 ** -18 * gates).all()
    wg = torch.stack([api.quantize_weights(api.Q4_K, rnd(2 * F, H) * 0.02) for _ in range(E)])
    wd = torch.stack([api.quantize_weights(api.Q4_K, rnd(H, F) * 0.02) for _ in range(E)])
    ex = api.moe_experts(E, H, F, api.Q4_K, api.Q4_K, wg, wd)
    ids, gates = api.route_select(logits, k, 1, bias=rnd(E) * 0.1, groups=4, keep=2, scale=2.5)
    assert torch.isfinite(api.moe_run(ex, ids, gates, x)).all()
    assert lib.get_device_error() == 0
