"""Adapters against 64 bits.

Tolerance, in units of 2^-24 of |scale| sum |B| sum |A x|: a lane adds 8 products
for each of its windows of 256 columns (16 splits at most: 8 ceil(K / 4096)), 5 steps
over lanes, 16 splits, the scale 1; then 8 products, 5 steps; and one unit of y."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import step_ref

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]


def pool(seed, n, r, K, M, dtype, scaled=True, ranked=True):
    g = torch.Generator().manual_seed(seed)
    A = (torch.randn(n, r, K, generator=g) / K ** 0.5).to(dtype).cuda()
    B = (torch.randn(n, M, r, generator=g) / r ** 0.5).to(dtype).cuda()
    scales = (torch.rand(n, generator=g) + 0.5).cuda() if scaled else None
    ranks = torch.randint(0, r + 1, (n,), generator=g, dtype=torch.int32).cuda() if ranked else None
    return api.lora(A, B, scales, ranks), A, B, scales, ranks


def check(y, A, B, ids, x, r, scales, ranks):
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want, mag = step_ref.lora(f(A), f(B), ids, f(x), f(r), f(scales), None if ranks is None else ranks.tolist())
    units = 8 * -(-A.shape[2] // 4096) + 5 + 16 + 1 + 8 + 5
    err = np.abs(y.double().cpu().numpy() - want)
    bound = 2.0 ** -24 * (units * mag + np.abs(want)) + 1e-37
    assert (err <= bound).all(), (err / bound).max()


def run(d, ids, x, r, **kw):
    return api.lora_run(d, torch.tensor(ids, dtype=torch.int32).cuda(), x, r, **kw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("K,M,r", [(8, 1, 4), (256, 64, 16), (264, 130, 8), (1000, 333, 12), (2048, 777, 64), (520, 1025, 128),
                                   (4104, 96, 20), (5120, 200, 32), (17408, 40, 8)])
@pytest.mark.parametrize("n", [1, 5, 8, 32, 33, 64])
def test_against_64_bits(lib, dtype, K, M, r, n):
    d, A, B, scales, ranks = pool(K + M + n, 7, r, K, M, dtype)
    rng = np.random.default_rng(n)
    ids = rng.integers(-1, 7, n).tolist()
    x, res = torch.randn(n, K).cuda(), torch.randn(n, M).cuda()
    check(run(d, ids, x, res), A, B, ids, x, res, scales, ranks)
    assert lib.get_device_error() == 0


@pytest.mark.parametrize("ids", [[0] * 64, list(range(64)), [3] * 5 + [-1] * 9 + [3] * 5 + [2], [-1] * 10, [63],
                                 [0, 1] * 32, [5] * 3 + [6] * 4 + [7] * 8 + [8] * 9])
def test_groups_of_tokens(lib, ids):
    d, A, B, _, _ = pool(1, 64, 16, 512, 300, torch.bfloat16, False, False)
    x, res = torch.randn(len(ids), 512).cuda(), torch.randn(len(ids), 300).cuda()
    y = run(d, ids, x, res)
    check(y, A, B, ids, x, res, None, None)
    # in place, and each token as it would be alone with other company
    inplace = res.clone()
    assert torch.equal(run(d, ids, x, inplace, out=inplace), y)
    back = run(d, ids[::-1], x.flip(0).contiguous(), res.flip(0).contiguous())
    assert torch.equal(back.flip(0), y)
    assert lib.get_device_error() == 0


def test_ids_past_the_pool_go_without(lib):
    d, A, B, scales, ranks = pool(2, 3, 8, 64, 50, torch.float16)
    ids = [0, 3, 2**31 - 1, -2**31, 1]
    x, res = torch.randn(5, 64).cuda(), torch.randn(5, 50).cuda()
    y = run(d, ids, x, res)
    check(y, A, B, ids, x, res, scales, ranks)
    assert torch.equal(y[1:4], res[1:4])
    assert lib.get_device_error() == api.DEVERR_ADAPTER


def test_unused_ranks_are_not_looked_at(lib):
    # what lies past an adapter's rank may be anything
    d, A, B, scales, _ = pool(3, 4, 16, 128, 70, torch.bfloat16, True, False)
    ranks = torch.tensor([0, 1, 9, 16], dtype=torch.int32)
    for a, k in enumerate(ranks.tolist()):
        A[a, k:] = float("nan")
        B[a, :, k:] = float("inf")
    d = api.lora(A, B, scales, ranks.cuda())
    ids = [0, 1, 2, 3, 2]
    x, res = torch.randn(5, 128).cuda(), torch.randn(5, 70).cuda()
    y = run(d, ids, x, res)
    assert torch.isfinite(y).all()
    check(y, A.nan_to_num(0, 0, 0), B.nan_to_num(0, 0, 0), ids, x, res, scales, ranks)
    odd = torch.tensor([-3, 40, 9, 16], dtype=torch.int32)  # clamped to 0 and 16
    A2, B2 = torch.randn(4, 16, 128).bfloat16().cuda(), torch.randn(4, 70, 16).bfloat16().cuda()
    d = api.lora(A2, B2, None, odd.cuda())
    check(run(d, ids, x, res), A2, B2, ids, x, res, None, odd)


def test_a_wide_projection(lib):
    # as many rows as take tiles of several steps, odd
    d, A, B, scales, ranks = pool(4, 40, 64, 512, 17409, torch.bfloat16)
    ids = [i % 40 for i in range(64)]
    x, res = torch.randn(64, 512).cuda(), torch.randn(64, 17409).cuda()
    check(run(d, ids, x, res), A, B, ids, x, res, scales, ranks)


def test_a_pool_past_32_bits(lib):
    # the last adapter's values begin past 2^31 elements
    K, M, r, n = 4096, 4096, 64, 8200
    A = torch.zeros(n, r, K, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(n, M, r, dtype=torch.bfloat16, device="cuda")
    A[-1], B[-1] = torch.randn(r, K) / 64, torch.randn(M, r) / 8
    d = api.lora(A, B)
    x, res = torch.randn(2, K).cuda(), torch.randn(2, M).cuda()
    y = run(d, [n - 1, 0], x, res)
    check(y[:1], A[-1:], B[-1:], [0], x[:1], res[:1], None, None)
    assert torch.equal(y[1], res[1])
