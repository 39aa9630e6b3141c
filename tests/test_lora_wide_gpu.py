"""Adapters of very wide projections, whose columns take more splits than are chosen
from, against 64 bits and in their buffers.

Tolerance, in units of 2^-24 of |scale| sum |B| sum |A x|, from the real division: a lane
adds 8 products for each of its windows of 256 columns, 5 steps over lanes, one addition a
split, the scale 1; then 8 products, 5 steps; and one unit of y."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import step_ref
from tests.test_canary_gpu import Guarded
from tests.test_debug_gpu import both, same_bits

pytestmark = pytest.mark.gpu

# columns, rows, rank, tokens, splits: at 64 tokens from 18433 columns on, at any number from 32769 on
CASES = [(20488, 300, 8, 64, 11), (18432, 65, 4, 64, 9), (32768, 40, 12, 33, 16), (32776, 40, 12, 33, 17), (40008, 129, 16, 1, 20),
         (40008, 70, 64, 33, 20), (1 << 20, 33, 4, 3, 512), (1 << 20, 8, 128, 64, 512)]


def case(K, M, r, n, dtype, adapters):
    g = torch.Generator(device="cuda").manual_seed(K + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    A, B = (rnd(adapters, r, K) / K ** 0.5).to(dtype), (rnd(adapters, M, r) / r ** 0.5).to(dtype)
    scales = torch.rand(adapters, generator=g, device="cuda") + 0.5
    ranks = torch.tensor([max(1, r - i) for i in range(adapters)], dtype=torch.int32).cuda()
    ids = torch.tensor([(5 * i) % (adapters + 1) - 1 if n > 1 else 0 for i in range(n)], dtype=torch.int32).cuda()
    return api.lora(A, B, scales, ranks), ids, rnd(n, K), rnd(n, M)


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("K,M,r,n,splits", CASES)
def test_wide_projections(lib, dtype, K, M, r, n, splits):
    d, ids, x, res = case(K, M, r, n, dtype, 3 if r < 100 else 1)
    assert api.lora_workspace_bytes(d, n) == splits * n * r * 4
    y, ws = Guarded((n, M), torch.float32, 1), Guarded((splits * n * r * 4,), torch.uint8, 2)
    ws.t.fill_(0xFF)  # (NaN where it is not written)
    api.lora_run(d, ids, x, res, out=y.t, ws=ws.t)
    y.check_guards("y")
    ws.check_guards("ws")
    A, B, ranks, scales = d._tensors
    some = sorted(set(range(0, n, 1 if K * r < 1 << 23 else 16)) | {n - 1})  # (all but the largest case's)
    want, mag = step_ref.lora(f64(A), f64(B), [int(ids[t]) for t in some], f64(x[some]), f64(res[some]), f64(scales), ranks.tolist())
    windows = -(-(-(-K // 256)) // splits)
    units = 8 * windows + 5 + splits + 1 + 8 + 5
    err = np.abs(f64(y.t[some]) - want)
    bound = 2.0 ** -24 * (units * mag + np.abs(want)) + 1e-37
    assert (err <= bound).all(), (err / bound).max()
    # the same bits from the same call, in place, and for a token in other company
    assert same_bits(api.lora_run(d, ids, x, res), y.t)
    back = api.lora_run(d, ids.flip(0).contiguous(), x.flip(0).contiguous(), res.flip(0).contiguous())
    assert same_bits(back.flip(0), y.t)
    assert lib.get_device_error() == 0


def test_range_checked_build_gives_the_same_bits(lib):
    def run():
        out = []
        for K, M, r, n, _ in CASES:
            d, ids, x, res = case(K, M, r, n, torch.bfloat16, 2 if r < 100 else 1)
            out.append(api.lora_run(d, ids, x, res))
        return out

    rel, dbg, err = both(api.load_debug(), run)
    assert err == 0 and all(same_bits(a, b) for a, b in zip(rel, dbg))
