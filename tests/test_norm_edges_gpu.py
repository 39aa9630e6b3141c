"""Norm rows at the edges of its arithmetic."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]


def bits(t):
    """The tensor's bits; every NaN as the same ones."""
    return torch.where(t.isnan(), torch.nan, t).contiguous().view(torch.int32)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("K", [256, 512, 5120, 32768])
def test_codes_of_what_is_no_number(lib, dtype, K):
    # a zero row without eps, a NaN or an infinity in x, a NaN in w: the activation
    # rule's codes of y, as the library's quantizer makes them (0 for a NaN)
    x = torch.randn(6, K, generator=torch.Generator().manual_seed(K)).to(dtype).cuda()
    w = torch.ones(K, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, K - 1] = float("inf")
    for weights in (w, torch.where(torch.arange(K, device="cuda") == 77, torch.nan, w)):
        y, (q, d, s), _ = api.rms_norm(x.float(), weights, 0.0, want="both")
        assert y[1].isnan().all() and y[2].isnan().all() and y[3, K - 1].isnan()
        q2, d2, s2 = api.quantize_act(y)
        assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(bits(d), bits(d2))
        assert (q[1:3] == 0).all() and (s[1:3] == 0).all()
        alone = api.rms_norm(x, weights, 0.0, want="q8")[1]
        assert torch.equal(alone[0], q) and torch.equal(alone[2], s) and torch.equal(bits(alone[1]), bits(d))


@pytest.mark.parametrize("K", [16640, 32768, 32765])
def test_one_large_value_and_many_small_ones(lib, K):
    # Squares just under half a unit in the last place of the running sum: summed one
    # after another into one register, every one of them is lost (64 terms a thread:
    # 31 * 2^-24 of y).  Partial sums of eight values keep them: at most 8 + 8 terms
    # a thread and 10 levels, half of 26 * 2^-24 from the sum; the reciprocal root is off
    # by up to 4 * 2^-24, division, eps and the two products by 3 in all.
    for first in range(8):
        x = torch.full((1, K), 0.995 * 2.0 ** -12, device="cuda")
        if K % 8 == 0:  # eight neighbours a thread and step
            x[0, first:4096:8] = 1
        else:  # a thread's values lie 512 apart
            x[0, first * 512:first * 512 + 512] = 1
        y = api.rms_norm(x, torch.ones(K, device="cuda"), 0.0)[0].double().cpu().numpy()
        s = x.double().cpu().numpy()
        want = s / np.sqrt((s * s).mean())
        assert (np.abs(y - want) <= 20 * 2.0 ** -24 * np.abs(want)).all()
