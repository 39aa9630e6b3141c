"""Norm rows at the edges of its arithmetic."""
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
