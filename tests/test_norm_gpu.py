"""Root-mean-square norm with residual and 8-bit output against 64 bits.

Tolerance: with every operation rounded once in fp32, s = x + r is off by at
most 2^-24 of itself, a sum of at most 32 terms a thread and 10 levels of
pairwise sums by 42 * 2^-24, its root by half of that, and the division, root
and two products by 2^-24 each: |y - y64| <= 32 * 2^-24 |y64|, plus half a unit
of the output's type.  The 8-bit output is checked bit for bit as the
activation rule applied to the fp32 y that the same call returns."""
import numpy as np
import pytest
import torch

import oracle
from moe_matvec_gb300 import api

pytestmark = pytest.mark.gpu

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-38, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38}
DT = list(UNIT)


def make(n, K, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(n, K, generator=g) * scale).to(dtype).cuda()
    r = (torch.randn(n, K, generator=g) * 2 * scale).to(dtype).cuda()
    w = (1 + 0.2 * torch.randn(K, generator=g)).cuda()
    return x, r, w


def ref(x, r, w, eps):
    s = x.double().cpu().numpy()
    if r is not None:
        s = s + r.double().cpu().numpy()
    y = s / np.sqrt(np.mean(s * s, -1, keepdims=True) + eps) * w.double().cpu().numpy()
    return s, y


def check(got, want, dtype, rel):
    got = got.double().cpu().numpy()
    bound = (rel + UNIT[dtype]) * np.abs(want) + TINY[dtype]
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,K", [(1, 1), (1, 7), (3, 8), (2, 31), (5, 33), (1, 256), (64, 256), (700, 64), (300, 100),
                                 (2, 1000), (7, 2048), (3, 5120), (2, 8192), (2, 8200), (1, 8193), (2, 16384),
                                 (1, 32768), (1, 32765)])
def test_norm_values(lib, dtype, n, K):
    x, r, w = make(n, K, dtype, 10 + n + K)
    for res_in in (None, r):
        y, q8, res = api.rms_norm(x, w, 1e-5, r=res_in)
        s64, y64 = ref(x, res_in, w, 1e-5)
        check(y, y64, dtype, 32 * 2.0 ** -24)
        assert q8 is None
        if res_in is None:
            assert res is None
        else:
            check(res, s64, dtype, 2.0 ** -24)
    assert lib.get_device_error() == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,K", [(1, 256), (3, 512), (64, 4096), (200, 768), (2, 5120), (5, 8192), (1, 8448), (2, 32768)])
def test_q8_output_is_the_activation_rule_of_y(lib, dtype, n, K):
    x, r, w = make(n, K, dtype, 20 + n + K, 3.0)
    x32, r32 = x.float(), r.float()
    y, (q, d, s), _ = api.rms_norm(x32, w, 1e-6, r=r32, want="both")
    qo, do, so = oracle.act_quant(y.cpu().numpy())
    nat = q.cpu().numpy().reshape(n, K // 256, 2, 8, 16).transpose(0, 1, 3, 2, 4).reshape(n, K)
    assert np.array_equal(nat, qo.reshape(n, K))
    assert np.array_equal(d.cpu().numpy().view(np.uint32), do.reshape(n, -1).view(np.uint32))
    assert np.array_equal(s.cpu().numpy(), so.reshape(n, -1))
    # the same s in another type gives the same codes; q8 alone gives the same as both
    y2, q2, _ = api.rms_norm(x, w, 1e-6, r=r, want="q8")
    assert y2 is None and all(torch.equal(a, b) for a, b in zip(q2, (q, d, s)))
    for t in DT:
        back = api.dequantize_act(q, d, t)
        want = torch.from_numpy(nat.astype(np.float32) * np.repeat(do.reshape(n, -1), 32, 1)).to(t)
        assert torch.equal(back.cpu(), want)
    if n <= 64:
        from moe_matvec_gb300 import synth
        W = api.quantize_weights(0, torch.from_numpy(synth.weights(5, 40, K)).cuda())
        assert torch.equal(api.run_q8(0, W, q, d, s, 40, K), api.run(0, W, y, 40, K))


def test_rows_may_be_strided_and_results_in_place(lib):
    big = torch.randn(6, 5 * 512, device="cuda")
    w = torch.rand(512, device="cuda") + 0.5
    x = big[:, 512:1024]
    r = torch.randn(6, 512, device="cuda")
    want = api.rms_norm(x.contiguous(), w, r=r, want="both")
    before = big.clone()
    r2 = r.clone()
    y, q8, res = api.rms_norm(x, w, r=r2, res=r2, want="both")
    assert res.data_ptr() == r2.data_ptr() and torch.equal(res, want[2]) and torch.equal(y, want[0])
    assert all(torch.equal(a, b) for a, b in zip(q8, want[1]))
    assert torch.equal(big, before)
    # rows whose stride allows no wide loads take single ones
    odd = torch.randn(4, 515, device="cuda")
    y = api.rms_norm(odd[:, :512], w)[0]
    assert torch.allclose(y, api.rms_norm(odd[:, :512].contiguous(), w)[0], rtol=1e-5, atol=1e-6)


def test_zero_rows_large_and_small_values(lib):
    w = torch.ones(512, device="cuda")
    x = torch.zeros(4, 512, device="cuda")
    x[1] = 1e-20
    x[2] = 1e15
    x[3, 5] = 3.0
    y, (q, d, s), _ = api.rms_norm(x, w, 1e-6, want="both")
    _, y64 = ref(x, None, w, 1e-6)
    check(y, y64, torch.float32, 32 * 2.0 ** -24)
    assert (q[0] == 0).all() and (d[0] == 0).all() and (s[0] == 0).all()


def test_another_stream(lib):
    x, r, w = make(64, 4096, torch.float32, 3)
    want = api.rms_norm(x, w, r=r, want="both")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = api.rms_norm(x, w, r=r, want="both")
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
