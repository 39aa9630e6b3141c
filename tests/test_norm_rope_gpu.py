"""Head norm and rotation against 64 bits.

Tolerance, in units of 2^-24 of the magnitude |a| + |b| of a pair's values (|u| for
values that do not turn): the sum of squares is a chain of at most 16 roundings and
5 additions over lanes, which the root halves (10.5); its mean and eps 1; rsqrtf 2
ulp (4), two products (2); the angle's fraction is rounded once, at most 2^-26 of a
turn (1.6); sincospif 2 ulp (4); scale 1; the pair's products and sum 2: 26.1, for
which 2^-19 (32 units) stands.  Then the result's own rounding, half a step."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests import step_ref

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]
TOL = 2.0 ** -19


def close(got, want, mag, dtype):
    half = torch.finfo(dtype).eps / 2
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    bound = TOL * mag + half * np.abs(want) * (1 + TOL) + torch.finfo(dtype).smallest_normal * half
    live = ~np.isnan(want)
    assert np.isfinite(got[live]).all() and (err[live] <= bound[live]).all(), np.nanmax((err / bound)[live])


def freqs(R, base=10000.0):
    return torch.exp(torch.arange(R // 2, dtype=torch.float64) * (-2 * np.log(base) / R)).float()


def case(seed, n, H, Hk, D, dtype, strided=True):
    g = torch.Generator().manual_seed(seed)
    if strided:
        pad = 0 if (H + 2 * Hk) * D * 2 % 16 == 0 else 1
        assert pad == 0
        qkv = (2 * torch.randn(n, H + 2 * Hk, D, generator=g)).to(dtype).cuda()
        q, k = qkv[:, :H], qkv[:, H:H + Hk]
    else:
        q = (2 * torch.randn(n, H, D, generator=g)).to(dtype).cuda()
        k = (2 * torch.randn(n, Hk, D, generator=g)).to(dtype).cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2)]
    return q, k, w


def check(out, x, w, eps, pos, axis, freq, inter, scale, dtype):
    want, mag = step_ref.norm_rope(x.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), eps, pos,
                                   axis, freq.double().numpy(), inter, scale)
    close(out, want, mag, dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,R,H,Hk", [(128, 128, 8, 2), (64, 64, 5, 1), (64, 32, 3, 3), (192, 64, 2, 1), (256, 256, 3, 2),
                                      (80, 80, 4, 1), (72, 40, 2, 2), (128, 2, 3, 1), (128, 90, 4, 4), (128, 92, 3, 1), (68, 36, 4, 2), (8, 6, 2, 1),
                                      (256, 254, 1, 1)])
def test_explicit_positions(lib, dtype, norm, inter, D, R, H, Hk):
    n = 7
    q, k, w = case(D + R, n, H, Hk, D, dtype)
    freq = freqs(R)
    pos = torch.tensor([0, 1, 17, 4095, 131071, 1000003, 2**31 - 1], dtype=torch.int32)
    r = api.rope(D, freq.cuda(), interleaved=inter)
    qo, ko = api.norm_rope(r, q, k, *(w if norm else (None, None)), 1e-5, pos=pos[:, None].contiguous().cuda())
    at = [[int(p)] for p in pos]
    for o, x, ww in ((qo, q, w[0]), (ko, k, w[1])):
        assert o.dtype is dtype and o.is_contiguous()
        check(o, x, ww if norm else None, 1e-5, at, [0] * (R // 2), freq, inter, 1.0, dtype)
    assert lib.get_device_error() == 0


@pytest.mark.parametrize("n", [1, 2, 33, 700])
@pytest.mark.parametrize("D,R,H,Hk,dtype", [(128, 128, 32, 8, torch.float32), (128, 64, 7, 1, torch.bfloat16),
                                            (72, 22, 5, 5, torch.float16)])
def test_one_token_a_sequence(lib, n, D, R, H, Hk, dtype):
    q, k, w = case(n, n, H, Hk, D, dtype)
    rng = np.random.default_rng(n)
    lens = rng.integers(1, 300000, n).astype(np.int32)
    freq = freqs(R, 500000.0)
    r = api.rope(D, freq.cuda(), scale=1.25)
    qo, ko = api.norm_rope(r, q, k, w[0], w[1], lens=torch.from_numpy(lens).cuda())
    at = [[int(t) - 1] for t in lens]
    check(qo, q, w[0], 1e-6, at, [0] * (R // 2), freq, False, 1.25, dtype)
    check(ko, k, w[1], 1e-6, at, [0] * (R // 2), freq, False, 1.25, dtype)


@pytest.mark.parametrize("dtype", DT)
def test_ragged_runs_and_padding(lib, dtype):
    # padding before, between the last sequence and n_tok, and an empty sequence
    starts, lens, n = [2, 5, 5, 60, 61], [3, 0, 1000, 77], 64
    q, k, w = case(3, n, 4, 2, 64, dtype)
    freq = freqs(64)
    r = api.rope(64, freq.cuda())
    qo, ko = (torch.full((n, h, 64), 7.0, dtype=dtype, device="cuda") for h in (4, 2))
    got = api.norm_rope(r, q, k, w[0], w[1], lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                        starts=torch.tensor(starts, dtype=torch.int32).cuda(), q_out=qo, k_out=ko)
    assert got[0].data_ptr() == qo.data_ptr() and got[1].data_ptr() == ko.data_ptr()
    at = step_ref.positions(lens, starts, n)
    at = [None if p is None else [p] for p in at]
    assert [p is None for p in at].count(True) == 5
    check(qo, q, w[0], 1e-6, at, [0] * 32, freq, False, 1.0, dtype)
    check(ko, k, w[1], 1e-6, at, [0] * 32, freq, False, 1.0, dtype)
    out = torch.tensor([p is None for p in at])
    assert (qo[out] == 7).all() and (ko[out] == 7).all()
    assert lib.get_device_error() == 0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_several_axes(lib, axes, inter):
    n, D, R = 50, 128, 96
    q, k, w = case(axes, n, 4, 1, D, torch.bfloat16)
    g = torch.Generator().manual_seed(axes)
    pos = torch.randint(-5, 40000, (n, axes), generator=g, dtype=torch.int32)
    axis = torch.randint(0, axes, (R // 2,), generator=g).to(torch.uint8)
    freq = freqs(R)
    r = api.rope(D, freq.cuda(), axis=axis.cuda(), n_axes=axes, interleaved=inter)
    qo, ko = api.norm_rope(r, q, k, w[0], None, pos=pos.cuda())
    check(qo, q, w[0], 1e-6, pos.tolist(), axis.tolist(), freq, inter, 1.0, torch.bfloat16)
    check(ko, k, None, 1e-6, pos.tolist(), axis.tolist(), freq, inter, 1.0, torch.bfloat16)
    # by lengths all axes are the same
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    starts = torch.tensor([0, n], dtype=torch.int32).cuda()
    one = api.norm_rope(r, q, k, lens=lens, starts=starts)
    same = api.norm_rope(r, q, k, pos=torch.arange(n, dtype=torch.int32)[:, None].repeat(1, axes).contiguous().cuda())
    assert torch.equal(one[0], same[0]) and torch.equal(one[1], same[1])
    assert lib.get_device_error() == 0


def test_in_place_on_the_fused_projection(lib):
    n, H, Hk, D = 9, 6, 2, 128
    qkv = torch.randn(n, H + 2 * Hk, D, device="cuda")
    before = qkv.clone()
    q, k, v = qkv.split((H, Hk, Hk), 1)
    r = api.rope(D, freqs(D).cuda())
    lens = torch.arange(5, 5 + n, dtype=torch.int32, device="cuda")
    want = api.norm_rope(r, q, k, lens=lens)
    got = api.norm_rope(r, q, k, lens=lens, q_out=q, k_out=k)
    assert torch.equal(qkv[:, :H], want[0]) and torch.equal(qkv[:, H:H + Hk], want[1])
    assert torch.equal(qkv[:, H + Hk:], before[:, H + Hk:]) and got[0].data_ptr() == qkv.data_ptr()
    alone, none = api.norm_rope(r, before[:, :H], lens=lens)  # queries alone
    assert none is None and torch.equal(alone, want[0])


def test_edges_of_values_and_contradictions(lib):
    r = api.rope(64, freqs(64).cuda())
    x = torch.zeros(3, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    pos = torch.arange(3, dtype=torch.int32, device="cuda")[:, None].contiguous()
    assert (api.norm_rope(r, x, None, w, pos=pos)[0] == 0).all()  # eps keeps a zero head
    x[1, 1, 5] = float("nan")
    y = api.norm_rope(r, x, None, w, pos=pos)[0]
    assert torch.isnan(y[1, 1]).all() and (y[0] == 0).all() and (y[1, 0] == 0).all() and (y[2] == 0).all()
    y = api.norm_rope(r, x, pos=pos)[0]  # without the norm a value touches its pair alone
    assert int(torch.isnan(y).sum()) == 2
    assert lib.get_device_error() == 0
    # contradictory lens and starts, and an axis that is none: flagged, inside the buffers
    for lens, starts in (([3], [0, 9]), ([-4], [0, 3]), ([3], [-7, 3]), ([3], [5, 1])):
        api.norm_rope(r, x, lens=torch.tensor(lens, dtype=torch.int32).cuda(), starts=torch.tensor(starts, dtype=torch.int32).cuda())
        assert lib.get_device_error() == api.DEVERR_BATCH
    bad = api.rope(64, freqs(64).cuda(), axis=torch.full((32,), 3, dtype=torch.uint8).cuda(), n_axes=2)
    x = torch.randn(3, 2, 64, device="cuda")
    two = torch.stack([pos[:, 0], pos[:, 0] + 9], 1).contiguous()
    assert torch.equal(api.norm_rope(bad, x, pos=two)[0], api.norm_rope(r, x, pos=pos)[0])
    assert lib.get_device_error() == api.DEVERR_BATCH


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,R", [(128, 64), (128, 90), (128, 92), (72, 40), (256, 254), (192, 2)])
def test_what_does_not_turn_is_left_as_it_is(lib, D, R, inter, dtype):
    x = torch.randn(3, 8, D, device="cuda").to(dtype)
    x[:, :, R] = float("inf")
    x[:, :, R + 1::3] = -0.0
    x[1, 1:, D - 1] = -float("inf")
    pos = torch.tensor([[0], [5], [70000]], dtype=torch.int32).cuda()
    y = api.norm_rope(api.rope(D, freqs(R).cuda(), interleaved=inter), x, pos=pos)[0]
    bits = torch.int32 if dtype is torch.float32 else torch.int16
    assert torch.equal(y[:, :, R:].view(bits), x[:, :, R:].view(bits))
    assert torch.isfinite(y[:, :, :R]).all()


def test_many_tokens_and_far_strides(lib):
    n = 65535
    x = torch.randn(n, 1, 8, device="cuda", dtype=torch.bfloat16)
    r = api.rope(8, freqs(8).cuda())
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    y = api.norm_rope(r, x, pos=pos[:, None].contiguous())[0]
    angle = pos.double()[:, None] * freqs(8).double().cuda()
    a, b = x[:, 0, :4].double(), x[:, 0, 4:].double()
    want = torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], 1)
    mag = (a.abs() + b.abs()).repeat(1, 2)
    close(y[:, 0], want.cpu().numpy(), mag.cpu().numpy(), torch.bfloat16)
    # tokens 2^21 elements apart: their offsets pass 2^31
    wide = torch.empty(1100 << 21, dtype=torch.bfloat16, device="cuda")
    far = wide.as_strided((1100, 1, 8), (1 << 21, 8, 1))
    far.copy_(x[:1100])
    z = api.norm_rope(r, far, pos=pos[:1100, None].contiguous(), q_out=far)[0]
    assert torch.equal(z, y[:1100])
