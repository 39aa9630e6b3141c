"""Memory bounds, streams and graphs of the rotation, adapter, expert selection
and log probability kernels: guard bands around every result and workspace, the
range-checked build (the same bits, no failed check, checks that are live), dirty
workspaces, other streams, and captured calls replayed on changed inputs."""
import pytest
import torch

from moe_matvec_gb300 import api
from tests.test_canary_gpu import Guarded
from tests.test_debug_gpu import both, same_bits

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def dbg(lib):
    return api.load_debug()


def rnd(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def rope_case(D, R, H, Hk, n, dtype, inter=False):
    freq = torch.exp(-0.2 * torch.arange(R // 2)).cuda()
    r = api.rope(D, freq, interleaved=inter)
    q, k = rnd(D + n, n, H, D, dtype=dtype), rnd(R + n, n, Hk, D, dtype=dtype)
    w = rnd(1, D)
    lens = torch.arange(1, n + 1, dtype=torch.int32).cuda()
    return lambda **o: api.norm_rope(r, q, k, w, w, lens=lens, **o), (q, k)


def lora_case(n, K, M, r, dtype, pool=5):
    A, B = rnd(K, pool, r, K, dtype=dtype), rnd(M, pool, M, r, dtype=dtype)
    d = api.lora(A, B, rnd(3, pool), ints(*[max(0, r - i) for i in range(pool)]))
    ids = ints(*[(i * 7) % (pool + 1) - 1 for i in range(n)])
    x, res = rnd(n, n, K), rnd(n + 1, n, M)
    return lambda **o: api.lora_run(d, ids, x, res, **o), d, (A, B, x, res)


ROPES = [(128, 128, 8, 2, 1), (128, 64, 3, 1, 37), (72, 40, 2, 2, 5), (128, 90, 5, 1, 3), (256, 256, 9, 4, 70), (8, 2, 1, 1, 2),
         (192, 96, 2, 1, 4)]
LORAS = [(1, 8, 1, 4), (3, 264, 130, 8), (8, 4096, 333, 16), (9, 520, 1025, 128), (64, 2048, 77, 12), (33, 1000, 4099, 64)]
ROUTES = [(1, 1, 1, 1, 1, 1), (3, 8, 8, 1, 1, 1), (7, 256, 8, 8, 4, 2), (66, 100, 5, 5, 2, 2), (5, 510, 8, 17, 3, 1), (4000, 64, 6, 1, 1, 1)]
LOGPS = [(1, 1, 1, 1), (2, 37, 3, 5), (3, 5001, 2, 20), (1, 151936, 1, 32), (20, 40000, 1, 8), (200, 3001, 4, 0), (160, 9000, 0, 3)]


# ------------------------------------------------------------ guard bands
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,R,H,Hk,n", ROPES)
def test_norm_rope_stays_in_its_buffers(lib, dtype, D, R, H, Hk, n):
    if D * 2 % 16 and dtype is not torch.float32:
        pytest.skip("heads of whole 16 bytes")
    for inter in (False, True):
        call, given = rope_case(D, R, H, Hk, n, dtype, inter)
        keep = [t.clone() for t in given]
        want = call()
        q, k = Guarded((n, H, D), dtype, 1), Guarded((n, Hk, D), dtype, 2)
        call(q_out=q.t, k_out=k.t)
        q.check_guards("q")
        k.check_guards("k")
        assert same_bits(q.t, want[0]) and same_bits(k.t, want[1])
        assert all(same_bits(a, b) for a, b in zip(keep, given))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,K,M,r", LORAS)
def test_lora_stays_in_its_buffers(lib, dtype, n, K, M, r):
    call, d, given = lora_case(n, K, M, r, dtype)
    keep = [t.clone() for t in given]
    want = call()
    y = Guarded((n, M), torch.float32, 1)
    ws = Guarded((api.lora_workspace_bytes(d, n),), torch.uint8, 2)
    ws.t.fill_(0xFF)  # (NaN where it is not written)
    call(out=y.t, ws=ws.t)
    y.check_guards("y")
    ws.check_guards("ws")
    assert same_bits(y.t, want) and all(same_bits(a, b) for a, b in zip(keep, given))
    assert lib.get_device_error() == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,E,k,G,keep,top", ROUTES)
def test_route_select_stays_in_its_buffers(lib, dtype, n, E, k, G, keep, top):
    logits, bias = rnd(E + n, n, E, dtype=dtype), 0.2 * rnd(E, E)
    before = logits.clone(), bias.clone()
    for gating in (0, 1):
        args = dict(bias=bias, groups=G, keep=keep, group_top=top)
        want = api.route_select(logits, k, gating, **args)
        ids, gates = Guarded((n, k), torch.int32, 1), Guarded((n, k), torch.float32, 2)
        api.route_select(logits, k, gating, ids=ids.t, gates=gates.t, **args)
        ids.check_guards("ids")
        gates.check_guards("gates")
        assert same_bits(ids.t, want[0]) and same_bits(gates.t, want[1])
    assert same_bits(logits, before[0]) and same_bits(bias, before[1])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,V,given,top", LOGPS)
def test_logprobs_stays_in_its_buffers(lib, dtype, n, V, given, top):
    logits = 3 * rnd(V, n, V)
    logits = logits.to(dtype)
    before = logits.clone()
    tokens = torch.randint(0, V, (n, given), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda() if given else None
    want = api.logprobs(logits, tokens, top)
    shapes = {"logp": ((n, given), torch.float32), "lse": ((n,), torch.float32), "entropy": ((n,), torch.float32),
              "ids": ((n, top), torch.int32), "top": ((n, top), torch.float32)}
    names = [m for m in shapes if (given or m != "logp") and (top or m not in ("ids", "top"))]
    outs = {m: Guarded(*shapes[m], 3 + i) for i, m in enumerate(names)}
    api.logprobs(logits, tokens, top, **{m: g.t for m, g in outs.items()})
    for m, g in outs.items():
        g.check_guards(m)
        assert same_bits(g.t, want[list(shapes).index(m)]), m
    assert same_bits(logits, before)


# ------------------------------------------------------ range-checked build
@pytest.mark.parametrize("dtype", DT)
def test_range_checked_build_gives_the_same_bits(dbg, dtype):
    def run():
        out = []
        for c in ROPES:
            if c[0] * 2 % 16 == 0 or dtype is torch.float32:
                for inter in (False, True):
                    out += rope_case(*c, dtype, inter)[0]()
        for c in LORAS:
            out.append(lora_case(*c, dtype)[0]())
        for n, E, k, G, keep, top in ROUTES:
            logits, bias = rnd(E + n, n, E, dtype=dtype), 0.2 * rnd(E, E)
            for gating in (0, 1):
                out += api.route_select(logits, k, gating, bias=bias, groups=G, keep=keep, group_top=top)
                out += api.route_select(logits, k, gating, groups=G, keep=keep, group_top=top, renorm=False)
        for n, V, given, top in LOGPS:
            logits = (3 * rnd(V, n, V)).to(dtype)
            tokens = torch.zeros(n, given, dtype=torch.int32, device="cuda") if given else None
            out += [t for t in api.logprobs(logits, tokens, top) if t is not None]
        return out

    rel, d, err = both(dbg, run)
    assert err == 0
    assert len(rel) == len(d) and all(same_bits(a, b) for a, b in zip(rel, d))


def test_the_checks_are_live(dbg):
    rope, _ = rope_case(128, 128, 4, 2, 3, torch.float32)
    lora, _, _ = lora_case(3, 264, 130, 8, torch.float16)
    many, _, _ = lora_case(20, 264, 130, 8, torch.float16)
    logits = rnd(5, 12, 64)
    k2, g2 = torch.empty(3, 2, 128, device="cuda"), torch.empty(12, 4, device="cuda")
    lse = torch.empty(12, device="cuda")
    calls = {
        "rope": ((3, 4, 128), torch.float32, lambda o: rope(q_out=o, k_out=k2)),
        "lora": ((3, 130), torch.float32, lambda o: lora(out=o)),
        "lora of many": ((20, 130), torch.float32, lambda o: many(out=o)),
        "route": ((12, 4), torch.int32, lambda o: api.route_select(logits, 4, ids=o, gates=g2)),
        "logprobs": ((12, 4), torch.int32, lambda o: api.logprobs(logits, n_top=4, lse=lse, ids=o)),
    }
    for name, (shape, dt, call) in calls.items():
        want = torch.full(shape, 7, dtype=dt, device="cuda")
        call(want)
        got = torch.full(shape, 7, dtype=dt, device="cuda")
        with api.using(dbg):
            api.get_device_error()
            api.debug_shrink_outputs(8)
            try:
                call(got)
            finally:
                err = api.get_device_error()
                api.debug_shrink_outputs(0)
            assert err == api.DEVERR_RANGE, name
            flat, ref = got.flatten(), want.flatten()
            assert torch.equal(flat[:-16], ref[:-16]) and (flat[-8:] == 7).all(), name
            call(got)
            assert api.get_device_error() == 0 and torch.equal(got, want), name


# ------------------------------------------------------------ streams and graphs
def calls(n=6):
    """One of each as closures over buffers that can change: (inputs, call)."""
    r = api.rope(128, torch.exp(-0.2 * torch.arange(64)).cuda())
    q, lens, w = rnd(1, n, 4, 128), torch.arange(5, 5 + n, dtype=torch.int32).cuda(), rnd(2, 128)
    A, B = rnd(3, 4, 16, 512, dtype=torch.bfloat16), rnd(4, 4, 777, 16, dtype=torch.bfloat16)
    d, ids, x, res = api.lora(A, B), ints(*[i % 4 for i in range(n)]), rnd(5, n, 512), rnd(6, n, 777)
    wide = ints(*[i % 4 for i in range(40)]), rnd(7, 40, 512), rnd(8, 40, 777)
    logits, bias = rnd(9, n, 64), 0.1 * rnd(10, 64)
    head, tokens = 3 * rnd(11, n, 30000), torch.zeros(n, 1, dtype=torch.int32).cuda()
    return [((q, lens), lambda **s: api.norm_rope(r, q, None, w, lens=lens, **s)[:1]),
            ((ids, x, res), lambda **s: (api.lora_run(d, ids, x, res, **s),)),
            (wide, lambda **s: (api.lora_run(d, *wide, **s),)),
            ((logits,), lambda **s: api.route_select(logits, 4, 1, bias=bias, groups=4, keep=2, **s)),
            ((head, tokens), lambda **s: api.logprobs(head, tokens, 5, **s))]


def change(t, step):
    if t.dtype is torch.int32:
        t.copy_((t + step) % 4 if t.max() < 4 and t.dim() == 1 else t + step)
    else:
        t.mul_(-0.75).add_(0.25 * step)


def test_a_given_stream_and_memory_dropped_early(lib):
    side = torch.cuda.Stream()
    for inputs, call in calls():
        want = call()
        torch.cuda.synchronize()
        for _ in range(20):  # results and workspaces of this stream's calls are not handed to the current one's
            got = call(stream=side)
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 16, 1 << 20)]
            side.synchronize()
            assert all(same_bits(a, b) for a, b in zip(got, want))
            del junk, got


def test_captured_calls_follow_their_inputs(lib):
    for i in range(len(calls())):
        inputs, call = calls()[i]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                got = call()
            for step in range(4):
                for t in inputs:
                    change(t, step)
                graph.replay()
                want = call()
                side.synchronize()
                assert all(same_bits(a, b) for a, b in zip(got, want)), (i, step)
    assert lib.get_device_error() == 0


def test_two_graphs_share_a_workspace(lib):
    A, B = rnd(3, 9, 64, 2048, dtype=torch.bfloat16), rnd(4, 9, 4000, 64, dtype=torch.bfloat16)
    d = api.lora(A, B)
    ids = ints(*[i % 9 for i in range(30)])
    xs, rs = [rnd(i, 30, 2048) for i in (5, 6)], [rnd(i, 30, 4000) for i in (7, 8)]
    want = [api.lora_run(d, ids, x, r) for x, r in zip(xs, rs)]
    ws = torch.empty(api.lora_workspace_bytes(d, 30), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, got = [], []
    with torch.cuda.stream(side):
        for x, r in zip(xs, rs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                got.append(api.lora_run(d, ids, x, r, ws=ws))
            graphs.append(g)
        for _ in range(10):
            for g in graphs:
                g.replay()
        side.synchronize()
    assert all(same_bits(a, b) for a, b in zip(got, want))


def test_results_do_not_change_from_call_to_call(lib):
    for _, call in calls(40):
        want = call()
        for _ in range(5):
            assert all(same_bits(a, b) for a, b in zip(call(), want))


def test_descriptors_of_another_device_are_refused(lib):
    r = api.rope(64, torch.ones(32).cuda())
    d = api.lora(rnd(1, 2, 4, 64), rnd(2, 2, 10, 4))
    assert r.reserved == d.reserved == torch.cuda.current_device() + 1
    r.reserved = d.reserved = 2 + torch.cuda.current_device()  # as if they had been made there
    with pytest.raises(ValueError, match="current device"):
        api.norm_rope(r, rnd(3, 2, 1, 64), pos=ints(1, 2)[:, None].contiguous())
    with pytest.raises(ValueError, match="current device"):
        api.lora_run(d, ints(0, 1), rnd(4, 2, 64), rnd(5, 2, 10))
