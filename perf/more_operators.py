"""What a decode step needs between and after the library's matvecs, cache and
experts, case by case: what is run, in plain torch operations and through the
library's entry points.

Four operators.  `rope`: norm of each query and key head and the position
rotation, by one position a token or several (time, height, width).  `lora`:
low-rank adapters of many requests beside a shared projection,
y = r + scale_a B_a (A_a x) with each token's own adapter a.  `route`: experts
from router logits, with softmax or sigmoid scores, a bias for balance, groups,
top-k and renormalised weights.  `logp`: log probabilities of given tokens, with
log-sum-exp, entropy and the top alternatives.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _rope(name, tokens, heads, kv_heads, dim, rotary, interleaved, axes, norm, dtype, far, spread):
    """far: the largest position; spread: 0: one token a sequence, else ragged runs of tokens (both by the sequences'
    lengths), or with axes > 1 explicit positions."""
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "interleaved": interleaved, "axes": axes, "norm": norm, "dtype": dtype, "far": far,
            "spread": spread}


def _lora(name, tokens, cols, rows, adapters, rank, dtype, spread):
    """spread 0: token t has adapter t % adapters, all of full rank; else adapters at random, some tokens without one,
    and ranks from a quarter of the pool's on."""
    return {"name": name, "op": "lora", "tokens": tokens, "cols": cols, "rows": rows, "adapters": adapters,
            "rank": rank, "dtype": dtype, "spread": spread}


def _route(name, tokens, experts, top_k, gating, bias, groups, keep, group_top, renorm, scale, dtype):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "gating": gating,
            "bias": bias, "groups": groups, "keep": keep, "group_top": group_top, "renorm": renorm, "scale": scale,
            "dtype": dtype}


def _logp(name, rows, vocab, given, top, scale, dtype, sharp):
    """sharp: the logits' standard deviation."""
    return {"name": name, "op": "logp", "rows": rows, "vocab": vocab, "given": given, "top": top, "scale": scale,
            "dtype": dtype, "sharp": sharp}


def listed():
    return [
        # one user's next token: nothing but latency
        _rope("rope_1", 1, 32, 8, 128, 128, False, 1, True, "f32", 4000, 0),
        # a full decode batch on long contexts, half of each head turned
        _rope("rope_64", 64, 40, 8, 128, 64, False, 1, True, "f32", 200000, 0),
        # a prompt of text and images: three position axes
        _rope("rope_4096_axes3_bf16", 4096, 32, 8, 128, 128, False, 3, True, "bf16", 30000, 1),
        # one request with an adapter on a square projection
        _lora("lora_1", 1, 4096, 4096, 8, 16, "bf16", 0),
        # a decode batch of requests with adapters of different ranks, or none, on the widest projection
        _lora("lora_24_ragged", 24, 5120, 17408, 10, 64, "bf16", 3),
        # every request of a full batch has its own adapter
        _lora("lora_64_own", 64, 5120, 17408, 64, 64, "bf16", 0),
        # one token, grouped sigmoid routing with a balance bias
        _route("route_1", 1, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "f32"),
        # a decode batch, softmax over all experts
        _route("route_64", 64, 128, 8, "softmax", False, 1, 1, 1, True, 1.0, "f32"),
        # a prompt's tokens, grouped
        _route("route_16384", 16384, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "f32"),
        # one token with its 20 best alternatives
        _logp("logp_1", 1, 151936, 1, 20, 1.0, "f32", 3.0),
        # a batch of draft tokens to verify, at a sampling temperature
        _logp("logp_16", 16, 151936, 2, 8, 1.25, "f32", 4.0),
        # scoring prompts
        _logp("logp_2048_bf16", 2048, 151936, 1, 5, 1.0, "bf16", 3.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "lora", "route", "logp"])
    if op == "rope":
        dtype = rng.choice(["f32", "f16", "bf16"])
        dim = rng.choice([64, 128, 128, 192, 256, 80, 72])
        rotary = rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        kv_heads = rng.choice([1, 2, 4, 5, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
        tokens = min(_log(rng, 1, 4096), 4096 * 40 * 128 * 2 // ((heads + kv_heads) * dim * SIZES[dtype]))
        c = _rope("", tokens, heads, kv_heads, dim, rotary, rng.random() < 0.3, rng.choice([1, 1, 1, 2, 3]),
                  rng.random() < 0.7, dtype, _log(rng, 100, 1000000), rng.choice([0, rng.randrange(1, 1000)]))
    elif op == "lora":
        tokens, rank = _log(rng, 1, 64), rng.choice([4, 8, 16, 24, 32, 64])
        cols, rows = 8 * _log(rng, 64, 2176), _log(rng, 200, 17408)
        cols, rows = min(cols, 17408), min(rows, 22528 - min(cols, 5120))
        adapters = _log(rng, 1, 64)
        if rank * (cols + rows) * adapters > 64 * 22528 * 64:
            adapters = max(1, 64 * 22528 * 64 // (rank * (cols + rows)))
        c = _lora("", tokens, cols, rows, adapters, rank, rng.choice(["bf16", "bf16", "f16", "f32"]) if adapters <= 32
                  else "bf16", rng.choice([0, rng.randrange(1, 1000), rng.randrange(1, 1000)]))
    elif op == "route":
        groups = rng.choice([1, 1, 2, 4, 5, 8, 16])
        experts = groups * rng.randint(max(2, 16 // groups), 512 // groups)
        keep = rng.randint(1, groups)
        top_k = rng.randint(1, min(8, keep * (experts // groups)))
        tokens = min(_log(rng, 1, 16384), 16384 * 256 // experts)
        c = _route("", tokens, experts, top_k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, groups, keep,
                   rng.choice([1, 2]), rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.choice(["f32", "f32", "bf16", "f16"]))
    else:
        dtype = rng.choice(["f32", "f16", "bf16"])
        vocab = rng.choice([_log(rng, 1000, 262144), 151936, 32000, 128256])
        rows = min(_log(rng, 1, 2048), 2048 * 151936 * 2 // (vocab * SIZES[dtype]))
        c = _logp("", rows, vocab, rng.randint(0, 4), rng.choice([0, 1, 5, 20, 32, rng.randint(2, 31)]),
                  rng.choice([1.0, 1.0, 0.7, 1.25]), dtype, round(rng.uniform(0.5, 8.0), 2))
    return {k: v for k, v in c.items() if k != "name"}


def _runs(case):
    """Lengths of the sequences (the call's tokens among them) and how many tokens of each the call has."""
    n, far, r = case["tokens"], case["far"], random.Random(case["spread"])
    if not case["spread"]:  # one token a sequence
        news = [1] * n
    else:
        news = []
        while sum(news) < n:
            news.append(min(n - sum(news), r.randint(1, max(1, n // 3))))
    return [max(c, r.randint(max(1, far // 2), far)) for c in news], news


def _adapters(case):
    """Each token's adapter (-1: none) and each adapter's rank."""
    n, a, rank = case["tokens"], case["adapters"], case["rank"]
    if not case["spread"]:
        return [t % a for t in range(n)], [rank] * a
    r = random.Random(case["spread"])
    return [r.randrange(-1, a) for _ in range(n)], [r.randint(max(1, rank // 4), rank) for _ in range(a)]


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    st = {"case": case}
    if case["op"] == "rope":
        n, H, Hk, D, R, dt = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "rotary", "dtype"))
        qkv = (2 * randn(n, H + 2 * Hk, D)).to(DTYPES[dt])  # the fused projection's result
        st["q"], st["k"] = qkv[:, :H], qkv[:, H:H + Hk]
        st["freq"] = torch.exp(torch.arange(R // 2, device=dev) * (-2 * math.log(1000000.0) / R))
        st["q_w"] = 1 + 0.1 * randn(D) if case["norm"] else None
        st["k_w"] = 1 + 0.1 * randn(D) if case["norm"] else None
        lens, news = _runs(case)
        st["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
        st["starts"] = torch.tensor(np.concatenate([[0], np.cumsum(news)]), device=dev, dtype=torch.int32)
        st["axis"] = st["pos"] = None
        if case["axes"] > 1:  # pairs take the axes in turn, and a token's positions differ
            st["axis"] = (torch.arange(R // 2, device=dev) % case["axes"]).to(torch.uint8)
            first = torch.randint(0, case["far"] - 99, (n, 1), generator=g, device=dev)
            step = torch.randint(0, 100, (n, case["axes"]), generator=g, device=dev)
            st["pos"] = (first + step).to(torch.int32)
        return st
    if case["op"] == "lora":
        n, K, M, a, r, dt = (case[k] for k in ("tokens", "cols", "rows", "adapters", "rank", "dtype"))
        ids, ranks = _adapters(case)
        st["A"] = (randn(a, r, K) / math.sqrt(K)).to(DTYPES[dt])
        st["B"] = (randn(a, M, r) / math.sqrt(r)).to(DTYPES[dt])
        st["scales"] = 0.5 + torch.rand(a, generator=g, device=dev)
        st["ids"] = torch.tensor(ids, device=dev, dtype=torch.int32)
        st["ranks"] = torch.tensor(ranks, device=dev, dtype=torch.int32)
        st["x"], st["r"] = randn(n, K), randn(n, M)
        return st
    if case["op"] == "route":
        n, E = case["tokens"], case["experts"]
        st["logits"] = (1.5 * randn(n, E) + 0.5 * randn(E)).to(DTYPES[case["dtype"]])
        st["bias"] = 0.2 * randn(E) if case["bias"] else None
        return st
    n, V = case["rows"], case["vocab"]
    st["logits"] = torch.empty(n, V, device=dev, dtype=DTYPES[case["dtype"]])
    step = max(1, (1 << 26) // V)
    for a in range(0, n, step):
        st["logits"][a:a + step] = case["sharp"] * randn(min(step, n - a), V)
    st["tokens"] = None
    if case["given"]:
        st["tokens"] = torch.randint(0, V, (n, case["given"]), generator=g, device=dev).to(torch.int32)
        likely = st["logits"].argmax(-1).to(torch.int32)  # most tokens of a text are likely ones
        st["tokens"][::2, 0] = likely[::2]
    return st


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"rope": _plain_rope, "lora": _plain_lora, "route": _plain_route, "logp": _plain_logp}[case["op"]](case, state)


def _run_own(case, st):
    from moe_matvec_gb300 import api
    if case["op"] == "rope":
        rope = st.get("rope")
        if rope is None:  # the descriptor that a program makes once for a model
            rope = st["rope"] = api.rope(case["dim"], st["freq"], axis=st["axis"], n_axes=case["axes"],
                                         interleaved=case["interleaved"])
        if st["pos"] is not None:
            q, k = api.norm_rope(rope, st["q"], st["k"], st["q_w"], st["k_w"], EPS, pos=st["pos"])
        else:
            starts = st["starts"] if case["spread"] else None
            q, k = api.norm_rope(rope, st["q"], st["k"], st["q_w"], st["k_w"], EPS, lens=st["lens"], starts=starts)
        return {"q": q, "k": k}
    if case["op"] == "lora":
        lora = st.get("lora")
        if lora is None:  # the pool's descriptor
            lora = st["lora"] = api.lora(st["A"], st["B"], scales=st["scales"], ranks=st["ranks"])
        return {"y": api.lora_run(lora, st["ids"], st["x"], st["r"])}
    if case["op"] == "route":
        gating = api.GATING_SIGMOID if case["gating"] == "sigmoid" else api.GATING_SOFTMAX
        ids, gates = api.route_select(st["logits"], case["top_k"], gating, bias=st["bias"], groups=case["groups"],
                                      keep=case["keep"], group_top=case["group_top"], renorm=case["renorm"],
                                      scale=case["scale"])
        return {"ids": ids, "gates": gates}
    logp, lse, entropy, ids, top = api.logprobs(st["logits"], st["tokens"], n_top=case["top"], scale=case["scale"])
    return {"logp": logp, "lse": lse, "entropy": entropy, "ids": ids, "top": top}


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _plain_rope(case, st):
    R, dt, n = case["rotary"], st["q"].dtype, case["tokens"]
    if st["pos"] is not None:
        pos = st["pos"].long()[:, st["axis"].long()]
    else:  # the last tokens of their sequences
        t = torch.arange(n, device=st["lens"].device)
        starts = st["starts"].long()
        seq = torch.searchsorted(starts, t, right=True) - 1
        pos = (st["lens"].long()[seq] - starts[seq + 1] + t)[:, None]
    angle = pos.double() * st["freq"].double()  # 32 bits lose the turn of far positions
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * (1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * w
        y = x.clone()
        if case["interleaved"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :R // 2], x[..., R // 2:R]
            y[..., :R // 2], y[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
        return y.to(dt)

    return {"q": turned(st["q"], st["q_w"]), "k": turned(st["k"], st["k_w"])}


def _plain_lora(case, st):
    ids = st["ids"].long()
    a = ids.clamp(min=0)
    v = (st["A"][a].float() @ st["x"][..., None])[..., 0]
    live = torch.arange(case["rank"], device=v.device) < st["ranks"][a][:, None]
    v = torch.where(live & (ids >= 0)[:, None], v, 0.0)
    return {"y": st["r"] + st["scales"][a][:, None] * (st["B"][a].float() @ v[..., None])[..., 0]}


def _plain_route(case, st):
    # 64 bits: what is picked is decided by differences of nearly equal scores
    l = st["logits"].double()
    if case["gating"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
    c = s if st["bias"] is None else s + st["bias"].double()
    by_group = c.unflatten(-1, (case["groups"], -1)).sort(dim=-1, descending=True).values
    score = by_group[..., :case["group_top"]].sum(-1)
    kept = score.sort(dim=-1, descending=True, stable=True).indices[:, :case["keep"]]
    mask = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
    mask = mask.repeat_interleave(case["experts"] // case["groups"], 1)
    ids = torch.where(mask, c, -torch.inf).sort(dim=-1, descending=True, stable=True).indices[:, :case["top_k"]]
    gates = s.gather(1, ids)
    if case["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "gates": (gates * case["scale"]).float()}


def _plain_logp(case, st):
    l = st["logits"].float()
    top = l.amax(-1, keepdim=True)
    d = (l - top) * case["scale"]
    e = torch.exp(d)
    total = e.sum(-1, dtype=torch.float64)  # long sums in 64 bits
    log_total = total.log()
    entropy = log_total - (e * d).sum(-1, dtype=torch.float64) / total
    out = {"lse": (top[:, 0].double() * case["scale"] + log_total).float(), "entropy": entropy.float(),
           "logp": None, "ids": None, "top": None}
    if st["tokens"] is not None:
        out["logp"] = (d.gather(1, st["tokens"].long()).double() - log_total[:, None]).float()
    if case["top"]:  # the largest values; of equal ones the lowest index first
        bits = (l + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() * (1 << 32) - torch.arange(case["vocab"], device=l.device)
        ids = key.topk(case["top"], dim=-1, sorted=True).indices
        out["ids"] = ids.to(torch.int32)
        out["top"] = (d.gather(1, ids).double() - log_total[:, None]).float()
    return out


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * SIZES[case["dtype"]] * n + 4 * case["tokens"] * case["axes"], "flops": 8 * n}
    if case["op"] == "lora":
        ids, ranks = _adapters(case)
        wide = case["cols"] + case["rows"]
        read = sum(ranks[a] for a in set(ids) if a >= 0) * wide * SIZES[case["dtype"]]
        return {"bytes": read + 4 * case["tokens"] * (case["cols"] + 2 * case["rows"]),
                "flops": 2 * sum(ranks[a] for a in ids if a >= 0) * wide}
    if case["op"] == "route":
        n = case["tokens"] * case["experts"]
        return {"bytes": n * SIZES[case["dtype"]] + 8 * case["tokens"] * case["top_k"], "flops": 6 * n}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * SIZES[case["dtype"]] + 8 * case["rows"] * (1 + case["given"] + case["top"]), "flops": 6 * n}


# --------------------------------------------------------------------------
# The operators' definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, st)
    if case["op"] == "lora":
        x, y = st["x"].cpu().double().numpy(), st["r"].cpu().double().numpy()
        ids, ranks = _adapters(case)
        for t, a in enumerate(ids):
            if a >= 0:
                A, B = st["A"][a, :ranks[a]].cpu().double().numpy(), st["B"][a, :, :ranks[a]].cpu().double().numpy()
                y[t] += float(st["scales"][a]) * (B @ (A @ x[t]))
        return {"y": torch.from_numpy(y)}
    if case["op"] == "route":
        return _exact_route(case, st)
    return _exact_logp(case, st)


def _exact_rope(case, st):
    n, R, D, out = case["tokens"], case["rotary"], case["dim"], {}
    if st["pos"] is not None:
        pos = st["pos"].cpu().numpy().astype(np.float64)[:, st["axis"].cpu().numpy().astype(np.int64)]
    else:
        lens, news = _runs(case)
        pos = np.concatenate([np.arange(t - c, t) for t, c in zip(lens, news)]).astype(np.float64)[:, None]
    turn = np.exp(1j * pos * st["freq"].cpu().numpy().astype(np.float64))[:, None]
    for name in ("q", "k"):
        x = st[name].cpu().double().numpy()
        if case["norm"]:
            x = x / np.sqrt(np.mean(np.square(x), -1, keepdims=True) + EPS) * st[name + "_w"].cpu().double().numpy()
        i = np.arange(R // 2)
        one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
        z = (x[..., one] + 1j * x[..., two]) * turn
        y = np.array(x)
        y[..., one], y[..., two] = z.real, z.imag
        out[name] = torch.from_numpy(y.reshape(n, -1, D))
    return out


def _exact_route(case, st):
    l = st["logits"].cpu().double().numpy()
    n, E, G = l.shape[0], case["experts"], case["groups"]
    with np.errstate(over="ignore"):
        if case["gating"] == "sigmoid":
            s = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
        else:
            s = np.exp(l - l.max(1, keepdims=True))
            s /= s.sum(1, keepdims=True)
    b = st["bias"].cpu().double().numpy() if st["bias"] is not None else np.zeros(E)
    ids, gates = np.empty((n, case["top_k"]), np.int32), np.empty((n, case["top_k"]))
    for t in range(n):
        c = s[t] + b
        score = np.sort(c.reshape(G, -1), -1)[:, ::-1][:, :case["group_top"]].sum(-1)
        kept = set(np.argsort(-score, kind="stable")[:case["keep"]].tolist())
        c = np.where([g in kept for g in range(G)], c.reshape(G, -1).T, -np.inf).T.reshape(-1)
        ids[t] = np.argsort(-c, kind="stable")[:case["top_k"]]
        w = s[t, ids[t]]
        gates[t] = w / (w.sum() if case["renorm"] else 1) * case["scale"]
    return {"ids": torch.from_numpy(ids), "gates": torch.from_numpy(gates)}


def _exact_logp(case, st):
    n, V = case["rows"], case["vocab"]
    out = {"logp": None, "lse": np.empty(n), "entropy": np.empty(n), "ids": None, "top": None}
    if case["given"]:
        out["logp"], tokens = np.empty((n, case["given"])), st["tokens"].cpu().numpy()
    if case["top"]:
        out["ids"], out["top"] = np.empty((n, case["top"]), np.int32), np.empty((n, case["top"]))
    for t in range(n):
        row = st["logits"][t].double()
        z = row * case["scale"]
        p = torch.softmax(z, -1)
        lse = torch.logsumexp(z, -1)
        logs = z - lse
        out["lse"][t], out["entropy"][t] = float(lse), float(-(p * logs).sum())
        if case["given"]:
            out["logp"][t] = logs[torch.from_numpy(tokens[t]).long().cuda()].cpu().numpy()
        if case["top"]:
            least = row.topk(case["top"]).values[-1]
            at = torch.nonzero(row >= least)[:, 0].cpu().numpy()
            at = at[np.argsort(-row[torch.from_numpy(at).cuda()].cpu().numpy(), kind="stable")][:case["top"]]
            out["ids"][t], out["top"][t] = at, logs[torch.from_numpy(at).cuda()].cpu().numpy()
    return {k: None if v is None else torch.from_numpy(v) for k, v in out.items()}
