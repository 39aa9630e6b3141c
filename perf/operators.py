"""The attention half of a decode layer, case by case: what is run, in plain
torch operations and through the library's entry points.

Four operators.  `norm`: root-mean-square norm with the residual's addition,
its output as floats and / or in the library's 8-bit activation layout.
`append`: new keys and values into the paged 8-bit cache (one scale per page
and head), and the touched pages read back.  `attend`: attention of the last
tokens of each sequence over that cache.  `sparse`: one decode step with page
selection (append, score and select pages, attend over the selected ones).

A cache page of one head is a record of 16 + 2 P D bytes: two fp32 scales
(keys, values) and 8 spare bytes, then the key codes [D / 64][P][64], then the
value codes [D][P]; a byte b stands for scale * (b - 128).  The bounds of a
page are 16 + 2 D bytes: the fp32 key scale and 12 spare bytes, then the
smallest and the largest key code of each dimension (int8).  Page 0 of every
pool here is a spare that no sequence owns.
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
def _norm(name, rows, dim, dtype, residual, out):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "dtype": dtype, "residual": residual, "out": out}


def _cache(name, op, seqs, ctx, new, heads, kv_heads, dim, page, dtype, spread, window=0, select=0):
    return {"name": name, "op": op, "seqs": seqs, "ctx": ctx, "new": new, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "dtype": dtype, "spread": spread, "window": window, "select": select}


def listed():
    return [
        # the norm in front of a matvec, one user: nothing but latency
        _norm("norm_1x5120", 1, 5120, "f32", True, "q8"),
        # a full decode batch, both outputs (8 bits for the matvecs, floats for the router)
        _norm("norm_64x4096", 64, 4096, "f32", True, "both"),
        # a prompt's tokens in half precision
        _norm("norm_4096x5120_bf16", 4096, 5120, "bf16", True, "both"),
        # one sequence grows by one token
        _cache("append_1", "append", 1, 1000, 1, 32, 8, 128, 64, "f32", 0),
        # a decode batch, every sequence somewhere inside a page
        _cache("append_64", "append", 64, 3000, 1, 32, 8, 128, 32, "f32", 1),
        # ragged prompts written at once
        _cache("append_prompts", "append", 6, 6000, 6000, 32, 8, 128, 64, "bf16", 2),
        # one user, a short conversation: latency
        _cache("attend_1_ctx1000", "attend", 1, 1000, 1, 32, 8, 128, 64, "f32", 0),
        # the serving batch, ragged contexts
        _cache("attend_32_ctx8192", "attend", 32, 8192, 1, 40, 8, 128, 64, "f32", 3),
        # a few draft tokens checked per sequence, small heads, a sliding window, small pages
        _cache("attend_draft_ctx4000", "attend", 12, 4000, 8, 28, 4, 64, 16, "bf16", 4, window=2500),
        # one very long context
        _cache("attend_1_ctx131072", "attend", 1, 131072, 1, 64, 8, 128, 64, "bf16", 0),
        # a long conversation of a few users, an eighth of the pages read
        _cache("sparse_2_ctx16384", "sparse", 2, 16384, 1, 32, 8, 128, 64, "f32", 5, select=32),
        # many long contexts, a sixteenth of the pages read
        _cache("sparse_16_ctx65536", "sparse", 16, 65536, 1, 32, 8, 128, 64, "f32", 6, select=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "attend", "sparse"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "norm":
        out = rng.choice(["q8", "float", "both"])
        rows = _log(rng, 1, 4096)
        if out == "float":
            dim = _log(rng, 64, 8192) | 1  # any length: odd ones
        else:
            dim = 256 * rng.choice([1, 2, 3, 5, 7, 8, 16, 20, 24, 28, 32])
        return {k: v for k, v in _norm("", rows, dim, dtype, rng.random() < 0.7, out).items() if k != "name"}
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    dim = rng.choice([64, 128, 128, 192, 256])
    page = rng.choice([16, 32, 64])
    seqs = _log(rng, 1, 64)
    # tokens held by all sequences of the batch, up to about those of the largest listed cases
    budget = (1 << 18) * 8 * 128 // (kv_heads * dim)
    select = window = 0
    if op == "append":
        new = rng.choice([1, 1, _log(rng, 1, 2000)])
        new = max(1, min(new, 12000 // seqs))
        ctx = max(new, min(_log(rng, 1, 8000), budget // seqs))
    elif op == "attend":
        new = rng.choice([1, 1, 1, _log(rng, 1, 16)])
        ctx = max(new, min(_log(rng, 1, 65536), budget // seqs // (1 + new * heads // kv_heads // 8)))
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    else:
        new = rng.choice([1, 1, 1, 3])
        ctx = max(2 * page, min(_log(rng, 300, 65536), budget // seqs))
        select = max(1, min(128 // new, _log(rng, 2, max(3, ctx // page // 2))))
    c = _cache("", op, seqs, ctx, new, heads, kv_heads, dim, page, dtype, rng.randrange(1, 1000), window, select)
    return {k: v for k, v in c.items() if k != "name"}


def _lengths(case):
    """Tokens in the cache (the new ones among them) and new tokens of each sequence."""
    n, ctx, new, spread = case["seqs"], case["ctx"], case["new"], case["spread"]
    if not spread:
        return [ctx] * n, [new] * n
    r = random.Random(spread)
    news = [new] + [r.randint(max(1, new // 4), new) for _ in range(n - 1)]
    lens = [max(c, r.randint(max(1, ctx // 3), ctx)) for c in news]
    lens[0] = ctx
    if case["op"] == "append":  # a prompt starts its sequence, or goes on in the middle of a page
        lens = [c if new > 64 and i % 2 == 0 else t for i, (t, c) in enumerate(zip(lens, news))]
    return lens, news


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    dt = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        rows, dim = case["rows"], case["dim"]
        st = {"case": case, "x": randn(rows, dim).to(dt), "w": 1 + 0.1 * randn(dim),
              "r": (3 * randn(rows, dim)).to(dt) if case["residual"] else None}
        return st

    H, D, P, n = case["kv_heads"], case["dim"], case["page"], case["seqs"]
    lens, news = _lengths(case)
    pages = [-(-t // P) for t in lens]
    mp = max(pages)
    n_pages = 1 + sum(pages)
    perm = (1 + torch.randperm(n_pages - 1, generator=g, device=dev)).to(torch.int32)
    counts = torch.tensor(pages, device=dev)
    first = torch.cumsum(counts, 0) - counts
    col = torch.arange(mp, device=dev)
    inside = col < counts[:, None]
    table = torch.where(inside, perm[(first[:, None] + col).clamp(max=n_pages - 2)], -1).to(torch.int32).contiguous()
    lens_d = torch.tensor(lens, device=dev, dtype=torch.int32)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(news)]), device=dev, dtype=torch.int32)
    n_tok = sum(news)

    # the cache as earlier steps left it: keys of a page share an offset, as neighbouring tokens do
    pool = torch.empty(n_pages, H, 16 + 2 * P * D, dtype=torch.uint8, device=dev)
    bounds = None
    if case["op"] == "sparse":
        bounds = torch.zeros(n_pages, H, 16 + 2 * D, dtype=torch.uint8, device=dev)
        held = torch.zeros(n_pages, dtype=torch.int64, device=dev)
        before = torch.tensor([t - c for t, c in zip(lens, news)], device=dev)
        inpage = (before[:, None] - col * P).clamp(0, P)
        held[table.clamp(min=0).long().flatten()] = inpage.flatten()
        held[0] = 0
    step = max(1, (1 << 26) // (H * P * D))
    for a in range(0, n_pages, step):
        b = min(n_pages, a + step)
        scales = 0.027 * torch.exp(0.1 * randn(b - a, H, 2))
        pool[a:b, :, :16] = 0
        pool[a:b, :, :8] = scales.view(torch.uint8).reshape(b - a, H, 8)
        k = randn(b - a, H, P, D, dtype=torch.float16).mul_(28).add_(randn(b - a, H, 1, D, dtype=torch.float16), alpha=24)
        k = k.round_().clamp_(-127, 127)
        pool[a:b, :, 16:16 + P * D] = (k + 128).to(torch.uint8).unflatten(-1, (D // 64, 64)).transpose(2, 3).reshape(b - a, H, P * D)
        if bounds is not None:
            used = (torch.arange(P, device=dev) < held[a:b, None])[:, None, :, None]
            bounds[a:b, :, :4] = scales[..., :1].contiguous().view(torch.uint8).reshape(b - a, H, 4)
            bounds[a:b, :, 16:16 + D] = torch.where(used, k, 127).amin(2).to(torch.int8).view(torch.uint8)
            bounds[a:b, :, 16 + D:] = torch.where(used, k, -127).amax(2).to(torch.int8).view(torch.uint8)
        v = randn(b - a, H, D * P, dtype=torch.float16).mul_(36).round_().clamp_(-127, 127)
        pool[a:b, :, 16 + P * D:] = (v + 128).to(torch.uint8)
    st = {"case": case, "pool": pool, "bounds": bounds, "table": table, "lens": lens_d, "starts": starts,
          "n_tok": n_tok, "max_new": max(news), "n_pages": n_pages}
    # the largest number of pages that one sequence's new tokens touch
    st["touched"] = max((t - 1) // P - (t - c) // P + 1 for t, c in zip(lens, news))
    if case["op"] in ("append", "sparse"):
        st["k"] = randn(n_tok, H, D).to(dt)
        st["v"] = randn(n_tok, H, D).to(dt)
    if case["op"] == "append":  # what is read back: every token of the touched pages
        back = [t - (t - c) // P * P for t, c in zip(lens, news)]
        st["back"] = torch.tensor(np.concatenate([[0], np.cumsum(back)]), device=dev, dtype=torch.int32)
        st["n_back"] = sum(back)
    else:
        st["q"] = (2 * randn(n_tok, case["heads"], D)).to(dt)
        st["ws"] = torch.empty(256 << 20, dtype=torch.uint8, device=dev)
    return st


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "norm":
        return _plain_norm(case, state)
    if case["op"] == "append":
        _plain_append(case, state)
        return _plain_read(case, state)
    if case["op"] == "attend":
        return _plain_attend(case, state)
    _plain_append(case, state)
    ids = _plain_select(case, state)
    return {"ids": ids, "out": _plain_attend_pages(case, state, ids)}


def _run_own(case, st):
    from moe_matvec_gb300 import api
    if case["op"] == "norm":
        out = {}
        y, q8, res = api.rms_norm(st["x"], st["w"], EPS, r=st["r"], want=case["out"])
        if st["r"] is not None:
            out["res"] = res
        if y is not None:
            out["y"] = y
        if q8 is not None:
            out["y8"] = api.dequantize_act(q8[0], q8[1], torch.bfloat16)
        return out
    cache = st.get("cache")
    if cache is None:  # the descriptor that a program makes once for its cache
        cache = st["cache"] = api.kv_cache(case["kv_heads"], case["dim"], case["page"], st["n_pages"],
                                           pages=st["pool"], bounds=st["bounds"])
    starts = None if case["new"] == 1 else st["starts"]
    if case["op"] == "append":
        api.kv_append(cache, st["k"], st["v"], st["table"], st["lens"], starts)
        k, v = api.kv_read(cache, st["table"], st["lens"], st["back"], st["n_back"], st["k"].dtype)
        return {"k": k, "v": v}
    if case["op"] == "attend":
        return api.kv_attend(cache, st["q"], st["table"], st["lens"], starts, window=case["window"], ws=st["ws"])
    api.kv_append(cache, st["k"], st["v"], st["table"], st["lens"], starts)
    ids = api.kv_select(cache, st["q"], st["table"], st["lens"], case["select"], starts, ws=st["ws"])
    return {"ids": ids, "out": api.kv_attend(cache, st["q"], st["table"], st["lens"], starts, pages=ids, ws=st["ws"])}


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _scale_of(amax):
    """d = amax / 127 and 1 / d of the activation rule (a tensor divisor: a true division)."""
    d = amax / torch.full_like(amax, 127.0)
    return d, torch.where(d > 0, 1 / d, torch.zeros_like(d))


def _codes(x, inv):
    return torch.nan_to_num(x * inv, nan=0.0).round().clamp(-127, 127)


def _plain_norm(case, st):
    x = st["x"].float()
    out = {}
    if st["r"] is not None:
        x = x + st["r"].float()
        out["res"] = x.to(st["x"].dtype)
    y = x * (1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * st["w"]
    if case["out"] in ("float", "both"):
        out["y"] = y.to(st["x"].dtype)
    if case["out"] in ("q8", "both"):
        b = y.unflatten(-1, (-1, 32))
        d, inv = _scale_of(b.abs().amax(-1, keepdim=True))
        out["y8"] = (_codes(b, inv) * d).flatten(-2).to(torch.bfloat16)
    return out


def _views(case, st):
    """The key codes [pages][H][D / 64][P][64] and value codes [pages][H][D][P] (bytes), as views of the pool."""
    P, D, pool = case["page"], case["dim"], st["pool"]
    return pool[..., 16:16 + P * D].unflatten(-1, (D // 64, P, 64)), pool[..., 16 + P * D:].unflatten(-1, (D, P))


def _scales(rec):
    return rec[..., :8].contiguous().view(torch.float32)


def _token_places(st, starts, n):
    """Sequence and position of each of n tokens, the last ones of their sequences."""
    t = torch.arange(n, device=starts.device)
    seq = torch.searchsorted(starts, t.to(torch.int32), right=True) - 1
    pos = st["lens"].long()[seq] - starts.long()[seq + 1] + t
    return seq, pos


def _plain_append(case, st):
    P, D, H = case["page"], case["dim"], case["kv_heads"]
    pool, bounds, starts = st["pool"], st["bounds"], st["starts"].long()
    lens = st["lens"].long()
    pos0 = lens - (starts[1:] - starts[:-1])
    page = pos0[:, None] // P + torch.arange(st["touched"], device=pool.device)  # [n][M]
    live = page * P < lens[:, None]
    mp = st["table"].shape[1]
    phys = torch.where(live, st["table"].long().gather(1, page.clamp(max=mp - 1)), 0)
    pos = page[..., None] * P + torch.arange(P, device=pool.device)  # [n][M][P]
    fresh = (pos >= pos0[:, None, None]) & (pos < lens[:, None, None]) & live[..., None]
    old = pos < pos0[:, None, None]
    src = torch.where(fresh, starts[:-1, None, None] + pos - pos0[:, None, None], 0)
    rec = pool[phys]  # [n][M][H][..]
    sc = _scales(rec)
    had = old.any(-1)[..., None]
    m = fresh[..., None, None]
    new_sc, body, extremes = [], [], None
    for part in (0, 1):  # keys, values
        x = torch.where(m, (st["k"], st["v"])[part].float()[src], 0.0)  # [n][M][P][H][D]
        cand, _ = _scale_of(x.abs().amax((2, 4)))
        d_old = torch.where(had, sc[..., part], 0.0)
        d = torch.maximum(cand, d_old)
        inv = torch.where(d > 0, 1 / d, 0.0)
        ratio = torch.where(d > 0, d_old / d, 0.0)
        c = _codes(x, inv[:, :, None, :, None]).permute(0, 1, 3, 2, 4)  # [n][M][H][P][D]
        if part == 0:
            was = rec[..., 16:16 + P * D].unflatten(-1, (D // 64, P, 64)).transpose(-2, -3).flatten(-2)
        else:
            was = rec[..., 16 + P * D:].unflatten(-1, (D, P)).transpose(-1, -2)
        kept = ((was.float() - 128) * ratio[..., None, None]).round()
        f, o = fresh[:, :, None, :, None], old[:, :, None, :, None]
        now = torch.where(f, c + 128, torch.where(o, kept + 128, was.float())).to(torch.uint8)
        if part == 0:
            body.append(now.unflatten(-1, (D // 64, 64)).transpose(-2, -3).flatten(-3))
            if bounds is not None:
                bd = bounds[phys][..., 16:].view(torch.int8).unflatten(-1, (2, D)).float()
                bd = (bd * ratio[..., None, None]).round()
                lo = torch.where(had[..., None], bd[..., 0, :], 127.0)
                hi = torch.where(had[..., None], bd[..., 1, :], -127.0)
                lo = torch.minimum(lo, torch.where(f, c, 127.0).amin(-2))
                hi = torch.maximum(hi, torch.where(f, c, -127.0).amax(-2))
                extremes = torch.stack([lo, hi], -2).to(torch.int8).view(torch.uint8).flatten(-2)
        else:
            body.append(now.transpose(-1, -2).flatten(-2))
        new_sc.append(d)
    head = torch.stack(new_sc, -1).contiguous().view(torch.uint8)
    pool[phys] = torch.cat([head, rec[..., 8:16], body[0], body[1]], -1)
    if bounds is not None:
        key = new_sc[0][..., None].contiguous().view(torch.uint8)
        bounds[phys] = torch.cat([key, torch.zeros_like(rec[..., :12]), extremes], -1)


def _plain_read(case, st):
    P, dt = case["page"], st["k"].dtype
    kc, vc = _views(case, st)
    seq, pos = _token_places(st, st["back"], st["n_back"])
    phys, slot = st["table"].long()[seq, pos // P], pos % P
    sc = _scales(st["pool"])[phys]
    k = (kc[phys, :, :, slot].flatten(-2).float() - 128) * sc[..., :1]
    v = (vc[phys, :, :, slot].float() - 128) * sc[..., 1:]
    return {"k": k.to(dt), "v": v.to(dt)}


def _softmax(s, mask):
    """Softmax over the last axis of what the mask lets through; zeros where it lets nothing through."""
    s = torch.where(mask, s, -torch.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top.isfinite(), top, 0.0))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0)


def _plain_attend(case, st):
    P, D, H = case["page"], case["dim"], case["kv_heads"]
    G, T, n = case["heads"] // H, st["max_new"], case["seqs"]
    seq, pos = _token_places(st, st["starts"], st["n_tok"])
    i = torch.arange(st["n_tok"], device=pos.device) - st["starts"].long()[seq]
    q = torch.zeros(n, T, H, G, D, device=pos.device)
    q[seq, i] = st["q"].float().unflatten(1, (H, G))
    at = torch.full((n, T), -1, device=pos.device)
    at[seq, i] = pos
    rec = st["pool"][st["table"].clamp(min=0).long()]  # [n][pages][H][..]
    sc = _scales(rec)
    k = (rec[..., 16:16 + P * D].unflatten(-1, (D // 64, P, 64)).transpose(-2, -3).flatten(-2).float() - 128) * sc[..., :1, None]
    v = (rec[..., 16 + P * D:].unflatten(-1, (D, P)).transpose(-1, -2).float() - 128) * sc[..., 1:, None]
    k, v = (a.transpose(1, 2).flatten(2, 3) for a in (k, v))  # [n][H][tokens][D]
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [n][H][T G][D]
    s = (q @ k.transpose(-1, -2)) / math.sqrt(D)
    key = torch.arange(k.shape[2], device=pos.device)
    mask = key <= at[..., None]
    if case["window"]:
        mask &= key > at[..., None] - case["window"]
    p = _softmax(s, mask.repeat_interleave(G, 1)[:, None])
    o = (p @ v).unflatten(2, (T, G)).permute(0, 2, 1, 3, 4)
    return o[seq, i].flatten(1, 2).to(st["q"].dtype)


def _plain_select(case, st):
    P, D, H = case["page"], case["dim"], case["kv_heads"]
    seq, pos = _token_places(st, st["starts"], st["n_tok"])
    q = st["q"].float().unflatten(1, (H, -1))
    dq, inv = _scale_of(q.abs().amax(-1, keepdim=True))
    qc = _codes(q, inv)
    b = st["bounds"][st["table"].clamp(min=0).long()]  # [n][pages][H][..]
    dk = b[..., :4].contiguous().view(torch.float32)[..., 0].transpose(1, 2)[seq]
    ext = b[..., 16:].view(torch.int8).unflatten(-1, (2, D)).float().permute(0, 2, 3, 4, 1)[seq]  # [t][H][2][D][pages]
    # whole numbers below 2^24: exact in fp32 in any order
    u = qc.clamp(min=0) @ ext[:, :, 1] + qc.clamp(max=0) @ ext[:, :, 0]
    score = (u * dq).amax(2) * dk
    page = torch.arange(score.shape[-1], device=score.device)
    last = (pos // P)[:, None, None]
    score = torch.where(page == last, torch.inf, torch.where(page < last, score, -torch.inf))
    n = min(case["select"], score.shape[-1])
    top, ids = score.sort(dim=-1, descending=True, stable=True)
    none = score.shape[-1]
    ids = torch.where(top[..., :n] > -torch.inf, ids[..., :n], none).sort(-1).values
    ids = torch.nn.functional.pad(ids, (0, case["select"] - n), value=none)
    return torch.where(ids == none, -1, ids).to(torch.int32)


def _plain_attend_pages(case, st, ids):
    P, D, H = case["page"], case["dim"], case["kv_heads"]
    seq, pos = _token_places(st, st["starts"], st["n_tok"])
    ids = ids.long()
    phys = st["table"].long()[seq[:, None, None], ids.clamp(min=0)]  # [t][H][n]
    rec = st["pool"][phys, torch.arange(H, device=phys.device)[None, :, None]]
    sc = _scales(rec)
    k = (rec[..., 16:16 + P * D].unflatten(-1, (D // 64, P, 64)).transpose(-2, -3).flatten(-2).float() - 128) * sc[..., :1, None]
    v = (rec[..., 16 + P * D:].unflatten(-1, (D, P)).transpose(-1, -2).float() - 128) * sc[..., 1:, None]
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    key = (ids[..., None] * P + torch.arange(P, device=phys.device)).flatten(2)
    mask = (key <= pos[:, None, None]) & (ids >= 0).repeat_interleave(P, 2)
    q = st["q"].float().unflatten(1, (H, -1))
    p = _softmax((q @ k.transpose(-1, -2)) / math.sqrt(D), mask[:, :, None])
    return (p @ v).flatten(1, 2).to(st["q"].dtype)


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    e = SIZES[case["dtype"]]
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        per = e * (1 + 2 * case["residual"]) + (e if case["out"] != "q8" else 0) + (2 if case["out"] != "float" else 0)
        return {"bytes": n * per + 4 * case["dim"], "flops": 6 * n}
    H, D, P, G = case["kv_heads"], case["dim"], case["page"], case["heads"] // case["kv_heads"]
    lens, news = _lengths(case)
    if case["op"] == "append":
        back = sum(t - (t - c) // P * P for t, c in zip(lens, news))
        return {"bytes": 2 * H * D * (sum(news) * (e + 1) + back * e), "flops": 4 * H * D * sum(news)}
    io = 2 * e * sum(news) * case["heads"] * D
    if case["op"] == "attend":
        w = case["window"] or max(lens)
        seen = sum(min(t, w + c - 1) for t, c in zip(lens, news))
        pairs = sum(min(t - j, w) for t, c in zip(lens, news) for j in range(c))
        return {"bytes": io + seen * H * (2 * D + 8 / P), "flops": 4 * pairs * case["heads"] * D}
    pages = [-(-t // P) for t in lens]
    some = sum(min(p, case["select"]) for p in pages)
    return {"bytes": io + 2 * e * sum(news) * H * D + sum(pages) * H * (2 * D + 4) + some * H * (2 * P * D + 8),
            "flops": 4 * some * P * case["heads"] * D + 4 * sum(pages) * case["heads"] * D}


# --------------------------------------------------------------------------
# The operators' definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, st)
    H, D, P = case["kv_heads"], case["dim"], case["page"]
    lens, news = _lengths(case)
    table = st["table"].cpu().numpy()
    starts = np.concatenate([[0], np.cumsum(news)])
    pool = st["pool"].cpu().numpy()

    def load(page):  # one page's codes and scales, [H][P][D] each
        r = pool[page]
        sc = np.ascontiguousarray(r[:, :8]).view(np.float32)
        k = r[:, 16:16 + P * D].reshape(H, D // 64, P, 64).transpose(0, 2, 1, 3).reshape(H, P, D).astype(np.float64) - 128
        v = r[:, 16 + P * D:].reshape(H, D, P).transpose(0, 2, 1).astype(np.float64) - 128
        return [k, v], [sc[:, 0].copy(), sc[:, 1].copy()]

    changed = {}  # pages that the new tokens touch, as the append leaves them
    if case["op"] in ("append", "sparse"):
        xs = [st["k"].float().cpu().numpy(), st["v"].float().cpu().numpy()]
        ext = {}
        for s, (t, c) in enumerate(zip(lens, news)):
            for page in range((t - c) // P, (t - 1) // P + 1):
                lo, hi = max(t - c, page * P) - page * P, min(t, page * P + P) - page * P
                a = starts[s] + page * P + lo - (t - c)
                phys = table[s, page]
                codes, sc = load(phys)
                for part in (0, 1):
                    x = xs[part][a:a + hi - lo].transpose(1, 0, 2)  # [H][m][D]
                    d_old = sc[part] if lo else np.zeros(H, np.float32)
                    # scales and codes are defined in fp32
                    d = np.maximum(np.abs(x).max((1, 2)) / np.float32(127), d_old)
                    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
                        inv = np.where(d > 0, np.float32(1) / d, np.float32(0))
                        ratio = np.where(d > 0, d_old / d, np.float32(0)).astype(np.float32)
                        z = np.nan_to_num(x * inv[:, None, None], nan=0.0, posinf=127, neginf=-127)
                    codes[part][:, :lo] = np.rint(codes[part][:, :lo].astype(np.float32) * ratio[:, None, None])
                    codes[part][:, lo:hi] = np.clip(np.rint(z), -127, 127)
                    sc[part] = d
                    if part == 0 and st["bounds"] is not None:
                        mine = codes[0][:, lo:hi]
                        low, top = mine.min(1), mine.max(1)
                        if lo:
                            b = st["bounds"][int(phys)].cpu().numpy()[:, 16:].view(np.int8).astype(np.float32).reshape(H, 2, D)
                            b = np.rint(b * ratio[:, None, None])
                            low, top = np.minimum(low, b[:, 0]), np.maximum(top, b[:, 1])
                        ext[phys] = (low, top, sc[0])
                changed[phys] = (codes, sc)
    if case["op"] == "append":
        ks, vs = [], []
        for s, (t, c) in enumerate(zip(lens, news)):
            for page in range((t - c) // P, (t - 1) // P + 1):
                codes, sc = changed[table[s, page]]
                m = min(P, t - page * P)
                ks.append((codes[0][:, :m] * sc[0].astype(np.float64)[:, None, None]).transpose(1, 0, 2))
                vs.append((codes[1][:, :m] * sc[1].astype(np.float64)[:, None, None]).transpose(1, 0, 2))
        return {"k": torch.from_numpy(np.concatenate(ks)), "v": torch.from_numpy(np.concatenate(vs))}

    G = case["heads"] // H
    q = st["q"].float().cpu().numpy().reshape(-1, H, G, D)
    out = torch.zeros(st["n_tok"], H, G, D, dtype=torch.float64)
    for phys, (codes, sc) in changed.items():
        r = np.zeros((H, 16 + 2 * P * D), np.uint8)
        r[:, :8] = np.stack(sc, -1).astype(np.float32).view(np.uint8)
        r[:, 16:16 + P * D] = (codes[0] + 128).reshape(H, P, D // 64, 64).transpose(0, 2, 1, 3).reshape(H, -1)
        r[:, 16 + P * D:] = (codes[1] + 128).transpose(0, 2, 1).reshape(H, -1)
        st["pool"][int(phys)] = torch.from_numpy(r).cuda()
    picks = None
    if case["op"] == "sparse":
        picks = np.full((st["n_tok"], H, case["select"]), -1, np.int32)
        amax = np.abs(q).max(-1, keepdims=True)
        dq = amax / np.float32(127)
        with np.errstate(divide="ignore", invalid="ignore"):
            z = np.nan_to_num(q * np.where(dq > 0, np.float32(1) / dq, np.float32(0)), nan=0.0)
        qc = np.clip(np.rint(z), -127, 127).astype(np.float64)
    for s, (t, c) in enumerate(zip(lens, news)):
        have = -(-t // P)
        rec = st["pool"][torch.from_numpy(table[s, :have].astype(np.int64)).cuda()]
        sc = rec[..., :8].contiguous().view(torch.float32).double()
        if picks is not None:
            b = st["bounds"][torch.from_numpy(table[s, :have].astype(np.int64)).cuda()].cpu().numpy()
            low = b[..., 16:16 + D].view(np.int8).astype(np.float64)
            top = b[..., 16 + D:].view(np.int8).astype(np.float64)
            dk = np.ascontiguousarray(b[..., :4]).view(np.float32)[..., 0].copy()
            for page in range((t - c) // P, have):
                low[page], top[page], dk[page] = ext[table[s, page]]
        for h in range(H):
            k = (rec[:, h, 16:16 + P * D].reshape(have, D // 64, P, 64).permute(0, 2, 1, 3).reshape(have, P, D).double() - 128) * sc[:, h, :1, None]
            v = (rec[:, h, 16 + P * D:].reshape(have, D, P).permute(0, 2, 1).double() - 128) * sc[:, h, 1:, None]
            for j in range(c):
                i, pos = starts[s] + j, t - c + j
                lo, hi = max(0, pos - case["window"] + 1) if case["window"] else 0, pos + 1
                keys, vals = k.reshape(-1, D), v.reshape(-1, D)
                if picks is None:
                    keys, vals = keys[lo:hi], vals[lo:hi]
                else:
                    x = qc[i, h]  # [G][D]
                    u = np.maximum(x, 0) @ top[:, h].T + np.minimum(x, 0) @ low[:, h].T
                    score = (u.astype(np.float32) * dq[i, h]).max(0) * dk[:, h]
                    score[pos // P] = np.inf
                    chosen = np.sort(np.argsort(-score, kind="stable")[:case["select"]])
                    picks[i, h, :len(chosen)] = chosen
                    at = torch.from_numpy((chosen[:, None] * P + np.arange(P)).reshape(-1)).cuda()
                    at = at[at <= pos]
                    keys, vals = keys[at], vals[at]
                w = torch.from_numpy(q[i, h]).double().cuda() @ keys.T / math.sqrt(D)
                out[i, h] = (torch.softmax(w, -1) @ vals).cpu()
    out = out.flatten(1, 2)
    return out if picks is None else {"ids": torch.from_numpy(picks), "out": out}


def _exact_norm(case, st):
    x = st["x"].cpu().double().numpy()
    out = {}
    if st["r"] is not None:
        x = x + st["r"].cpu().double().numpy()
        out["res"] = torch.from_numpy(x)
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + EPS) * st["w"].cpu().double().numpy()
    if case["out"] != "q8":
        out["y"] = torch.from_numpy(y)
    if case["out"] != "float":
        b = y.reshape(y.shape[0], -1, 32)
        d = np.abs(b).max(-1, keepdims=True) / 127
        d = np.where(d > 0, d, 1.0)
        out["y8"] = torch.from_numpy((np.rint(b / d) * d).reshape(y.shape))
    return out
