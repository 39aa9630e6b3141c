"""Plain 64-bit forms of the head norm and rotation, adapters, expert selection
and log probabilities (numpy; loops over tokens)."""
import numpy as np


def positions(lens, starts, n_tok):
    """Each token's position, None where no sequence covers it."""
    at = [None] * n_tok
    for s in range(len(lens)):
        a, b = starts[s], starts[s + 1]
        for t in range(a, b):
            at[t] = lens[s] - (b - a) + t - a
    return at


def norm_rope(x, w, eps, pos, axis, freq, interleaved, scale):
    """x [n][H][D] float64, pos list of per-axis position lists (None: left out).  Returns (y, magnitude): the sum of
    the absolute values that each result is a difference of."""
    n, H, D = x.shape
    R = 2 * len(freq)
    y, mag = np.full(x.shape, np.nan), np.full(x.shape, np.nan)
    for t in range(n):
        if pos[t] is None:
            continue
        u = x[t]
        if w is not None:
            u = u * (1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)) * w
        y[t], mag[t] = u, np.abs(u)
        for i in range(R // 2):
            angle = float(int(pos[t][axis[i]])) * float(freq[i])
            c, s = np.cos(angle), np.sin(angle)
            one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            a, b = u[:, one], u[:, two]
            y[t, :, one], y[t, :, two] = scale * (a * c - b * s), scale * (b * c + a * s)
            mag[t, :, one] = mag[t, :, two] = abs(scale) * (np.abs(a) + np.abs(b))
    return y, mag


def lora(A, B, ids, x, r, scales, ranks):
    """Returns (y, magnitude of the sums)."""
    y, mag = r.copy(), np.zeros_like(r)
    for t, a in enumerate(ids):
        if 0 <= a < len(A):
            k = A.shape[1] if ranks is None else min(max(int(ranks[a]), 0), A.shape[1])
            s = 1.0 if scales is None else float(scales[a])
            y[t] += s * (B[a][:, :k] @ (A[a][:k] @ x[t]))
            mag[t] = abs(s) * (np.abs(B[a][:, :k]) @ (np.abs(A[a][:k]) @ np.abs(x[t])))
    return y, mag


def route(logits, top_k, sigmoid, bias, groups, keep, group_top, renorm, scale):
    """Picks and gates, and each pick's distance of its logit from the row's largest."""
    n, E = logits.shape
    size = E // groups
    ids, gates, below = np.zeros((n, top_k), np.int32), np.zeros((n, top_k)), np.zeros((n, top_k))
    for t in range(n):
        l = np.where(np.isnan(logits[t]), -np.inf, np.minimum(logits[t], np.finfo(np.float32).max))
        top = l.max()
        with np.errstate(all="ignore"):
            if sigmoid:
                s = np.where(l == -np.inf, 0.0, 1 / (1 + np.exp(-l)))
            elif top == -np.inf:
                s = np.zeros(E)
            else:
                s = np.where(l == -np.inf, 0.0, np.exp(l - top))
                s = s / s.sum()
        c = s + (0.0 if bias is None else bias)
        c = np.where(np.isnan(c), -np.inf, c)
        score = [sum(sorted(c[g * size:(g + 1) * size])[::-1][:group_top]) for g in range(groups)]
        kept = sorted(range(groups), key=lambda g: (-score[g], g))[:keep]
        key = l if bias is None else c
        mine = [e for g in sorted(kept) for e in range(g * size, (g + 1) * size)]
        ids[t] = sorted(mine, key=lambda e: (-key[e], e))[:top_k]
        w = s[ids[t]]
        total = w.sum()
        gates[t] = scale * (w if not renorm else w / total if total > 0 else np.zeros(top_k))
        with np.errstate(all="ignore"):
            d = np.abs(l[ids[t]] - top)
        below[t] = np.where(np.isfinite(d), np.minimum(d, 200), 0)
    return ids, gates, below


def logprobs(logits, tokens, n_top, scale):
    """(logp, lse, entropy, ids, top), and s = the sum over the row but for its largest term, relative to that."""
    n, V = logits.shape
    out = [np.zeros((n, tokens.shape[1])) if tokens is not None else None, np.zeros(n), np.zeros(n),
           np.full((n, n_top), -1, np.int32), np.full((n, n_top), -np.inf)]
    rest = np.zeros(n)
    for r in range(n):
        l = logits[r]
        fine = l[~np.isnan(l)]
        bad = len(fine) < V or (fine == np.inf).any()
        order = [i for i in np.lexsort((np.arange(V), -np.where(np.isnan(l), -np.inf, l)))[:n_top]
                 if not np.isnan(l[i]) and l[i] > -np.inf]
        out[3][r, :len(order)] = order
        top = fine.max() if len(fine) else -np.inf
        if bad:
            logs, lse, h = np.full(V, np.nan), np.nan, np.nan
        elif top == -np.inf:
            logs, lse, h = np.full(V, -np.inf), -np.inf, 0.0
        else:
            d = (l - top) * scale
            e = np.exp(d)
            first = int(np.argmax(l))
            rest[r] = e[:first].sum() + e[first + 1:].sum()
            log_s = np.log1p(rest[r])
            logs, lse = d - log_s, top * scale + log_s
            h = log_s - np.where(e > 0, e * np.where(e > 0, d, 0), 0).sum() / (1 + rest[r])
        out[1][r], out[2][r] = lse, h
        out[4][r, :len(order)] = logs[order]
        if tokens is not None:
            for j, t in enumerate(tokens[r]):
                out[0][r, j] = 0.0 if t < 0 else np.nan if t >= V else logs[t]
    return (*out, rest)
