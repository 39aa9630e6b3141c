"""Plain restatement of the paged 8-bit cache, its attention and its page
selection, one (page, head) or token at a time: bytes and picks as the header
defines them (scales and codes in fp32 operations), sums in 64 bits."""
import numpy as np

F = np.float32


def rule(x, d):
    """The activation rule's codes of x under scale d (fp32)."""
    with np.errstate(all="ignore"):
        inv = F(1) / d if d > 0 else F(0)
        z = (x.astype(F) * inv).astype(F)
        z = np.where(np.isnan(z), F(0), z)
        return np.clip(np.rint(z), -127, 127).astype(np.int32)


class Cache:
    """Byte image of the library's cache; every byte starts as `fill`."""

    def __init__(self, H, D, P, n_pages, fill=0xFF):
        self.H, self.D, self.P = H, D, P
        self.pages = np.full((n_pages, H, 16 + 2 * P * D), fill, np.uint8)
        self.bounds = np.full((n_pages, H, 16 + 2 * D), fill, np.uint8)

    def scales(self, page, h):
        return self.pages[page, h, :8].view(F)

    def codes(self, page, h):
        """(K [P][D], V [P][D]) int32 codes."""
        r = self.pages[page, h, 16:].astype(np.int32) - 128
        n = self.P * self.D
        k = r[:n].reshape(self.D // 64, self.P, 64).transpose(1, 0, 2).reshape(self.P, self.D)
        return k, r[n:].reshape(self.D, self.P).T

    def put(self, page, h, k, v):
        P, D = self.P, self.D
        body = np.concatenate([(k + 128).reshape(P, D // 64, 64).transpose(1, 0, 2).ravel(), (v + 128).T.ravel()])
        self.pages[page, h, 16:] = body.astype(np.uint8)

    def extremes(self, page, h):
        b = self.bounds[page, h]
        return b[:4].view(F)[0], b[16:16 + self.D].view(np.int8).astype(np.int32), \
            b[16 + self.D:].view(np.int8).astype(np.int32)

    def append(self, k, v, table, lens, starts):
        """k, v fp32 [n_tok][H][D]: the last starts[s+1] - starts[s] tokens of each sequence."""
        for s, length in enumerate(lens):
            n = starts[s + 1] - starts[s]
            pos = length - n
            while pos < length:
                pg, lo = divmod(pos, self.P)
                m = min(length - pos, self.P - lo)
                a = starts[s] + pos - (length - n)
                for h in range(self.H):
                    self._append(table[s, pg], h, lo, k[a:a + m, h], v[a:a + m, h])
                pos += m

    def _append(self, page, h, lo, k, v):
        sc = self.scales(page, h)
        old = list(self.codes(page, h))
        m = len(k)
        for part, x in enumerate((k, v)):
            d_old = sc[part] if lo else F(0)
            d = max(d_old, np.abs(x).max().astype(F) / F(127))
            ratio = F(d_old / d) if d > 0 else F(0)
            c = old[part].copy()
            c[:lo] = np.rint(c[:lo].astype(F) * ratio).astype(np.int32)
            c[lo:lo + m] = rule(x, d)
            if part == 0:
                low, top = c[lo:lo + m].min(0), c[lo:lo + m].max(0)
                if lo:
                    _, bl, bt = self.extremes(page, h)
                    low = np.minimum(low, np.rint(bl.astype(F) * ratio).astype(np.int32))
                    top = np.maximum(top, np.rint(bt.astype(F) * ratio).astype(np.int32))
                b = self.bounds[page, h]
                b[:4] = np.array([d], F).view(np.uint8)
                b[16:16 + self.D] = low.astype(np.int8).view(np.uint8)
                b[16 + self.D:] = top.astype(np.int8).view(np.uint8)
            old[part] = c
            sc[part] = d
        self.put(page, h, *old)

    def values(self, table_row, h, length):
        """(K, V) of positions [0, length) of a sequence, 64 bits."""
        ks, vs = [np.zeros((0, self.D))], [np.zeros((0, self.D))]
        for pg in range(-(-length // self.P)):
            k, v = self.codes(table_row[pg], h)
            sc = self.scales(table_row[pg], h).astype(np.float64)
            m = min(self.P, length - pg * self.P)
            ks.append(k[:m] * sc[0])
            vs.append(v[:m] * sc[1])
        return np.concatenate(ks), np.concatenate(vs)


def attend(cache, q, table, lens, starts, scale, causal=True, window=0, pages=None):
    """(out, sum of weight * |v|, largest scale * max|q| * sum|k|) in 64 bits."""
    n_tok, heads, D = q.shape
    G = heads // cache.H
    out, mag, arg = np.zeros((n_tok, heads, D)), np.zeros((n_tok, heads, D)), np.zeros((n_tok, heads, 1))
    for s, length in enumerate(lens):
        n = starts[s + 1] - starts[s]
        for h in range(cache.H):
            k, v = cache.values(table[s], h, length)
            for i in range(n):
                t, pos = starts[s] + i, length - n + i
                see = np.arange(length)
                keep = np.ones(length, bool)
                if causal:
                    keep &= see <= pos
                if window:
                    keep &= see > pos - window
                if pages is not None:
                    keep &= np.isin(see // cache.P, pages[t, h][pages[t, h] >= 0])
                if not keep.any():
                    continue
                for g in range(h * G, h * G + G):
                    x = q[t, g].astype(np.float64)
                    z = scale * (k[keep] @ x)
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    out[t, g] = w @ v[keep]
                    mag[t, g] = w @ np.abs(v[keep])
                    arg[t, g] = abs(scale) * np.abs(x).max() * np.abs(k[keep]).sum(1).max()
    return out, mag, arg


def select(cache, q, table, lens, starts, n_sel):
    n_tok, heads, D = q.shape
    G = heads // cache.H
    ids = np.full((n_tok, cache.H, n_sel), -1, np.int32)
    for s, length in enumerate(lens):
        n = starts[s + 1] - starts[s]
        for i in range(n):
            t, pos = starts[s] + i, length - n + i
            if pos < 0:
                continue
            last = pos // cache.P
            for h in range(cache.H):
                qs = []
                for g in range(h * G, h * G + G):
                    d = np.abs(q[t, g]).max().astype(F) / F(127)
                    qs.append((d, rule(q[t, g], d)))
                score = np.empty(last, F)
                for pg in range(last):
                    dk, low, top = cache.extremes(table[s, pg], h)
                    score[pg] = max(F(F(np.maximum(c * low, c * top).sum()) * d) for d, c in qs) * dk
                best = np.argsort(-score, kind="stable")[:n_sel - 1] if n_sel > 1 else np.zeros(0, int)
                pick = np.sort(np.concatenate([best, [last]]))
                ids[t, h, :len(pick)] = pick
    return ids
