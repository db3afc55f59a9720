"""Plain model of the paged 8-bit K/V cache: numpy, float64, position by position.

Written from the format's definition (include/nt.h, nt_kv8_cache) without the library; tables, lengths, counts and the page
operators are the 4-bit cache's model's.
"""
import numpy as np

import kv4_ref

EMIN, EMAX = -100, 100
MOST = 448.0 * 2.0 ** EMAX


def _number(b):
    e, m, s = b >> 3 & 15, b & 7, -1.0 if b & 128 else 1.0
    return np.nan if b & 127 == 127 else s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


NUMBER = np.array([_number(b) for b in range(256)])          # what each code stands for
_UP = NUMBER[:127]                                           # 0 .. 448, ascending


def code(x):
    """Codes of numbers up to 448 in magnitude (NaN: 127): the nearest, ties to the even code."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isnan(x), 0, x))
    i = np.clip(np.searchsorted(_UP, a, side="right") - 1, 0, 126)
    j = np.minimum(i + 1, 126)
    up = (a - _UP[i] > _UP[j] - a) | ((a - _UP[i] == _UP[j] - a) & (i % 2 == 1) & (j > i))
    c = np.where(up, j, i) | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, c).astype(np.uint8)


def exponent(x):
    """Exponent that the values need."""
    a = np.abs(np.asarray(x, np.float64))
    a = a[a <= MOST]
    top = a.max() if a.size else 0.0
    e = EMIN
    if top > 448 * 2.0 ** EMIN:
        e = int(np.floor(np.log2(top / 448))) - 1
        while 448 * 2.0 ** e < top:
            e += 1
    return max(e, EMIN)


def codes(x, e):
    x = np.asarray(x, np.float64)
    return code(np.where(np.abs(x) <= MOST, x * 2.0 ** -e, np.nan))


def rotate(x, pos, freq):
    """[rows, heads, hd] by the rows' positions, rounded to fp32 once."""
    if freq is None:
        return np.asarray(x, np.float32)
    x = np.asarray(x, np.float64)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(freq)
    c, s = np.cos(ang), np.sin(ang)
    out = np.empty(x.shape)
    with np.errstate(invalid="ignore", over="ignore"):
        out[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
        out[..., 1::2] = x[..., 0::2] * s + x[..., 1::2] * c
        return out.astype(np.float32)


class RefCache(kv4_ref.RefCache):
    def __init__(self, n_layers, n_kv, hd, page_len, n_pages, max_seqs, max_pages, fill=0):
        super().__init__(1, n_kv, hd, page_len, 1, max_seqs, max_pages)
        self.shape.update(n_layers=n_layers, n_pages=n_pages)
        self.L, self.P = n_layers, n_pages
        self.page_bytes = n_kv * (2 * page_len * hd + 16 + 2 * hd)
        self.pool = np.full((n_layers, n_pages, self.page_bytes), fill, np.uint8)
        self.refs = np.zeros(n_pages, np.int32)

    # -- addresses within a page -----------------------------------------------
    def k_at(self, g, t, d):
        return g * 2 * self.pl * self.hd + t // 8 * (8 * self.hd) + d // 16 * 128 + t % 8 * 16 + d % 16

    def v_at(self, g, t, d):
        return (2 * g + 1) * self.pl * self.hd + t // 16 * (16 * self.hd) + d * 16 + t % 16

    def exp_at(self, g, v):
        return self.n_kv * 2 * self.pl * self.hd + g * (16 + 2 * self.hd) + v

    def page_kv(self, row, g):
        """float64 K and V [page_len, hd] of a page's bytes, and its exponents."""
        t, d = np.arange(self.pl)[:, None], np.arange(self.hd)
        e = [int(row[self.exp_at(g, v):][:1].view(np.int8)[0]) for v in (0, 1)]
        return NUMBER[row[self.k_at(g, t, d)]], NUMBER[row[self.v_at(g, t, d)]], e

    def bounds(self, row, g):
        at = self.exp_at(g, 0) + 16
        return row[at:at + 2 * self.hd].view(np.int8).astype(np.int64).reshape(2, self.hd)

    def randomize(self, rng):
        """Random codes (NaN aside), exponents near -8 and bounds that hold for the keys, in every page."""
        c = rng.integers(0, 254, self.pool.shape).astype(np.uint8)
        self.pool[:] = np.where(c >= 127, c + 1, c)
        for row in self.pool.reshape(-1, self.page_bytes):
            for g in range(self.n_kv):
                for v in (0, 1):
                    row[self.exp_at(g, v)] = np.int8(rng.integers(-9, -6)).view(np.uint8)
                k = self.page_kv(row, g)[0]
                at = self.exp_at(g, 0) + 16
                row[at:at + 2 * self.hd] = np.concatenate([np.floor(k.min(0) / 4), np.ceil(k.max(0) / 4)]).astype(np.int8).view(np.uint8)

    def kv(self, layer, s, g, n=None):
        """float64 [n, hd] keys and values of a sequence."""
        n = int(self.len[s]) if n is None else n
        ks, vs = [np.zeros((0, self.hd))], [np.zeros((0, self.hd))]
        for j in range(self.pages(n)):
            k, v, e = self.page_kv(self.pool[layer, self.table[s, j]], g)
            ks.append(k * 2.0 ** e[0])
            vs.append(v * 2.0 ** e[1])
        return np.concatenate(ks)[:n], np.concatenate(vs)[:n]

    # -- rows ----------------------------------------------------------------------
    def append(self, layer, s, k, v, freq=None):
        """fp32 (or f16) rows [R, kv, hd] become the last positions of sequence s."""
        R, n = len(k), int(self.len[s])
        pos = np.arange(n - R, n)
        k, v = rotate(k, pos, freq).astype(np.float64), np.asarray(v, np.float64)
        d = np.arange(self.hd)
        for j in sorted(set(pos // self.pl)):
            mine = pos // self.pl == j
            at = pos[mine] % self.pl
            row = self.pool[layer, self.table[s, j]]
            fresh, older = at[0] == 0, np.arange(at[0])[:, None]
            for g in range(self.n_kv):
                for i, x, where in ((0, k[mine, g], self.k_at), (1, v[mine, g], self.v_at)):
                    was = int(row[self.exp_at(g, i):][:1].view(np.int8)[0])
                    e = exponent(x)
                    if not fresh:
                        e = max(e, was)
                        held = NUMBER[row[where(g, older, d)]]
                        row[where(g, older, d)] = code(held * 2.0 ** (was - e))
                    row[self.exp_at(g, i)] = np.int8(e).view(np.uint8)
                    new = codes(x, e)
                    row[where(g, at[:, None], d)] = new
                    if i:
                        continue
                    y = NUMBER[new]
                    nan = np.isnan(y).any(0)
                    y = np.where(nan, 0, y)
                    lo = np.where(nan, -127, np.floor(y.min(0) / 4))
                    hi = np.where(nan, 127, np.ceil(y.max(0) / 4))
                    if not fresh:
                        b = self.bounds(row, g).astype(np.float64)
                        lo = np.minimum(lo, np.where(b[0] == -127, -127, np.floor(b[0] * 2.0 ** (was - e))))
                        hi = np.maximum(hi, np.where(b[1] == 127, 127, np.ceil(b[1] * 2.0 ** (was - e))))
                    where_b = self.exp_at(g, 0) + 16
                    row[where_b:where_b + 2 * self.hd] = np.concatenate([lo, hi]).astype(np.int8).view(np.uint8)

    # -- selection -------------------------------------------------------------------
    def select(self, layer, s, g, q, top, first, last, n=None):
        """Places of the pages that the group's queries q [G, hd] (fp32) choose, -1 behind."""
        n = int(self.len[s]) if n is None else n
        m = self.pages(n)
        q = np.asarray(q, np.float64)
        size = np.abs(q[np.isfinite(q)])
        big = size.max() if size.size else 0.0
        f = 0
        if big > 0:
            f = int(np.floor(np.log2(big / 63))) - 1
            while 63 * 2.0 ** f < big:
                f += 1
        w = np.where(np.isnan(q), 0, np.clip(np.where(np.isinf(q), np.sign(q) * 63 * 2.0 ** f, q) * 2.0 ** -f, -63, 63))
        w = np.rint(np.nan_to_num(w)).astype(np.int64)
        score = np.zeros(m)
        for j in range(m):
            p = self.table[s, j]
            if 0 <= p < self.P:
                lo, hi = self.bounds(self.pool[layer, p], g)
                e = int(self.pool[layer, p][self.exp_at(g, 0):][:1].view(np.int8)[0])
                score[j] = float(np.maximum(w * lo, w * hi).sum()) * 2.0 ** e
        place = np.arange(m)
        score[(place < first) | (place >= m - last)] = np.inf
        pick = np.sort(np.argsort(-score, kind="stable")[:top])
        return np.concatenate([pick, np.full(top - len(pick), -1)]).astype(np.int32)


def attend(q, k, v):
    """float64 attention of [G, hd] queries over [T, hd], and what bounds its error: out [G, hd], the weighted magnitudes
    sum p |v| [G, hd], the largest sum |q||k| / sqrt(hd) [G, 1], the sum of the weights relative to the largest [G, 1]."""
    if len(k) == 0:
        z = np.zeros(q.shape)
        return z, z, z[:, :1], z[:, :1] + 1
    r = 1 / np.sqrt(q.shape[1])
    s = q @ k.T * r
    w = np.exp(s - s.max(1, keepdims=True))
    p = w / w.sum(1, keepdims=True)
    return p @ v, p @ np.abs(v), (np.abs(q) @ np.abs(k).T).max(1, keepdims=True) * r, w.sum(1, keepdims=True)
