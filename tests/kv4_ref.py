"""Plain model of the paged 4-bit K/V cache: numpy and Python loops, float64 attention.

Written from the format's definition (include/nt.h, nt_kv4_cache) without the library: byte addresses of codes and scales,
the quantizer in fp32 steps, the page operators as list manipulation.
"""
import numpy as np

BAD_SEQ, BAD_LEN, BAD_PAGE, NO_PAGE = 1, 2, 4, 8


def scale_of(block):
    """f16 scale of 32 fp32 values: max|x| by 1 / 7 in fp32, to f16, to six mantissa bits; NaN where it cannot be held."""
    block = np.asarray(block, np.float32)
    if not np.isfinite(block).all():
        return np.float16(np.nan)
    with np.errstate(over="ignore"):
        h = np.float16(np.float32(np.abs(block).max()) * np.float32(1 / 7))
    bits = (int(h.view(np.uint16)) + 8) & 0xFFF0
    d = np.array([bits], np.uint16).view(np.float16)[0]
    return d if np.isfinite(d) and d <= 896 else np.float16(np.nan)


def codes_of(block, d):
    if not np.isfinite(d) or d == 0:
        return np.full(32, 8, np.int64)
    r = (np.asarray(block, np.float32) / np.float32(d)).astype(np.float64)
    r = np.sign(r) * np.floor(np.abs(r) + 0.5)              # halves away from zero
    return np.clip(r + 8, 0, 15).astype(np.int64)


def quantize(x):
    """fp32 [..., hd] -> (codes [..., hd] int64, scales [..., hd / 32] f16)."""
    x = np.asarray(x, np.float32)
    b = x.reshape(-1, 32)
    d = np.array([scale_of(r) for r in b], np.float16)
    q = np.stack([codes_of(r, s) for r, s in zip(b, d)]) if len(b) else np.zeros((0, 32), np.int64)
    return q.reshape(x.shape), d.reshape(x.shape[:-1] + (x.shape[-1] // 32,))


def values(q, d):
    """float64 values of codes and scales."""
    b = (q.reshape(q.shape[:-1] + (q.shape[-1] // 32, 32)) - 8).astype(np.float64) * d.astype(np.float64)[..., None]
    return b.reshape(q.shape)


class RefCache:
    def __init__(self, n_layers, n_kv, hd, page_len, n_pages, max_seqs, max_pages, fill=0):
        self.shape = dict(n_layers=n_layers, n_kv_heads=n_kv, head_dim=hd, page_len=page_len, n_pages=n_pages,
                          max_seqs=max_seqs, max_pages=max_pages)
        self.L, self.n_kv, self.hd, self.pl, self.P = n_layers, n_kv, hd, page_len, n_pages
        self.S, self.M, self.ng = max_seqs, max_pages, hd // 32
        self.chunk = 18 * hd
        self.page_bytes = n_kv * (page_len // 16) * self.chunk
        self.pool = np.full((n_layers, n_pages, self.page_bytes), fill, np.uint8)
        self.table = np.full((max_seqs, max_pages), -1, np.int32)
        self.len = np.zeros(max_seqs, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.error = 0

    # -- addresses ------------------------------------------------------------
    def _chunk(self, g, at):
        return (g * (self.pl // 16) + at // 16) * self.chunk

    def _k_code(self, g, at, e):
        p = at % 16
        return self._chunk(g, at) + ((p * 4 + e % 32 // 8) * self.ng + e // 32) * 4 + e % 8 // 2, 4 * (e % 2)

    def _v_code(self, g, at, e):
        p = at % 16
        w = ((p // 8 * 8 + e % 32 // 4) * 4 + p % 8 // 2) * self.ng + e // 32
        return self._chunk(g, at) + 8 * self.hd + 4 * w + 2 * (p % 2) + e % 4 // 2, 4 * (e % 2)

    def _k_scale(self, g, at, j):
        return self._chunk(g, at) + 16 * self.hd + 2 * (at % 16 * self.ng + j)

    def _v_scale(self, g, at, j):
        p = at % 16
        return self._chunk(g, at) + 17 * self.hd + 2 * ((p // 2 * self.ng + j) * 2 + p % 2)

    def put(self, layer, page, g, at, k, v):
        """One position's key and value (fp32 vectors) of one kv head."""
        row = self.pool[layer, page]
        for x, code, scale in ((k, self._k_code, self._k_scale), (v, self._v_code, self._v_scale)):
            q, d = quantize(x)
            for e in range(self.hd):
                b, sh = code(g, at, e)
                row[b] = (int(row[b]) & ~(15 << sh)) | int(q[e]) << sh
            for j in range(self.ng):
                b = scale(g, at, j)
                row[b:b + 2] = np.array([d[j]], np.float16).view(np.uint8)

    def get(self, layer, page, g, at):
        """float64 key and value of one position and kv head."""
        e, j = np.arange(self.hd), np.arange(self.ng)
        row = self.pool[layer, page]
        out = []
        for code, scale in ((self._k_code, self._k_scale), (self._v_code, self._v_scale)):
            b, sh = code(g, at, e)
            q = (row[b].astype(np.int64) >> sh) & 15
            s = scale(g, at, j)
            d = np.stack([row[s], row[s + 1]], -1).copy().view(np.float16)[:, 0]
            out.append(values(q, d))
        return out

    def kv(self, layer, s, g):
        """float64 [len, hd] keys and values of a sequence."""
        t = np.arange(int(self.len[s]))
        page, at, pool = self.table[s, t // self.pl][:, None], (t % self.pl)[:, None], self.pool[layer]
        e, j, out = np.arange(self.hd), np.arange(self.ng), []
        for code, scale in ((self._k_code, self._k_scale), (self._v_code, self._v_scale)):
            b, sh = code(g, at, e)
            d = scale(g, at, j)
            d = (pool[page, d].astype(np.uint16) | pool[page, d + 1].astype(np.uint16) << 8).view(np.float16)
            out.append(values((pool[page, b].astype(np.int64) >> sh) & 15, d))
        return out

    def randomize(self, rng, lo=0.05, hi=0.4):
        """Random codes and scales in every page."""
        self.pool[:] = rng.integers(0, 256, self.pool.shape, np.uint8)
        d = rng.uniform(lo, hi, (self.L, self.P, self.n_kv, self.pl // 16, self.hd)).astype(np.float16).view(np.uint16) & 0xFFF0
        self.pool.reshape(self.L, self.P, self.n_kv, self.pl // 16, -1)[..., 16 * self.hd:] = d.view(np.uint8)

    def hold(self, lens, rng=None):
        """Sequences 0.. of the given lengths, their pages in a random order."""
        order = list(range(self.P)) if rng is None else list(rng.permutation(self.P))
        for s, n in enumerate(lens):
            for k in range(self.pages(n)):
                self.table[s, k] = order.pop()
                self.refs[self.table[s, k]] = 1
            self.len[s] = n

    # -- operators --------------------------------------------------------------
    def pages(self, n):
        return -(-n // self.pl)

    def free_pages(self, n):
        return [p for p in range(self.P) if self.refs[p] == 0][:n]

    def extend(self, seqs, counts):
        bad, plan = 0, []
        for i, (s, c) in enumerate(zip(seqs, counts)):
            if not 0 <= s < self.S:
                bad |= BAD_SEQ
                continue
            if s in list(seqs)[:i]:
                bad |= BAD_SEQ
            n = int(self.len[s])
            if c < 0 or n + c > self.M * self.pl:
                bad |= BAD_LEN
                continue
            tail = int(self.table[s, n // self.pl]) if c and n % self.pl else -1
            copied = tail >= 0 and self.refs[tail] > 1
            plan.append((s, n, c, tail if copied else -1, self.pages(n + c) - self.pages(n) + copied))
        pages = self.free_pages(sum(x[4] for x in plan))
        if not bad and len(pages) < sum(x[4] for x in plan):
            bad |= NO_PAGE
        self.error |= bad
        if bad:
            return
        for s, n, c, tail, need in plan:
            mine, pages = pages[:need], pages[need:]
            for p in mine:
                self.refs[p] = 1
            if tail >= 0:
                self.pool[:, mine[0]] = self.pool[:, tail]
                self.refs[tail] -= 1
                self.table[s, n // self.pl] = mine[0]
                mine = mine[1:]
            for k, p in enumerate(mine):
                self.table[s, self.pages(n) + k] = p
            self.len[s] = n + c

    def fork(self, src, dst, keep=None):
        bad, need = 0, 0
        keep = [int(self.len[s]) if 0 <= s < self.S else 0 for s in src] if keep is None else list(keep)
        for i, (s, d, k) in enumerate(zip(src, dst, keep)):
            if not 0 <= d < self.S or d in list(dst)[:i] or not 0 <= s < self.S or s in list(dst) or self.len[d] != 0:
                bad |= BAD_SEQ
            if 0 <= s < self.S and not 0 <= k <= self.len[s]:
                bad |= BAD_LEN
            need += k % self.pl != 0
        pages = self.free_pages(need)
        if not bad and len(pages) < need:
            bad |= NO_PAGE
        self.error |= bad
        if bad:
            return
        for s, d, k in zip(src, dst, keep):
            full = k // self.pl
            self.table[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                self.refs[p] += 1
            if k % self.pl:
                p = pages.pop(0)
                self.refs[p] = 1
                self.pool[:, p] = self.pool[:, self.table[s, full]]
                self.table[d, full] = p
            self.len[d] = k

    def free(self, seqs, keep=None):
        keep = [0] * len(seqs) if keep is None else keep
        for i, (s, k) in enumerate(zip(seqs, keep)):
            if not 0 <= s < self.S or s in list(seqs)[:i]:
                self.error |= BAD_SEQ
                continue
            if not 0 <= k <= self.len[s]:
                self.error |= BAD_LEN
                continue
            for j in range(self.pages(k), self.pages(int(self.len[s]))):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.len[s] = k

    def copy_pages(self, src, dst):
        before = self.pool.copy()
        for i, (s, d) in enumerate(zip(src, dst)):
            others = [x for j, x in enumerate(dst) if j != i]
            if not (0 <= s < self.P and 0 <= d < self.P) or d in list(dst)[:i] or s in others:
                self.error |= BAD_PAGE
                continue
            self.pool[:, d] = before[:, s]

    def compact(self):
        used = [p for p in range(self.P) if self.refs[p] > 0]
        n = len(used)
        to = {p: p for p in used}
        to.update(zip([p for p in used if p >= n], [p for p in range(n) if self.refs[p] <= 0]))
        refs = np.zeros_like(self.refs)
        for p, d in to.items():
            refs[d] = self.refs[p]
            if p != d:
                self.pool[:, d] = self.pool[:, p]
        table = self.table.copy()
        for e in np.ndindex(table.shape):
            if table[e] >= 0:
                table[e] = to[int(table[e])]
        return table, refs, n


def attend(q, k, v):
    """float64 softmax attention of one query over [T, hd] keys and values; zeros where T = 0."""
    if len(k) == 0:
        return np.zeros(len(q))
    s = k @ q / np.sqrt(len(q))
    p = np.exp(s - s.max())
    return p @ v / p.sum()
