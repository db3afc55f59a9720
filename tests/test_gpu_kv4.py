"""GPU: the paged 4-bit K/V cache -- rows in and out, attention, page operators and a run of them together -- against the
plain model of kv4_ref.py (whole bytes, tables and counts equal; attention within a bound derived from its arithmetic)."""
import numpy as np
import pytest

import kv4_ref as R
from gpu_util import torch_cuda, ensure_built

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def nt():
    torch_cuda()
    ensure_built()
    from quantized_decode_dequant_gb300 import nt as _nt
    return _nt


class Dev:
    """A RefCache's buffers on the device, and the library's calls on them."""

    def __init__(self, nt, ref, n_heads=None, pool=None):
        import torch
        self.nt, self.torch, self.ref = nt, torch, ref
        up = lambda a: torch.from_numpy(a.copy()).cuda()   # noqa: E731
        self.pool = up(ref.pool) if pool is None else pool
        self.table, self.len, self.refs = up(ref.table), up(ref.len), up(ref.refs)
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.c = nt.make_kv4_cache(**ref.shape, pool=self.pool.data_ptr(), table=self.table.data_ptr(),
                                   len=self.len.data_ptr(), refs=self.refs.data_ptr(), error=self.error.data_ptr())
        self.heads = n_heads or ref.n_kv
        self.wb = nt.nt_kv4_workspace_bytes(self.c, self.heads, max(ref.S, 8))
        self.ws = torch.full((self.wb,), 0x7F, dtype=torch.uint8, device="cuda")
        self.alive = []

    def ints(self, x):
        if x is None:
            return None
        t = self.torch.tensor(list(map(int, x)), dtype=self.torch.int32, device="cuda")
        self.alive.append(t)
        return t.data_ptr()

    def stream(self):
        return self.torch.cuda.current_stream()

    def extend(self, seqs, counts):
        self.nt.nt_kv4_extend(self.c, len(counts), self.ints(seqs), self.ints(counts), self.ws.data_ptr(), self.wb,
                              self.stream())

    def fork(self, src, dst, keep=None):
        self.nt.nt_kv4_fork(self.c, len(src), self.ints(src), self.ints(dst), self.ints(keep), self.ws.data_ptr(), self.wb,
                            self.stream())

    def free(self, seqs, keep=None):
        self.nt.nt_kv4_free(self.c, len(seqs), self.ints(seqs), self.ints(keep), self.stream())

    def copy_pages(self, src, dst):
        self.nt.nt_kv4_copy_pages(self.c, len(src), self.ints(src), self.ints(dst), self.stream())

    def compact(self, table_out=None, refs_out=None):
        live = self.torch.full((1,), -7, dtype=self.torch.int32, device="cuda")
        table_out = self.table if table_out is None else table_out
        refs_out = self.refs if refs_out is None else refs_out
        self.nt.nt_kv4_compact(self.c, table_out.data_ptr(), refs_out.data_ptr(), live.data_ptr(), self.ws.data_ptr(),
                               self.wb, self.stream())
        return int(live.cpu()[0])

    def rows(self, k, v, begin, seqs=None, layer=0, read=False):
        """append or read torch k, v [rows, kv, hd] of any strides; begin None: a row each."""
        n = (len(begin) - 1) if begin is not None else (len(seqs) if seqs is not None else k.shape[0])
        f = self.nt.nt_kv4_read if read else self.nt.nt_kv4_append
        assert k.stride() == v.stride()
        f(self.c, layer, n, self.ints(seqs), self.ints(begin), k.shape[0], "f16" if k.dtype == self.torch.float16 else "f32",
          k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), self.stream())

    def attention(self, q, seqs=None, layer=0, q_stride=None, out=None, out_stride=None, ws=None, stream=None):
        torch, n = self.torch, q.shape[0]
        row = self.heads * self.ref.hd
        out = torch.full((n, out_stride or row), float("inf"), device="cuda") if out is None else out
        self.nt.nt_attention_kv4(self.c, layer, self.heads, n, self.ints(seqs), q.data_ptr(), q_stride or row,
                                 out.data_ptr(), out_stride or row, (self.ws if ws is None else ws).data_ptr(), self.wb,
                                 stream or self.stream())
        return out

    def check(self, error=0):
        """The device's state is the model's."""
        self.torch.cuda.synchronize()
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.ref.table)
        np.testing.assert_array_equal(self.len.cpu().numpy(), self.ref.len)
        np.testing.assert_array_equal(self.refs.cpu().numpy(), self.ref.refs)
        np.testing.assert_array_equal(self.pool.cpu().numpy(), self.ref.pool)
        assert int(self.error.cpu()[0]) == error == self.ref.error


# -------------------------------------------------------------- append, read --

def _rows(rng, n, n_kv, hd):
    x = rng.standard_normal((2, n, n_kv, hd)) * np.exp(rng.standard_normal((2, n, n_kv, 1)) * 2)
    return x.astype(np.float32)


def _layout(torch, x, how):
    """[rows, kv, hd] k and v of x [2, rows, kv, hd] as a user may hold them."""
    t = torch.from_numpy(x).cuda()
    if how == "rows":            # a projection's rows
        return t[0], t[1]
    if how == "cache":           # [kv][position][dim]
        t = t.transpose(1, 2).contiguous().transpose(1, 2)
        return t[0], t[1]
    t = t.permute(1, 0, 2, 3).contiguous()   # K and V next to each other in every row
    return t[:, 0], t[:, 1]


def _store(ref, x, begin, seqs, layer=0):
    for i, s in enumerate(seqs):
        n = begin[i + 1] - begin[i]
        for r in range(begin[i], begin[i + 1]):
            pos = int(ref.len[s]) - n + r - begin[i]
            for g in range(ref.n_kv):
                ref.put(layer, int(ref.table[s, pos // ref.pl]), g, pos % ref.pl, x[0, r, g], x[1, r, g])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("how", ["rows", "cache", "side"])
def test_append_and_read_are_exact(nt, hd, half, how):
    torch = torch_cuda()
    rng = np.random.default_rng([hd, half])
    ref = R.RefCache(2, 3, hd, 48, 12, 5, 4, fill=0xC3)
    ref.hold([50, 1, 0, 191, 17], rng)
    dev = Dev(nt, ref)
    seqs, begin = [3, 0, 4, 1], [2, 103, 120, 121, 122]   # rows 0, 1 and those behind 122 belong to nobody
    x = _rows(rng, 130, 3, hd)
    if half:
        x = x.astype(np.float16)
    k, v = _layout(torch, x, how)
    dev.rows(k, v, begin, seqs, layer=1)
    _store(ref, x.astype(np.float32), begin, seqs, layer=1)
    dev.check()
    out = torch.full((2,) + tuple(k.shape), 5.5, dtype=k.dtype, device="cuda").cpu().numpy()
    ko, vo = _layout(torch, out, how)
    dev.rows(ko, vo, begin, seqs, layer=1, read=True)
    torch.cuda.synchronize()
    want = np.full(x.shape, 5.5)
    for side in (0, 1):
        want[side, 2:122] = R.values(*R.quantize(x[side, 2:122]))
    np.testing.assert_array_equal(torch.stack([ko, vo]).cpu().numpy().astype(np.float64), want)
    dev.check()


@pytest.mark.parametrize("n", [1, 2, 5])
def test_one_token_each_without_lists(nt, n):
    torch = torch_cuda()
    rng = np.random.default_rng(n)
    ref = R.RefCache(1, 2, 64, 16, 12, 5, 3)
    ref.hold([1, 16, 17, 33, 48], rng)
    dev = Dev(nt, ref)
    x = _rows(rng, n, 2, 64)
    k, v = _layout(torch, x, "rows")
    dev.rows(k, v, None)
    _store(ref, x, list(range(n + 1)), list(range(n)))
    dev.check()
    # more rows than sequences (a padded batch): those behind are not read
    y = np.concatenate([x, np.full((2, 3, 2, 64), np.nan, np.float32)], 1)
    k, v = _layout(torch, y, "rows")
    nt.nt_kv4_append(dev.c, 0, n, None, None, n + 3, "f32", k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1),
                     dev.stream())
    dev.check()


def test_blocks_that_cannot_be_held_read_as_nan_and_others_are_exact(nt):
    torch = torch_cuda()
    rng = np.random.default_rng(9)
    x = _rows(rng, 24, 1, 64)
    for r, v in enumerate([np.nan, np.inf, -np.inf, 6400.0, -1e30, 7 * 896.0, 65504.0, 3e38]):
        x[:, r, 0, 7] = v                     # the first block of eight rows; the second block stays ordinary
    x[:, 8] = 0
    x[:, 9] = 6.5 * 2.0 ** -21
    x[:, 10] *= 1e-6
    x[:, 11] *= 1e-38
    x[:, 12, 0, :8] = [7, -7, 3.5, -3.5, 0.5, -0.5, 1.5, 2.5]   # halves, scale 1
    x[:, 12, 0, 8:32] = np.nextafter(np.float32(0.5), np.float32(0))
    x[:, 13] = -0.0
    ref = R.RefCache(1, 1, 64, 16, 2, 1, 2)
    ref.hold([24])
    dev = Dev(nt, ref)
    k, v = _layout(torch, x, "rows")
    dev.rows(k, v, [0, 24])
    _store(ref, x, [0, 24], [0])
    dev.check()
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    dev.rows(ko, vo, [0, 24], read=True)
    want = R.values(*R.quantize(x[0]))
    np.testing.assert_array_equal(ko.cpu().numpy().astype(np.float64), want)
    assert np.isnan(want[[0, 1, 2, 3, 4, 6, 7], 0, :32]).all() and np.isfinite(want[:8, 0, 32:]).all()


@pytest.mark.parametrize("half", [False, True])
def test_quotients_next_to_halves(nt, half):
    """Values at, just below and just above every half of the scale, for scales over the whole range: the codes are those
    of the fp32 quotient, halves away from zero."""
    torch = torch_cuda()
    rng = np.random.default_rng(33)
    ref = R.RefCache(1, 1, 128, 16, 32, 1, 32)
    ref.hold([512])
    dev = Dev(nt, ref)
    kind = np.float16 if half else np.float32
    x = np.zeros((2, 512, 1, 128), np.float32)
    bits = rng.integers(1, 0x631, (2, 512, 4)).astype(np.uint16) << 4        # scales that the format holds
    d = bits.view(np.float16).astype(np.float64)
    for side in (0, 1):
        for r in range(512):
            for j in range(4):
                h = (rng.integers(0, 7, 32) + 0.5) * rng.choice([-1, 1], 32)
                v = (h * d[side, r, j]).astype(kind)
                way = rng.integers(-2, 3, 32)                                    # steps of the type towards 0 or away
                for _ in range(2):
                    v = np.where(way > 0, np.nextafter(v, kind(np.inf) * np.sign(v)), np.where(way < 0, np.nextafter(v, kind(0)), v))
                    way = way - np.sign(way)
                v[int(rng.integers(0, 32))] = 7 * d[side, r, j]
                x[side, r, 0, 32 * j:32 * j + 32] = v
    x = x.astype(kind)
    k, v = _layout(torch, x, "rows")
    dev.rows(k, v, [0, 512])
    _store(ref, x.astype(np.float32), [0, 512], [0])
    dev.check()


def test_rows_that_do_not_fit_are_flagged_and_passed_over(nt):
    torch = torch_cuda()
    rng = np.random.default_rng(10)

    def fresh():
        ref = R.RefCache(1, 1, 64, 16, 8, 4, 3, fill=1)
        ref.hold([20, 3, 0, 40], rng)
        return ref, Dev(nt, ref)

    x = _rows(rng, 6, 1, 64)
    k, v = _layout(torch, x, "rows")
    # out-of-range sequences; a row count above the length; the good entry between them is stored
    ref, dev = fresh()
    dev.rows(k, v, [0, 1, 2, 4, 6], [-1, 4, 0, 2])
    _store(ref, x, [2, 4], [0])
    ref.error = R.BAD_SEQ | R.BAD_LEN
    dev.check(ref.error)
    # a page that is shared, one that nobody holds, one out of range
    for what in ("shared", "unheld", "low", "high"):
        ref, dev = fresh()
        page = int(ref.table[3, 2])
        if what == "shared":
            ref.refs[page] = 2
        elif what == "unheld":
            ref.refs[page] = 0
        else:
            ref.table[3, 2] = -5 if what == "low" else ref.P
        dev = Dev(nt, ref)
        dev.rows(k, v, [0, 2, 6], [1, 3])
        _store(ref, x, [0, 2], [1])
        ref.error = R.BAD_PAGE
        dev.check(R.BAD_PAGE)
    # a length that the table cannot hold
    ref, _ = fresh()
    ref.len[3] = 49
    dev = Dev(nt, ref)
    dev.rows(k, v, [0, 2, 6], [1, 3])
    _store(ref, x, [0, 2], [1])
    ref.error = R.BAD_LEN
    dev.check(R.BAD_LEN)
    # a sequence listed twice is flagged
    ref, dev = fresh()
    dev.rows(k, v, [0, 1, 2, 3], [1, 0, 1])
    torch.cuda.synchronize()
    assert int(dev.error.cpu()[0]) == R.BAD_SEQ
    # row ranges that run backwards
    ref, dev = fresh()
    dev.rows(k, v, [3, 1, 5], [0, 3])
    torch.cuda.synchronize()


# ---------------------------------------------------------------- attention --

def _bound(ref, s, q, heads, layer=0):
    """First-order error bound of each head's output, from the kernel's arithmetic.
    K and V are exact.  q, scaled by a power of two so that its largest element is of the order 2^10, and the softmax
    weights, scaled so that the largest is at least 2^6, enter the f16 matrix products as hi = f16(x) and lo = f16(x - hi):
    relative residual 2^-22, and 2^-25 absolute where lo falls below f16's normal range (2^-35 of the largest q, 2^-31
    of the largest weight).  A score sums hd / 16 steps in fp32, two roundings a step (u = 2^-24), then three roundings
    of the score itself on the way to the exponent:
      |ds| <= ((hd / 16 + 3) 2u + 2^-22) sum |q K| / sqrt(hd) + 2^-35 max|q| sum|K| / sqrt(hd) + 6u max|s|.
    A change ds of the scores moves the output by at most 2 max|V| max|ds|.  The weights' exponential is within 2^-22,
    their split 2^-22; sums of weights and of weighted V take one step of two roundings per 16 positions, and at most 64
    more where partial results meet, each in numerator and denominator."""
    n, hd, G = int(ref.len[s]), ref.hd, heads // ref.n_kv
    out = np.zeros(heads)
    for j in range(heads if n else 0):
        k, v = ref.kv(layer, s, j // G)
        dot, sc = np.abs(k) @ np.abs(q[j]) / np.sqrt(hd), np.abs(k @ q[j]) / np.sqrt(hd)
        ds = (((hd // 16 + 3) * 2 * U + 2.0 ** -22) * dot).max() + 6 * U * sc.max()
        ds += 2.0 ** -35 * np.abs(q[j]).max() * np.abs(k).sum(1).max() / np.sqrt(hd)
        vm = np.abs(v).max()
        out[j] = 2 * vm * ds + vm * ((n / 16 + 64) * 4 * U + 3 * 2.0 ** -22 + n * 2.0 ** -31)
    return out


def _want(ref, seqs, q, heads, layer=0):
    G = heads // ref.n_kv
    out = np.zeros((len(seqs), heads, ref.hd))
    for i, s in enumerate(seqs):
        for g in range(ref.n_kv):
            k, v = ref.kv(layer, s, g)
            for j in range(g * G, (g + 1) * G):
                out[i, j] = R.attend(q[i, j], k, v)
    return out


# (n_kv, G, hd, page_len, lengths)
SHAPES = [
    (8, 8, 128, 64, [4161]),                                   # one 70B-shaped sequence
    (8, 4, 128, 32, [0, 1, 15, 16, 17, 31, 32, 33, 700, 0]),   # 8B-shaped, lengths on the chunk and page boundaries
    (2, 4, 64, 16, [37]),                                      # the tiny model
    (2, 4, 64, 16, [1]),
    (1, 16, 128, 48, [3001, 5, 49]),                           # one kv head, 16 query heads
    (3, 16, 64, 256, [255, 256, 257, 1023]),
    (4, 1, 128, 16, [129, 1, 0, 640, 333]),                    # a query head per kv head
    (5, 2, 64, 112, [111, 112, 113, 2000]),
    (1, 1, 64, 16, [16000]),                                   # long and narrow: many CTAs on one head
    (2, 8, 128, 16, [(i * 37) % 90 for i in range(70)]),       # many short ones
]


@pytest.mark.parametrize("n_kv,G,hd,page_len,lens", SHAPES)
@pytest.mark.parametrize("q_std", [0.3, 4.0])
def test_attention_matches_float64(nt, n_kv, G, hd, page_len, lens, q_std):
    torch = torch_cuda()
    rng = np.random.default_rng([n_kv, G, hd, page_len])
    pages = sum(-(-n // page_len) for n in lens)
    ref = R.RefCache(1, n_kv, hd, page_len, pages + 2, len(lens), max(1, max(-(-n // page_len) for n in lens)) + 1)
    ref.randomize(rng)
    ref.hold(lens, rng)
    heads = n_kv * G
    dev = Dev(nt, ref, heads)
    q = (rng.standard_normal((len(lens), heads, hd)) * q_std).astype(np.float32)
    got = dev.attention(torch.from_numpy(q).cuda()).cpu().numpy().reshape(q.shape)
    want = _want(ref, range(len(lens)), q.astype(np.float64), heads)
    assert int(dev.error.cpu()[0]) == 0
    worst = 0.0
    for s, n in enumerate(lens):
        if n == 0:
            assert (got[s].view(np.uint32) == 0).all()
            continue
        b = _bound(ref, s, q[s].astype(np.float64), heads)
        err = np.abs(got[s] - want[s]).max(axis=1)
        assert (err <= b).all(), (s, n, float((err / b).max()))
        worst = max(worst, float((err / b).max()))
        if 1 < n < 400 and q_std < 1:
            # the bound sees a position too few
            ref.len[s] -= 1
            less = _want(ref, [s], q[s:s + 1].astype(np.float64), heads)[0]
            ref.len[s] += 1
            assert (np.abs(less - want[s]).max(axis=1) > b).any(), n
    rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
    print(f"kv {n_kv} G {G} hd {hd} page {page_len} n {len(lens)}: rel L2 {rel:.2e}, at most {worst:.2f} of the bound")


def test_attention_ignores_what_lies_behind_the_end(nt):
    """NaN and infinite scales, all-ones codes in dead positions, dead pages and other layers change no bit."""
    torch = torch_cuda()
    rng = np.random.default_rng(31)
    for hd, G in ((64, 4), (128, 16), (128, 2)):
        lens = [1, 5, 16, 45, 150]
        ref = R.RefCache(2, 2, hd, 32, 20, 5, 6)
        ref.randomize(rng)
        ref.hold(lens, rng)
        q = torch.from_numpy(rng.standard_normal((5, 2 * G, hd)).astype(np.float32)).cuda()
        first = Dev(nt, ref, 2 * G).attention(q, layer=1).cpu().numpy()
        for fill in (0xFFFF, 0x7C00, 0xFC00):   # NaN, and the two infinities
            other = R.RefCache(2, 2, hd, 32, 20, 5, 6)
            other.pool.view(np.uint16)[:] = fill
            other.table, other.len, other.refs = ref.table, ref.len, ref.refs
            k = np.arange(hd)
            for s, n in enumerate(lens):
                for t in range(n):
                    page, at = int(ref.table[s, t // 32]), t % 32
                    for g in range(2):
                        for code, scale in ((ref._k_code, ref._k_scale), (ref._v_code, ref._v_scale)):
                            for b in [code(g, at, k)[0], scale(g, at, np.arange(ref.ng)), scale(g, at, np.arange(ref.ng)) + 1]:
                                other.pool[1, page, b] = ref.pool[1, page, b]
            got = Dev(nt, other, 2 * G).attention(q, layer=1).cpu().numpy()
            np.testing.assert_array_equal(got.view(np.uint32), first.view(np.uint32))


def test_attention_lists_strides_workspaces_and_streams(nt):
    torch = torch_cuda()
    rng = np.random.default_rng(41)
    ref = R.RefCache(1, 2, 128, 32, 60, 6, 12)
    ref.randomize(rng)
    ref.hold([333, 40, 0, 97, 350, 8], rng)
    dev = Dev(nt, ref, 16)
    seqs = [4, 4, 0, 2, 5, 4, 3]
    q = torch.from_numpy(rng.standard_normal((7, 16, 128)).astype(np.float32)).cuda()
    first = dev.attention(q, seqs).cpu().numpy()
    q64 = q.cpu().numpy().astype(np.float64)
    want = _want(ref, seqs, q64, 16)
    for i, s in enumerate(seqs):
        assert (np.abs(first[i].reshape(16, 128) - want[i]).max(axis=1) <= _bound(ref, s, q64[i], 16)).all()
    wide = torch.full((7, 16 * 128 + 64), float("nan"), device="cuda")
    wide[:, :2048] = q.view(7, -1)
    out = torch.full((7, 2048 + 12), 3.25, device="cuda")
    for fill in (0, 0xFF, 0x7F):
        dev.ws.fill_(fill)
        got = dev.attention(wide, seqs, q_stride=2112, out=out, out_stride=2060)
        np.testing.assert_array_equal(got[:, :2048].cpu().numpy().view(np.uint32), first.view(np.uint32))
        assert (got[:, 2048:] == 3.25).all()
    # two calls at once, a workspace each
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    w2 = torch.empty_like(dev.ws)
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append(dev.attention(q, seqs, stream=a))
        outs.append(dev.attention(q, seqs, stream=b, ws=w2))
    torch.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(o.cpu().numpy().view(np.uint32), first.view(np.uint32))


@pytest.mark.parametrize("n", [129, 300, 1024, 1500])
def test_attention_of_many_listed_sequences(nt, n):
    """Lists beyond what a warp counts for itself, and beyond one launch; a sequence's result does not depend on its place
    but for the order in which partial sums meet."""
    torch = torch_cuda()
    rng = np.random.default_rng(43)
    ref = R.RefCache(1, 1, 64, 16, 60, 9, 9)
    ref.randomize(rng)
    lens = [1, 0, 17, 140, 32, 33, 100, 5, 64]
    ref.hold(lens, rng)
    dev = Dev(nt, ref, 2)
    seqs = rng.integers(0, 9, n)
    q = rng.standard_normal((9, 2, 64)).astype(np.float32)
    got = dev.attention(torch.from_numpy(q[seqs]).cuda(), seqs).cpu().numpy().reshape(n, 2, 64)
    want = _want(ref, range(9), q.astype(np.float64), 2)
    for s in range(9):
        b = _bound(ref, s, q[s].astype(np.float64), 2)
        assert (np.abs(got[seqs == s] - want[s]).max(axis=(0, 2)) <= b).all(), s
    assert int(dev.error.cpu()[0]) == 0


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 8, 16])
def test_attention_with_much_work_for_every_warp(nt, hd, G):
    """Over 32 steps a warp, so that sums are put aside within an item and items follow one another; rising scores, so
    that the maximum moves on again and again."""
    torch = torch_cuda()
    rng = np.random.default_rng([47, hd, G])
    lens = [3001, 2800, 17, 3100]
    ref = R.RefCache(1, 1, hd, 64, 160, 4, 50)
    ref.randomize(rng)
    ref.hold(lens, rng)
    for s in (1, 3):   # the second and fourth sequence's keys grow with their place
        for j, page in enumerate(ref.table[s][ref.table[s] >= 0]):
            ref.pool.reshape(1, 160, 4, -1)[0, page, :, 16 * hd:17 * hd] = np.full(
                hd // 2, 0.02 * (j + 1), np.float16).view(np.uint16).__and__(0xFFF0).view(np.uint8)
    dev = Dev(nt, ref, G)
    seqs = np.arange(1000) % 4
    q = (rng.standard_normal((4, G, hd)) * 2).astype(np.float32)
    got = dev.attention(torch.from_numpy(q[seqs]).cuda(), seqs).cpu().numpy().reshape(1000, G, hd)
    want = _want(ref, range(4), q.astype(np.float64), G)
    for s in range(4):
        b = _bound(ref, s, q[s].astype(np.float64), G)
        err = np.abs(got[seqs == s] - want[s]).max(axis=(0, 2))
        assert (err <= b).all(), (s, float((err / b).max()))
        rel = np.linalg.norm(got[seqs == s] - want[s]) / np.linalg.norm(np.broadcast_to(want[s], got[seqs == s].shape))
        print(f"hd {hd} G {G} n {lens[s]}: rel L2 {rel:.2e}")


def test_attention_of_what_it_cannot_read_is_nan(nt):
    torch = torch_cuda()
    rng = np.random.default_rng(51)
    ref = R.RefCache(1, 2, 64, 16, 30, 5, 6)
    ref.randomize(rng)
    ref.hold([90, 33, 0, 50, 96], rng)
    q = torch.from_numpy(rng.standard_normal((7, 4, 64)).astype(np.float32)).cuda()
    seqs = [0, 1, 2, 3, 4, -1, 5]
    fine = Dev(nt, ref, 4).attention(q[:5]).cpu().numpy()
    ref.table[0, 3] = 30
    ref.table[1, 2] = -1
    ref.len[4] = 97
    ref.len[2] = -2
    dev = Dev(nt, ref, 4)
    got = dev.attention(q, seqs).cpu().numpy()
    assert np.isnan(got[[0, 1, 2, 4, 5, 6]]).all()
    np.testing.assert_array_equal(got[3], fine[3])
    assert int(dev.error.cpu()[0]) == R.BAD_SEQ | R.BAD_LEN | R.BAD_PAGE


def test_attention_of_nan_blocks_and_extreme_inputs(nt):
    """A NaN key block makes every output of its kv head NaN, a NaN value block only its 32 dimensions; large and tiny
    queries and values keep their relative precision."""
    torch = torch_cuda()
    rng = np.random.default_rng(61)
    ref = R.RefCache(1, 2, 128, 16, 10, 1, 8)
    ref.randomize(rng)
    ref.hold([100], rng)
    q = rng.standard_normal((1, 8, 128)).astype(np.float32)
    page, at = int(ref.table[0, 3]), 5
    nan = np.array([np.nan], np.float16).view(np.uint8)
    clean = ref.pool.copy()
    b = ref._v_scale(1, at, 2)
    ref.pool[0, page, b:b + 2] = nan
    got = Dev(nt, ref, 8).attention(torch.from_numpy(q).cuda()).cpu().numpy().reshape(8, 128)
    assert np.isnan(got[4:, 64:96]).all() and np.isfinite(got[:4]).all()
    assert np.isfinite(got[4:, :64]).all() and np.isfinite(got[4:, 96:]).all()
    ref.pool[:] = clean
    b = ref._k_scale(0, at, 1)
    ref.pool[0, page, b:b + 2] = nan
    got = Dev(nt, ref, 8).attention(torch.from_numpy(q).cuda()).cpu().numpy().reshape(8, 128)
    assert np.isnan(got[:4]).all() and np.isfinite(got[4:]).all()
    for lo, hi, qs in ((1e-4, 1e-4, 1.0), (0.1, 0.4, 1e-30), (0.1, 0.4, 3e4), (800.0, 890.0, 1e-4), (2e-5, 800.0, 1e-3)):
        ref.randomize(rng, lo, hi)
        dev = Dev(nt, ref, 8)
        qq = (q * np.float32(qs)).astype(np.float32)
        got = dev.attention(torch.from_numpy(qq).cuda()).cpu().numpy().reshape(8, 128)
        want = _want(ref, [0], qq.astype(np.float64), 8)[0]
        err, b = np.abs(got - want).max(axis=1), _bound(ref, 0, qq[0].astype(np.float64), 8)
        assert (err <= b).all(), (lo, hi, qs, float((err / b).max()))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("page_len", [16, 80, 256])
def test_attention_where_the_capacity_is_large(nt, hd, G, page_len):
    """Tables of 16384 positions and more a sequence, so that the work is shared out over the whole GPU: lengths around
    chunks, tiles and pages; a sequence twice; dead positions of every kind; a head of NaN beside others; bad pages."""
    torch = torch_cuda()
    rng = np.random.default_rng([83, hd, G, page_len])
    lens = [1, 15, 16, 17, 0, 127, 128, 129, 255, 256, 257, 700, 1500]
    need = sum(-(-n // page_len) for n in lens)
    ref = R.RefCache(1, 2, hd, page_len, need + 3, len(lens), -(-16384 // page_len))
    ref.randomize(rng)
    ref.hold(lens, rng)
    heads = 2 * G
    seqs = list(range(len(lens))) + [11, 3]
    q = rng.standard_normal((len(lens), heads, hd)).astype(np.float32)
    want = _want(ref, range(len(lens)), q.astype(np.float64), heads)
    qd = torch.from_numpy(q[seqs]).cuda()
    dev = Dev(nt, ref, heads)
    first = dev.attention(qd, seqs).cpu().numpy().reshape(len(seqs), heads, hd)
    for i, s in enumerate(seqs):
        err, b = np.abs(first[i] - want[s]).max(axis=1), _bound(ref, s, q[s].astype(np.float64), heads)
        assert (err <= b).all(), (lens[s], float((err / b).max()))
    assert int(dev.error.cpu()[0]) == 0
    np.testing.assert_array_equal(first[[13, 14]].view(np.uint32), dev.attention(qd, seqs).cpu().numpy().reshape(
        len(seqs), heads, hd)[[13, 14]].view(np.uint32))   # the same again, to the bit

    # dead positions: every scale NaN or infinite, every code 15
    k = np.arange(hd)
    for fill in (0xFFFF, 0x7C00):
        other = R.RefCache(1, 2, hd, page_len, need + 3, len(lens), -(-16384 // page_len))
        other.pool.view(np.uint16)[:] = fill
        other.table, other.len, other.refs = ref.table, ref.len, ref.refs
        for s, n in enumerate(lens):
            for t in range(n):
                page, at = int(ref.table[s, t // page_len]), t % page_len
                for g in range(2):
                    for code, scale in ((ref._k_code, ref._k_scale), (ref._v_code, ref._v_scale)):
                        b0 = scale(g, at, np.arange(ref.ng))
                        for b in [code(g, at, k)[0], b0, b0 + 1]:
                            other.pool[0, page, b] = ref.pool[0, page, b]
        got = Dev(nt, other, heads).attention(qd, seqs).cpu().numpy().reshape(len(seqs), heads, hd)
        np.testing.assert_array_equal(got.view(np.uint32), first.view(np.uint32))

    # a head's NaN or infinity is its own affair
    for bad in (np.nan, np.inf):
        odd = q[seqs].copy()
        odd[:, 1, 7] = bad
        got = dev.attention(torch.from_numpy(odd).cuda(), seqs).cpu().numpy().reshape(len(seqs), heads, hd)
        rest = [h for h in range(heads) if h != 1]
        for i, s in enumerate(seqs):
            if lens[s]:
                assert np.isnan(got[i, 1]).all()
                b = _bound(ref, s, q[s].astype(np.float64), heads)
                assert (np.abs(got[i] - want[s]).max(axis=1)[rest] <= b[rest]).all(), lens[s]

    # a page that is none, in the middle and at the end of a sequence; one behind the end is not looked at
    ref.table[11, 0], ref.table[12, (1500 - 1) // page_len] = -1, need + 3
    ref.table[5, -1] = need + 99
    dev = Dev(nt, ref, heads)
    got = dev.attention(qd, seqs).cpu().numpy().reshape(len(seqs), heads, hd)
    assert np.isnan(got[[11, 12, 13]]).all() and np.isfinite(np.delete(got, [11, 12, 13], 0)).all()
    fine = [i for i in range(len(seqs)) if i not in (11, 12, 13)]
    np.testing.assert_array_equal(got[fine].view(np.uint32), first[fine].view(np.uint32))
    assert int(dev.error.cpu()[0]) == R.BAD_PAGE


@pytest.mark.parametrize("hd,G", [(128, 4), (128, 8), (128, 16), (64, 8)])
def test_attention_replayed_and_on_two_streams_at_once(nt, hd, G):
    """The shared-out forms in a captured graph whose lengths change between replays, and two callers at once with a
    workspace each: to the bit what calls one after the other give."""
    torch = torch_cuda()
    rng = np.random.default_rng([97, hd, G])
    ref = R.RefCache(1, 4, hd, 64, 120, 4, 512)
    ref.randomize(rng)
    ref.hold([2000, 1500, 900, 1800], rng)
    dev = Dev(nt, ref, 4 * G)
    q = torch.from_numpy(rng.standard_normal((4, 4 * G, hd)).astype(np.float32)).cuda()
    out = torch.empty(4, 4 * G * hd, device="cuda")
    lens = [[2000, 1500, 900, 1800], [1, 0, 900, 129], [1999, 128, 16, 17], [0, 0, 0, 0]]
    eager = []
    for n in lens:
        dev.len.copy_(torch.tensor(n, dtype=torch.int32))
        eager.append(dev.attention(q).clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dev.attention(q, out=out, stream=torch.cuda.current_stream())
    for n, want in list(zip(lens, eager)) * 2:
        dev.len.copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(float("inf"))
        graph.replay()
        assert torch.equal(out.view(torch.int32), want.view(torch.int32)), n
    dev.len.copy_(torch.tensor(lens[0], dtype=torch.int32))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.full((dev.wb,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.full((20, 4, 4 * G * hd), float("inf"), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for st, ws, o in zip(streams, spaces, outs):
            with torch.cuda.stream(st):
                dev.attention(q, out=o[i], ws=ws, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        for i in range(20):
            assert torch.equal(o[i].view(torch.int32), eager[0].view(torch.int32))
    assert int(dev.error.cpu()[0]) == 0


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 8, 16])
def test_attention_of_many_short_sequences(nt, hd, G):
    """More (sequence, kv head) items than the GPU holds at once, each of few positions: 80, 300 and 1500 entries of nine
    sequences, empty ones among them, in any order."""
    torch = torch_cuda()
    rng = np.random.default_rng([103, hd, G])
    lens = [0, 1, 16, 17, 33, 64, 100, 191, 192]
    ref = R.RefCache(1, 3, hd, 16, 60, 9, 12)
    ref.randomize(rng)
    ref.hold(lens, rng)
    heads = 3 * G
    q = rng.standard_normal((9, heads, hd)).astype(np.float32)
    want = _want(ref, range(9), q.astype(np.float64), heads)
    bounds = [_bound(ref, s, q[s].astype(np.float64), heads) for s in range(9)]
    dev = Dev(nt, ref, heads)
    for n in (80, 300, 1500):
        seqs = rng.integers(0, 9, n)
        seqs[-3:] = [0, 8, 0]
        got = dev.attention(torch.from_numpy(q[seqs]).cuda(), seqs).cpu().numpy().reshape(n, heads, hd)
        for s in range(9):
            mine = got[seqs == s]
            assert (np.abs(mine - want[s]).max(axis=(0, 2)) <= bounds[s]).all(), (n, lens[s])
            assert lens[s] or (mine == 0).all()
    assert int(dev.error.cpu()[0]) == 0


def test_offsets_beyond_32_bits(nt):
    """A pool of over 4 GB whose used pages lie at its end, in the last layer."""
    torch = torch_cuda()
    rng = np.random.default_rng(71)
    small = R.RefCache(1, 8, 128, 64, 6, 2, 3)
    small.randomize(rng)
    small.hold([150, 65], rng)
    pages, layers = 20000, 4
    pool = torch.zeros(layers, pages, small.page_bytes, dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    pool[-1, pages - 6:] = torch.from_numpy(small.pool[0]).cuda()
    big = R.RefCache(1, 8, 128, 64, 1, 2, 3)
    big.shape.update(n_pages=pages, n_layers=layers)
    big.table = np.where(small.table >= 0, small.table + pages - 6, -1).astype(np.int32)
    big.len, big.refs = small.len, np.zeros(pages, np.int32)
    big.refs[big.table[big.table >= 0]] = 1
    dev = Dev(nt, big, 64, pool=pool)
    q = torch.from_numpy(rng.standard_normal((2, 64, 128)).astype(np.float32)).cuda()
    got = dev.attention(q, layer=layers - 1).cpu().numpy()
    np.testing.assert_array_equal(got, Dev(nt, small, 64).attention(q).cpu().numpy())
    x = _rows(rng, 70, 8, 128)
    k, v = _layout(torch, x, "rows")
    dev.rows(k, v, [0, 5, 70], layer=layers - 1)
    _store(small, x, [0, 5, 70], [0, 1])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(pool[-1, pages - 6:].cpu().numpy(), small.pool[0])
    src, dst = [pages - 6, pages - 1], [0, pages - 7]
    dev.copy_pages(src, dst)
    torch.cuda.synchronize()
    for s, d in zip(src, dst):
        assert (pool[:, s] == pool[:, d]).all()
    assert not pool[0].any() and int(dev.error.cpu()[0]) == 0


# ------------------------------------------------------------ page operators --

def _cache(seed, n_layers=2, page_len=16, n_pages=24, max_seqs=8, max_pages=6, hd=64, n_kv=1):
    ref = R.RefCache(n_layers, n_kv, hd, page_len, n_pages, max_seqs, max_pages)
    ref.randomize(np.random.default_rng(seed))
    return ref


@pytest.mark.parametrize("seed", range(6))
def test_random_page_operators_follow_the_model(nt, seed):
    """Long random runs of extend, fork, free, copy and compact, invalid entries among them: tables, lengths, counts,
    error bits and every byte of the pool stay equal."""
    rng = np.random.default_rng(100 + seed)
    ref = _cache(seed, n_layers=1 + seed % 3, page_len=[16, 48][seed % 2], n_pages=[24, 9, 40][seed % 3])
    dev = Dev(nt, ref)
    cap = ref.M * ref.pl
    for step in range(60):
        n = int(rng.integers(1, 5))
        wild = rng.random() < 0.2
        seqs = rng.integers(-1, ref.S + 1, n) if wild else rng.permutation(ref.S)[:n]
        op = rng.integers(0, 6)
        if op <= 1:
            counts = rng.integers(-1 if wild else 0, [40, 3][op], n)
            for x in (ref, dev):
                x.extend(list(seqs), list(counts))
        elif op == 2:
            empty = [s for s in range(ref.S) if ref.len[s] == 0]
            held = [s for s in range(ref.S) if ref.len[s] > 0]
            if not held or not empty:
                continue
            n = min(n, len(empty))
            dst = list(rng.permutation(empty)[:n]) if not wild else list(rng.integers(0, ref.S, n))
            src = list(rng.choice(held, n))
            keep = None if rng.random() < 0.5 else [int(rng.integers(0, ref.len[s] + 1 + wild)) for s in src]
            for x in (ref, dev):
                x.fork(src, dst, keep)
        elif op == 3:
            keep = None if rng.random() < 0.3 else [int(rng.integers(0, ref.len[s] + 1)) if 0 <= s < ref.S else 0 for s in seqs]
            for x in (ref, dev):
                x.free(list(seqs), keep)
        elif op == 4:
            src, dst = rng.integers(-wild, ref.P + wild, n), rng.integers(-wild, ref.P + wild, n)
            for x in (ref, dev):
                x.copy_pages(list(map(int, src)), list(map(int, dst)))
        else:
            table, refs, live = ref.compact()
            assert dev.compact() == live
            ref.table, ref.refs = table, refs
        dev.check(ref.error)
        assert int(ref.len.max()) <= cap


def test_extend_and_fork_change_nothing_when_they_fail(nt):
    ref = _cache(5, n_pages=6)
    dev = Dev(nt, ref)
    for x in (ref, dev):
        x.extend([0, 1], [40, 20])          # 3 + 2 pages of 6
        x.extend([2, 3], [16, 1])           # one page left, two wanted
    dev.check(R.NO_PAGE)
    for x in (ref, dev):
        x.extend([2, 9], [16, 1])
        x.extend([2, 2], [1, 1])
        x.extend([2, 0], [1, 57])           # 97 of 96 positions
        x.fork([0, 1], [4, 5])              # two tails, one page
        x.fork([0], [1])
        x.fork([0, 4], [4, 5])
        x.fork([0], [4], [41])
        x.fork([0, 0], [4, 4])
    dev.check(R.NO_PAGE | R.BAD_SEQ | R.BAD_LEN)
    for x in (ref, dev):
        x.fork([0], [7], [32])              # full pages alone need no page
        x.extend([2], [16])
        x.extend(None if x is dev else [0], [0])
    dev.check(ref.error)


def test_writing_behind_a_shared_tail_copies_it(nt):
    """A sequence cut back into a page that another shares gets a page of its own when it grows."""
    ref = _cache(6)
    dev = Dev(nt, ref)
    for x in (ref, dev):
        x.extend([0], [64])
        x.fork([0, 0], [1, 2])
        x.free([1, 2], [40, 56])
        x.extend([1, 2, 0], [30, 3, 2])
    dev.check()
    assert ref.table[1, 2] != ref.table[0, 2] and ref.refs[ref.table[0, 2]] == 2


def test_large_plans(nt):
    """More entries than one pass of the planning CTA holds, and pages found across many of its rounds."""
    ref = R.RefCache(1, 1, 64, 16, 9000, 3000, 5)
    dev = Dev(nt, ref)
    rng = np.random.default_rng(7)
    counts = rng.integers(0, 60, 3000)
    seqs = rng.permutation(3000)[:2500]
    free = rng.permutation(3000)[:1700]
    for x in (ref, dev):
        x.extend(list(seqs), list(counts[:2500]))
        x.free(list(free))
    dev.check()
    held = [s for s in range(3000) if ref.len[s]]
    empty = [s for s in range(3000) if not ref.len[s]]
    src = list(rng.choice(held, 1200))
    for x in (ref, dev):
        x.fork(src, empty[:1200])
    dev.check()
    table, refs, live = ref.compact()
    t2, r2 = torch_cuda().empty_like(dev.table), torch_cuda().empty_like(dev.refs)
    assert dev.compact(t2, r2) == live
    dev.check()                                       # the pool has moved, the cache's own table and counts have not
    np.testing.assert_array_equal(t2.cpu().numpy(), table)
    np.testing.assert_array_equal(r2.cpu().numpy(), refs)


def test_copy_refuses_pairs_that_depend_on_their_order(nt):
    ref = _cache(8, n_pages=10)
    dev = Dev(nt, ref)
    for x in (ref, dev):
        x.copy_pages([0, 1, 2], [5, 5, 6])
    dev.check(R.BAD_PAGE)
    for x in (ref, dev):
        x.copy_pages([0, 7, 3, 4], [7, 8, 3, 9])
    dev.check(R.BAD_PAGE)
    for x in (ref, dev):
        x.copy_pages([-1, 10, 1, 1], [1, 2, 10, -1])
    dev.check(R.BAD_PAGE)


def test_compact_of_empty_full_and_single(nt):
    for lens in ([], [96] * 4, [1]):
        ref = _cache(9)
        ref.hold(lens, np.random.default_rng(3))
        dev = Dev(nt, ref)
        table, refs, live = ref.compact()
        assert dev.compact() == live == sum(-(-n // 16) for n in lens)
        ref.table, ref.refs = table, refs
        dev.check()


# ------------------------------------------------------------- used together --

def test_speculative_branches_of_one_prompt(nt):
    """A prompt is stored, branched, each branch grows by its own tokens, the losers are dropped, the cache is compacted:
    at every point the attention of every sequence is that of the rows stored for it."""
    torch = torch_cuda()
    rng = np.random.default_rng(81)
    layers, n_kv, heads, hd = 2, 2, 8, 128
    ref = R.RefCache(layers, n_kv, hd, 32, 40, 6, 8)
    dev = Dev(nt, ref, heads)
    held = {}

    def both(op, *a):
        for x in (ref, dev):
            getattr(x, op)(*a)

    def grow(seqs, counts):
        both("extend", seqs, counts)
        begin = [0] + list(np.cumsum(counts))
        for layer in range(layers):
            x = _rows(rng, begin[-1], n_kv, hd)
            k, v = _layout(torch, x, "side")
            dev.rows(k, v, begin, seqs, layer)
            _store(ref, x, begin, seqs, layer)
            for i, s in enumerate(seqs):
                part = [R.values(*R.quantize(y[begin[i]:begin[i + 1]])) for y in x]
                old = held.get((layer, s))
                held[layer, s] = part if old is None else [np.concatenate(p) for p in zip(old, part)]

    def look(seqs):
        outs = []
        for layer in range(layers):
            q = rng.standard_normal((len(seqs), heads, hd)).astype(np.float32)
            got = dev.attention(torch.from_numpy(q).cuda(), seqs, layer).cpu().numpy().reshape(q.shape)
            for i, s in enumerate(seqs):
                k, v = held[layer, s]
                assert len(k) == ref.len[s]
                b = _bound(ref, s, q[i].astype(np.float64), heads, layer)
                for j in range(heads):
                    w = R.attend(q[i, j].astype(np.float64), k[:, j // 4], v[:, j // 4])
                    assert np.abs(got[i, j] - w).max() <= b[j], (layer, s, j)
            outs.append(got)
        dev.check()
        return outs

    grow([0], [77])
    look([0])
    both("fork", [0, 0, 0], [1, 2, 3])
    for s in (1, 2, 3):
        for layer in range(layers):
            held[layer, s] = held[layer, 0]
    look([0, 1, 2, 3])
    for _ in range(3):
        grow([1, 2, 3], [1, 1, 1])
    grow([1, 3, 0], [30, 2, 20])
    look([3, 2, 1, 0])
    both("free", [2, 1], [79, 0])            # one draft token of 2 is refused, branch 1 is dropped
    for layer in range(layers):
        held[layer, 2] = [x[:79] for x in held[layer, 2]]
    look([2, 0, 3])
    table, refs, live = ref.compact()
    assert dev.compact() == live
    ref.table, ref.refs = table, refs
    look([2, 0, 3])
    grow([2, 3], [40, 1])
    look([3, 2, 0])


def test_a_captured_step_replays(nt):
    """extend, append and attention of a step in one CUDA graph, replayed token by token: the lengths live on the device."""
    torch = torch_cuda()
    rng = np.random.default_rng(91)
    ref = R.RefCache(1, 2, 64, 16, 40, 3, 8)
    dev = Dev(nt, ref, 4)
    x = _rows(rng, 61, 2, 64)
    k, v = _layout(torch, x, "rows")
    dev.extend([0, 2], [30, 1])
    dev.rows(k[:31], v[:31], [0, 30, 31], [0, 2])
    ref.extend([0, 2], [30, 1])
    _store(ref, x[:, :31], [0, 30, 31], [0, 2])
    dev.check()
    kb, vb = torch.zeros(2, 2, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda")
    q, out = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 256, device="cuda")
    seqs, ones = torch.tensor([2, 0], dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")

    def step():
        s = torch.cuda.current_stream()
        nt.nt_kv4_extend(dev.c, 2, seqs.data_ptr(), ones.data_ptr(), dev.ws.data_ptr(), dev.wb, s)
        nt.nt_kv4_append(dev.c, 0, 2, seqs.data_ptr(), None, 2, "f32", kb.data_ptr(), vb.data_ptr(), 128, 64, s)
        nt.nt_attention_kv4(dev.c, 0, 4, 2, seqs.data_ptr(), q.data_ptr(), 256, out.data_ptr(), 256, dev.ws.data_ptr(),
                            dev.wb, s)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for r in range(31, 61, 2):
        kb.copy_(k[r:r + 2])
        vb.copy_(v[r:r + 2])
        qn = rng.standard_normal((2, 4, 64)).astype(np.float32)
        q.copy_(torch.from_numpy(qn))
        graph.replay()
        ref.extend([2, 0], [1, 1])
        _store(ref, x[:, r:r + 2], [0, 1, 2], [2, 0])
        want = _want(ref, [2, 0], qn.astype(np.float64), 4)
        got = out.cpu().numpy().reshape(want.shape)
        for i, s in enumerate((2, 0)):
            assert (np.abs(got[i] - want[i]).max(axis=1) <= _bound(ref, s, qn[i].astype(np.float64), 4)).all()
    dev.check()


# ------------------------------------------------------------ rows at the limits --

@pytest.mark.parametrize("rows", [1, 16, 17, 40])
@pytest.mark.parametrize("padded", [0, 4096, 1 << 24])
def test_rows_of_the_longest_sequence_in_a_padded_batch(nt, rows, padded):
    """Length 2^31 - 256, and more rows in the call than anybody has: the chunks behind the entry's last one, positions
    beyond 2^31, are nobody's.  (Rows of stride 0: all are the same, so the padding needs no memory.)"""
    torch = torch_cuda()
    ref = R.RefCache(1, 1, 64, 256, 3, 3, (1 << 23) - 1, fill=0x5A)
    ref.len[2] = 256 * ref.M
    assert ref.len[2] == (1 << 31) - 256
    ref.table[2, -1], ref.refs[1] = 1, 1
    dev = Dev(nt, ref)
    x = np.repeat(_rows(np.random.default_rng(rows), 1, 1, 64), rows, 1)
    k, v = _layout(torch, x[:, :1], "rows")
    first = 3 if padded else 0
    begin = [first, first + rows]
    nt.nt_kv4_append(dev.c, 0, 1, dev.ints([2]), dev.ints(begin), begin[1] + padded, "f32", k.data_ptr(), v.data_ptr(), 0, 64,
                     dev.stream())
    _store(ref, np.pad(x, [(0, 0), (first, 0), (0, 0), (0, 0)]), begin, [2])
    dev.check()
    if padded <= 4096:
        out = torch.full((2, begin[1] + padded, 1, 64), 5.5, device="cuda")
        dev.rows(out[0], out[1], begin, [2], read=True)
        want = np.full(out.shape, 5.5)
        for side in (0, 1):
            want[side, first:begin[1]] = R.values(*R.quantize(x[side]))
        np.testing.assert_array_equal(out.cpu().numpy().astype(np.float64), want)
        dev.check()


# ------------------------------------------------------------ scores of any size --

@pytest.mark.parametrize("hd,G", [(64, 1), (64, 8), (64, 16), (128, 2), (128, 4), (128, 8), (128, 16)])
@pytest.mark.parametrize("capacity", [704, 16384])
def test_attention_where_scores_are_huge(nt, hd, G, capacity):
    """Scores from 2^24 to 2^104, whose fp32 neighbours are up to 2^80 apart: the largest takes all the weight.

    A score is off by at most (as in _bound) ((hd / 16 + 3) 2u + 2^-22) sum |q K| / sqrt(hd); with two scores further apart
    than twice that and 60 the other weights come to less than 2^-60 of the largest, and the output is the largest's value, whose
    weight enters as hi + lo (2^-22) into products and sums (an addition a step, 2u each, of numbers that are zero but for
    one), and is divided out (2u): 2^-21 of the value.  The inputs are such that this holds for every head."""
    torch = torch_cuda()
    rng = np.random.default_rng([113, hd, G])
    lens = [1, 2, 33, 129, 700]
    powers = [24, 26, 27, 28, 29, 30, 31, 34, 60, 102]
    n_kv, heads = 2, 2 * G
    ref = R.RefCache(1, n_kv, hd, 32, 40, len(lens), capacity // 32)
    ref.randomize(rng)
    ref.hold(lens, rng)
    dev = Dev(nt, ref, heads)
    kv = {(s, g): ref.kv(0, s, g) for s in range(len(lens)) for g in range(n_kv)}
    checked = 0
    for power in powers:
        q = (rng.standard_normal((len(lens), heads, hd)) * 2.0 ** power).astype(np.float32)
        got = dev.attention(torch.from_numpy(q).cuda()).cpu().numpy().reshape(q.shape)
        for s, n in enumerate(lens):
            for j in range(heads):
                k, v = kv[s, j // G]
                q64 = q[s, j].astype(np.float64)
                score, dot = k @ q64 / np.sqrt(hd), np.abs(k) @ np.abs(q64) / np.sqrt(hd)
                order = np.argsort(score)
                apart = score[order[-1]] - score[order[-2]] if n > 1 else np.inf
                if apart <= 2 * ((hd // 16 + 3) * 2 * U + 2.0 ** -22) * dot.max() + 60:
                    continue                       # (two keys that near: which one wins is not defined)
                want = v[order[-1]]
                err = np.abs(got[s, j] - want)
                assert (err <= 2.0 ** -21 * np.abs(want)).all(), (power, n, j, got[s, j][:4], want[:4])
                checked += 1
    assert checked >= 0.99 * len(powers) * len(lens) * heads
    assert int(dev.error.cpu()[0]) == 0


# ------------------------------------------------------------ forks of damaged tables --

@pytest.mark.parametrize("what", ["low", "high", "unheld"])
@pytest.mark.parametrize("where", ["first", "last full", "tail", "far"])
def test_fork_of_a_damaged_source_changes_nothing(nt, what, where):
    """A page of a source that is out of range or that nobody holds, among full pages or the partly filled one: nothing
    changes but the error word, whichever entry of the call it is."""
    rng = np.random.default_rng(17)
    pages = 70 if where == "far" else 5
    for entry in (0, 1, 37, 39):
        ref = R.RefCache(2, 1, 64, 16, 200, 60, 80)
        ref.randomize(rng)
        ref.hold([16 * pages - 7, 33, 40], rng)
        slot = {"first": 0, "last full": pages - 2, "tail": pages - 1, "far": 67}[where]
        if what == "unheld":
            low = ref.free_pages(1)[0]             # the page that the call would take first
            old = ref.table[0, slot]
            ref.refs[old], ref.table[0, slot] = 0, low if low < old else old
        else:
            ref.table[0, slot] = -3 if what == "low" else ref.P
        src = [1, 2] * 20
        src[entry] = 0
        dst = list(range(10, 50))
        dev = Dev(nt, ref)
        dev.fork(src, dst)
        ref.error = R.BAD_PAGE
        dev.check(R.BAD_PAGE)
        # what lies behind the positions that are kept is not looked at
        keep = [16 * slot if s == 0 else int(ref.len[s]) for s in src]
        for x in (ref, dev):
            x.fork(src, dst, keep)
        dev.check(R.BAD_PAGE)
        assert (ref.len[10:50] == keep).all()


# ------------------------------------------------------------ row ranges that do not fit --

BIG = (1 << 31) - 1


@pytest.mark.parametrize("begin,good", [
    ([3, 1, 5], [1]), ([6, 0], []), ([-100, -90], []), ([-100, 2], []), ([-1, 0, 3], [1]), ([100, 110], []),
    ([2, 7], []), ([0, 2, 7], [0]), ([1 << 30, BIG], []), ([-BIG - 1, BIG], []), ([0, 1, BIG, BIG], [0]),
    ([BIG, -BIG], []), ([0, 2, 2, 2, 4, 9], [0, 3])])
def test_row_ranges_outside_the_rows_are_flagged(nt, begin, good):
    """Ranges that run backwards, begin before the rows or end behind them, wholly or partly: a bit in the error word, and
    neither their rows nor the cache are touched; entries beside them that fit are stored and read."""
    torch = torch_cuda()
    rng = np.random.default_rng(12)
    ref = R.RefCache(1, 1, 64, 16, 16, 5, 4, fill=3)
    ref.hold([40, 33, 20, 50, 64], rng)
    dev = Dev(nt, ref)
    x = _rows(rng, 6, 1, 64)
    k, v = _layout(torch, x, "rows")
    dev.rows(k, v, begin)
    for i in good:
        _store(ref, x, [begin[i], begin[i + 1]], [i])
    ref.error = R.BAD_LEN
    dev.check(R.BAD_LEN)
    dev.error.zero_()
    out = torch.full((2, 6, 1, 64), 5.5, device="cuda")
    dev.rows(out[0], out[1], begin, read=True)
    want = np.full(out.shape, 5.5)
    for i in good:
        for side in (0, 1):
            want[side, begin[i]:begin[i + 1]] = R.values(*R.quantize(x[side, begin[i]:begin[i + 1]]))
    np.testing.assert_array_equal(out.cpu().numpy().astype(np.float64), want)
    dev.check(R.BAD_LEN)


def test_empty_row_ranges_are_no_fault(nt):
    """Entries without rows, wherever they stand, have none outside."""
    torch = torch_cuda()
    ref = R.RefCache(1, 1, 64, 16, 8, 3, 2, fill=3)
    ref.hold([20, 3, 0])
    dev = Dev(nt, ref)
    x = _rows(np.random.default_rng(1), 3, 1, 64)
    k, v = _layout(torch, x, "rows")
    for begin in ([0, 0, 0], [3, 3, 3, 3], [9, 9], [-4, -4], [0, 2, 2, 2]):
        dev.rows(k, v, begin)
        _store(ref, x, [0, begin[1] if begin[0] == 0 else 0], [0])
        dev.check()


def test_more_entries_than_rows_without_ranges_are_flagged(nt):
    torch = torch_cuda()
    rng = np.random.default_rng(13)
    ref = R.RefCache(1, 1, 64, 16, 400, 300, 2, fill=3)
    ref.hold([1 + s % 5 for s in range(300)], rng)
    x = _rows(rng, 2, 1, 64)
    for n in (3, 300):
        dev = Dev(nt, ref)
        k, v = _layout(torch, x, "rows")
        nt.nt_kv4_append(dev.c, 0, n, None, None, 2, "f32", k.data_ptr(), v.data_ptr(), 64, 64, dev.stream())
        _store(ref, x, [0, 1, 2], [0, 1])
        ref.error = R.BAD_LEN
        dev.check(R.BAD_LEN)
        dev.error.zero_()
        out = torch.full((2, 2, 1, 64), 5.5, device="cuda")
        nt.nt_kv4_read(dev.c, 0, n, None, None, 2, "f32", out[0].data_ptr(), out[1].data_ptr(), 64, 64, dev.stream())
        want = np.stack([R.values(*R.quantize(y)) for y in x])
        np.testing.assert_array_equal(out.cpu().numpy().astype(np.float64), want)
        dev.check(R.BAD_LEN)


def test_compact_copies_entries_that_name_no_page(nt):
    """Table entries out of range, below as well as above, come out as they are and are flagged; -1 is nothing of note."""
    ref = _cache(10)
    ref.hold([96, 20, 50], np.random.default_rng(4))
    dev = Dev(nt, ref)
    for x in (ref, dev):
        x.free([1])                                    # holes
    odd = {(4, 0): -2, (4, 1): -3, (5, 2): -(1 << 31), (6, 5): ref.P, (7, 5): (1 << 31) - 1}
    kept = ref.table.copy()
    table, refs, live = ref.compact()
    ref.table, ref.refs = table, refs
    for at, p in odd.items():
        assert kept[at] == -1
        ref.table[at] = p
        dev.table[at] = p
    assert dev.compact() == live
    ref.error = R.BAD_PAGE
    dev.check(R.BAD_PAGE)


def test_compact_drops_entries_that_name_free_pages(nt):
    """Below the number of pages in use as well as behind it: an entry of a page that nobody holds becomes -1."""
    ref = _cache(11)
    ref.hold([96, 20, 50], np.random.default_rng(5))
    ref.free([1])
    used = int((ref.refs > 0).sum())
    free = ref.free_pages(ref.P)
    assert free[0] < used <= free[-1]
    dev = Dev(nt, ref)
    dev.table[5, 0], dev.table[5, 1] = free[0], free[-1]
    table, refs, live = ref.compact()
    ref.table, ref.refs = table, refs
    assert dev.compact() == live == used
    ref.error = R.BAD_PAGE
    dev.check(R.BAD_PAGE)


# ------------------------------------------------------------ long sequences, as a whole --

def _rel_limit(k, q, hd):
    """What |got - want| / |want| over a head's outputs may be for values of mean zero that the weights' errors know nothing
    of.  With out = sum w V, relative errors e of the weights move it by sum w e (V - out), in the mean square by the root
    mean square of e times |out|.  e is the scores' error (see _bound) and 2^-22 each of the exponential and the split.  A sum
    is held over at most 64 additions in the matrix products (truncated, 2^-23 of the sum so far, which is half the final one
    in the mean) and then goes through at most 67 that round to nearest, each its own way: sqrt(67) u."""
    dot = np.abs(k) @ np.abs(q) / np.sqrt(hd)
    ds = ((hd // 16 + 3) * 2 * U + 2.0 ** -22) * dot + 6 * U * np.abs(k @ q / np.sqrt(hd))
    return np.sqrt((ds * ds).mean()) + 2 * 2.0 ** -22 + 64 / 2 * 2.0 ** -23 + np.sqrt(67) * U


def _balanced(ref, rng):
    """Random codes 1..15, the values' mean zero."""
    ref.randomize(rng)
    codes = ref.pool.reshape(ref.L, ref.P, ref.n_kv, ref.pl // 16, -1)[..., :16 * ref.hd]
    codes[:] = rng.integers(1, 16, codes.shape, np.uint8) | rng.integers(1, 16, codes.shape, np.uint8) << 4


# (n_kv, G, hd, page_len, capacity, lengths)
LONG = [
    (1, 8, 128, 64, 131136, [131077]),        # one item across every CTA
    (1, 16, 128, 64, 131136, [131077]),
    (1, 4, 128, 64, 131136, [131077]),
    (1, 8, 64, 16, 131136, [131077]),
    (4, 8, 128, 48, 131136, [131077]),
    (4, 4, 128, 256, 131328, [131077]),
    (2, 1, 64, 128, 131200, [131077, 70000, 129]),
    (2, 16, 64, 64, 131136, [131077, 40001]),
    (3, 8, 128, 64, 33024, [33001, 2047, 20000, 1]),
    (8, 8, 128, 64, 4224, [4161]),            # a cluster per item
    (8, 4, 128, 32, 9024, [9001, 5000, 4097]),
]


@pytest.mark.parametrize("n_kv,G,hd,page_len,capacity,lens", LONG)
def test_attention_of_long_sequences_misses_nothing(nt, n_kv, G, hd, page_len, capacity, lens):
    """Weights of the same size, so that every position counts: a position left out anywhere, or the lower terms of queries or
    weights, would show at many times what is allowed."""
    torch = torch_cuda()
    rng = np.random.default_rng([127, n_kv, G, hd])
    pages = sum(-(-n // page_len) for n in lens)
    ref = R.RefCache(1, n_kv, hd, page_len, pages + 2, len(lens), capacity // page_len)
    _balanced(ref, rng)
    ref.hold(lens, rng)
    heads = n_kv * G
    dev = Dev(nt, ref, heads)
    q = (rng.standard_normal((len(lens), heads, hd)) * 0.3).astype(np.float32)
    got = dev.attention(torch.from_numpy(q).cuda()).cpu().numpy().reshape(q.shape)
    assert int(dev.error.cpu()[0]) == 0
    worst = 0.0
    for s, n in enumerate(lens):
        for g in range(n_kv):
            k, v = ref.kv(0, s, g)
            for j in range(g * G, (g + 1) * G):
                qj = q[s, j].astype(np.float64)
                want, limit = R.attend(qj, k, v), _rel_limit(k, qj, hd)
                size = np.linalg.norm(want)
                rel = np.linalg.norm(got[s, j] - want) / size
                assert rel <= limit, (n, j, rel, limit)
                worst = max(worst, rel)
                if j % G == 0 and n > 2000:
                    for lost in (0, n // 3, n - 1):
                        less = R.attend(qj, np.delete(k, lost, 0), np.delete(v, lost, 0)) if n < 20000 else (
                            want - (v[lost] - want) * np.exp(k[lost] @ qj / np.sqrt(hd)) / np.exp(k @ qj / np.sqrt(hd)).sum())
                        assert np.linalg.norm(less - want) > 20 * limit * size, (n, lost)
                    coarse = qj.astype(np.float16).astype(np.float64)
                    assert np.linalg.norm(R.attend(coarse, k, v) - want) > 2 * limit * size
                    p = np.exp(k @ qj / np.sqrt(hd) - 1)
                    assert np.linalg.norm(p.astype(np.float16).astype(np.float64) @ v / p.sum() - want) > 2 * limit * size
    print(f"kv {n_kv} G {G} hd {hd} page {page_len} lengths {lens}: rel L2 {worst:.2e}, allowed {limit:.2e}")


@pytest.mark.parametrize("n_kv,G,hd,page_len,capacity,lens", [x for x in LONG if x[0] < 8])
def test_attention_of_long_sequences_with_a_few_positions_that_count(nt, n_kv, G, hd, page_len, capacity, lens):
    """Every 61st position of the last two thirds, and the last one, has the same key, whose score is 30 and more above all
    others': the output is the mean of those positions' values.  References move in the middle of the work, and the first
    third's partial results vanish in the merges.  The others' weights are below 2^-40 of the largest, all 131077 together
    below 2^-22 of a position that counts.  Equal keys go through the same products, so of the scores' error only the roundings
    on the way to the exponent are left (6u of the score), then 2^-22 of the exponential, the split and the others, and the sums'
    as in _rel_limit."""
    torch = torch_cuda()
    rng = np.random.default_rng([131, n_kv, G, hd])
    pages = sum(-(-n // page_len) for n in lens)
    ref = R.RefCache(1, n_kv, hd, page_len, pages + 2, len(lens), capacity // page_len)
    _balanced(ref, rng)
    ref.hold(lens, rng)
    heads = n_kv * G
    u = rng.choice([-1.0, 1.0], (n_kv, hd))
    e, j = np.arange(hd), np.arange(ref.ng)
    quarter = np.array([0.25], np.float16).view(np.uint8)
    places = []
    for s, n in enumerate(lens):
        t = np.unique(np.append(np.arange(n - 1 - n // 3 * 2, n, 61), n - 1))
        t = t[t >= 0]
        places.append(t)
        page, at = ref.table[s, t // page_len][:, None], (t % page_len)[:, None]
        for g in range(n_kv):
            for half in (0, 1):                           # the low and the high codes of a byte: +-7 times 0.25
                b, sh = ref._k_code(g, at, e[half::2])
                code = (8 + 7 * u[g, half::2]).astype(np.uint8)
                old = ref.pool[0][page, b]
                ref.pool[0][page, b] = (old & (0xF0 if half == 0 else 0x0F)) | (code << (4 * half))
            b = ref._k_scale(g, at, j)
            ref.pool[0][page, b], ref.pool[0][page, b + 1] = quarter
    q = (u.repeat(G, 0) * rng.uniform(3.6, 4.0, (len(lens), heads, 1)) * np.sqrt(128 / hd)).astype(np.float32)
    dev = Dev(nt, ref, heads)
    got = dev.attention(torch.from_numpy(q).cuda()).cpu().numpy().reshape(q.shape)
    assert int(dev.error.cpu()[0]) == 0
    for s, n in enumerate(lens):
        for g in range(n_kv):
            k, v = ref.kv(0, s, g)
            for h in range(g * G, (g + 1) * G):
                qh = q[s, h].astype(np.float64)
                score, t = k @ qh / np.sqrt(hd), places[s]
                rest = np.delete(score, t)
                assert np.ptp(score[t]) < 1e-9 and (not len(rest) or score[t[0]] - rest.max() > 30)
                want, limit = v[t].mean(0), 6 * U * score[t[0]] + 4 * 2.0 ** -22 + 64 / 2 * 2.0 ** -23 + np.sqrt(67) * U
                assert np.linalg.norm(got[s, h] - want) <= limit * np.linalg.norm(want), (n, h)
                if len(t) > 1:
                    less = v[np.delete(t, len(t) // 2)].mean(0)
                    assert np.linalg.norm(less - want) > 100 * limit * np.linalg.norm(want)


# ------------------------------------------------------------ lists and lengths at the limits --

@pytest.mark.parametrize("bad", [None, 1, 1500, 2499])
def test_row_ranges_of_many_entries(nt, bad):
    """More entries than one CTA looks over; one of them, early or late, runs backwards."""
    torch = torch_cuda()
    rng = np.random.default_rng(19)
    ref = R.RefCache(1, 1, 64, 16, 8000, 2500, 3, fill=3)
    ref.hold(rng.integers(16, 48, 2500), rng)
    seqs = rng.permutation(2500)
    counts = rng.integers(0, 5, 2500)
    begin = [2] + [int(b) for b in 2 + np.cumsum(counts)]
    rows = begin[-1] + 3
    x = _rows(rng, rows, 1, 64)
    k, v = _layout(torch, x, "rows")
    dev = Dev(nt, ref)
    want = np.full((2, rows, 1, 64), 5.5)
    for i, s in enumerate(seqs):
        _store(ref, x[:, begin[i]:begin[i + 1]], [0, int(counts[i])], [s])
        for side in (0, 1):
            want[side, begin[i]:begin[i + 1]] = R.values(*R.quantize(x[side, begin[i]:begin[i + 1]]))
    near = []
    if bad is not None:                       # entry `bad` ends a row before it begins; the next one has some of its rows
        near = [seqs[i] for i in (bad, bad + 1) if i < 2500]
        want[:, begin[bad] - 1:begin[min(bad + 2, 2500)]] = np.nan
        begin[bad + 1] = begin[bad] - 1
    dev.rows(k, v, begin, seqs)
    out = torch.full((2, rows, 1, 64), 5.5, device="cuda")
    dev.rows(out[0], out[1], begin, seqs, read=True)
    torch.cuda.synchronize()
    assert int(dev.error.cpu()[0]) == (0 if bad is None else R.BAD_LEN)
    pool, got = dev.pool.cpu().numpy(), out.cpu().numpy().astype(np.float64)
    sure = np.ones(ref.P, bool)
    sure[ref.table[near].reshape(-1)] = False
    np.testing.assert_array_equal(pool[:, sure], ref.pool[:, sure])
    np.testing.assert_array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_fork_of_many_with_one_damaged_source(nt):
    rng = np.random.default_rng(23)
    ref = R.RefCache(1, 1, 64, 16, 9000, 4000, 9)
    ref.randomize(rng)
    ref.hold(rng.integers(1, 140, 900), rng)
    src, dst = [int(s) for s in rng.integers(0, 899, 2600)], list(range(1000, 3600))
    for i in (0, 1023, 1024, 2599):
        dev = Dev(nt, ref)
        odd = list(src)
        odd[i] = 899
        last = (int(ref.len[899]) - 1) // 16
        dev.table[899, last] = -2
        dev.fork(odd, dst)
        torch_cuda().cuda.synchronize()
        assert int(dev.error.cpu()[0]) == R.BAD_PAGE
        assert not dev.len[1000:].any() and (dev.table[1000:] == -1).all()
        np.testing.assert_array_equal(dev.refs.cpu().numpy(), ref.refs)
    dev = Dev(nt, ref)
    for x in (ref, dev):
        x.fork(src, dst)
    dev.check()


@pytest.mark.parametrize("hd,G", [(64, 8), (128, 4), (128, 16)])
def test_huge_scores_of_many_short_sequences(nt, hd, G):
    """The form of whole items for the CTAs; limits as where scores are huge."""
    torch = torch_cuda()
    rng = np.random.default_rng([137, hd, G])
    lens = [1, 15, 100, 300]
    ref = R.RefCache(1, 2, hd, 16, 40, 4, 19)
    ref.randomize(rng)
    ref.hold(lens, rng)
    dev = Dev(nt, ref, 2 * G)
    seqs = np.arange(200) % 4
    checked = 0
    for power in (20, 27, 30, 80):
        q = (rng.standard_normal((4, 2 * G, hd)) * 2.0 ** power).astype(np.float32)
        got = dev.attention(torch.from_numpy(q[seqs]).cuda(), seqs).cpu().numpy().reshape(200, 2 * G, hd)
        for s in range(4):
            for j in range(2 * G):
                k, v = ref.kv(0, s, j // G)
                q64 = q[s, j].astype(np.float64)
                score, dot = k @ q64 / np.sqrt(hd), np.abs(k) @ np.abs(q64) / np.sqrt(hd)
                order = np.argsort(score)
                if lens[s] > 1 and score[order[-1]] - score[order[-2]] <= 2 * (
                        (hd // 16 + 3) * 2 * U + 2.0 ** -22) * dot.max() + 60:
                    continue
                want = v[order[-1]]
                assert (np.abs(got[seqs == s, j] - want) <= 2.0 ** -21 * np.abs(want)).all(), (power, s, j)
                checked += 1
    assert checked >= 0.98 * 4 * 4 * 2 * G


@pytest.mark.parametrize("hd,G", [(64, 1), (128, 8)])
def test_attention_of_the_longest_sequence(nt, hd, G):
    """2^31 - 256 positions, the pages of all columns of the table the same one: what attention over that page gives.  Then
    a page of its own in the last column, whose last key outweighs all others.  Seventeen entries, so that the call is cut
    into two launches.

    A thread adds up the weights of all its steps (a pair of chunks, or a tile of 128) one after the other in fp32, of
    which there are at most 2^31 / 32 / (152 * 12) = 36793; the outputs take fewer."""
    torch = torch_cuda()
    rng = np.random.default_rng([139, hd, G])
    ref = R.RefCache(1, 1, hd, 256, 2, 1, 1)
    ref.randomize(rng)
    ref.table[0, 0], ref.len[0] = 0, 256
    columns = (1 << 23) - 1
    long = R.RefCache(1, 1, hd, 256, 2, 1, 1)
    long.shape.update(max_pages=columns)
    long.pool[:], long.len[0], long.refs[0] = ref.pool, 256 * columns, 1
    dev = Dev(nt, long, G)
    dev.table = torch.zeros((1, columns), dtype=torch.int32, device="cuda")
    dev.c.table = dev.table.data_ptr()
    q = rng.standard_normal((1, G, hd)).astype(np.float32)
    got = dev.attention(torch.from_numpy(q).cuda(), [0]).cpu().numpy().reshape(G, hd)
    q64 = q[0].astype(np.float64)
    want = _want(ref, [0], q64[None], G)[0]
    vm = np.abs(ref.kv(0, 0, 0)[1]).max()
    bound = _bound(ref, 0, q64, G) + 2 * vm * 36793 * U + 2 * vm * 36793 * 2.0 ** -31
    assert (np.abs(got - want).max(axis=1) <= bound).all()
    # the last key: the sign of the first head's query, for all heads; half of them
    ref.table[0, 0] = 1
    sign = np.where(rng.integers(0, 2, hd) > 0, 1.0, -1.0)
    ref.put(0, 1, 0, 255, (sign * 700).astype(np.float32), rng.standard_normal(hd).astype(np.float32))
    dev.pool.copy_(torch.from_numpy(ref.pool))
    dev.table[0, -1] = 1
    q = (np.broadcast_to(sign, (17, G, hd)) * rng.uniform(1, 2, (17, G, 1))).astype(np.float32)
    got = dev.attention(torch.from_numpy(q).cuda(), [0] * 17).cpu().numpy().reshape(17, G, hd)
    v = ref.kv(0, 0, 0)[1][255]
    assert (np.abs(got - v) <= 2.0 ** -21 * np.abs(v)).all()
    assert int(dev.error.cpu()[0]) == 0


FIRST_CALLS = """
import sys
sys.path[:0] = ["tests", "."]
import numpy as np, torch
import kv4_ref as R
from test_gpu_kv4 import Dev, _rows, _layout
from quantized_decode_dequant_gb300 import nt
torch.zeros(1, device="cuda")
rng = np.random.default_rng(5)

def make():
    ref = R.RefCache(2, 2, 128, 32, 80, 8, 1024)
    ref.randomize(np.random.default_rng(6))
    ref.hold([300, 65, 0, 40], np.random.default_rng(7))
    return ref

x = _rows(rng, 2, 2, 128)
q = torch.from_numpy(rng.standard_normal((2, 16, 128)).astype(np.float32)).cuda()
k, v = _layout(torch, x, "rows")

def calls(dev, out, back):
    dev.fork(dev.l_src, dev.l_dst)
    dev.extend(dev.l_dst, dev.l_one)
    for layer in (0, 1):
        dev.rows(k, v, None, dev.l_dst, layer)
        dev.rows(back[layer][0], back[layer][1], None, dev.l_dst, layer, read=True)
        dev.attention(q, dev.l_dst, layer, out=out[layer])
    dev.free(dev.l_drop)
    dev.copy_pages(dev.l_from, dev.l_to)

class Fixed(Dev):
    def ints(self, x):          # lists made before the capture
        return None if x is None else x.data_ptr()

    def compact_only(self, live):
        self.nt.nt_kv4_compact(self.c, self.table.data_ptr(), self.refs.data_ptr(), live.data_ptr(), self.ws.data_ptr(),
                               self.wb, self.stream())

def fresh():
    dev = Fixed(nt, make(), 16)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    dev.l_src, dev.l_dst, dev.l_one, dev.l_drop = i32(0, 1), i32(4, 5), i32(1, 1), i32(1)
    dev.l_from, dev.l_to, dev.live = i32(3, 4), i32(78, 79), i32(0)
    return dev, torch.zeros(2, 2, 2048, device="cuda"), torch.zeros(2, 2, 2, 2, 128, device="cuda")

dev, out, back = fresh()
side = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):        # every operator for the first time in this process
    calls(dev, out, back)
    dev.compact_only(dev.live)
graph.replay()
torch.cuda.synchronize()
dev2, out2, back2 = fresh()
calls(dev2, out2, back2)
dev2.compact_only(dev2.live)
torch.cuda.synchronize()
for a, b in ((out, out2), (back, back2), (dev.pool, dev2.pool), (dev.table, dev2.table), (dev.len, dev2.len),
             (dev.refs, dev2.refs), (dev.error, dev2.error), (dev.live, dev2.live)):
    assert torch.equal(a, b)
assert int(dev.error) == 0 and torch.isfinite(out).all() and out.any()
print("captured")
"""


def test_first_calls_of_a_process_inside_a_capture(nt):
    """What a kernel is set up with at its first launch does not disturb a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
