"""GPU: the paged 8-bit K/V cache -- rows in and out with the rotation, page operators, selection and attention, and a run of
them together -- against the plain model of kv8_ref.py (bytes, tables and choices equal; attention within a bound derived from
its arithmetic)."""
import numpy as np
import pytest

import kv8_ref as R
from gpu_util import torch_cuda, ensure_built

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def nt():
    torch_cuda()
    ensure_built()
    from quantized_decode_dequant_gb300 import nt as _nt
    return _nt


def freqs(hd, theta=500000.0):
    return [theta ** (-2.0 * i / hd) for i in range(hd // 2)]


class Dev:
    """A RefCache's buffers on the device, and the library's calls on them."""

    def __init__(self, nt, ref, n_heads=None, n=None):
        import torch
        self.nt, self.torch, self.ref = nt, torch, ref
        up = lambda a: torch.from_numpy(a.copy()).cuda()   # noqa: E731
        self.pool, self.table, self.len, self.refs = up(ref.pool), up(ref.table), up(ref.len), up(ref.refs)
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.c = nt.make_kv8_cache(**ref.shape, pool=self.pool.data_ptr(), table=self.table.data_ptr(),
                                   len=self.len.data_ptr(), refs=self.refs.data_ptr(), error=self.error.data_ptr())
        self.heads = n_heads or ref.n_kv
        self.wb = nt.nt_kv8_workspace_bytes(self.c, self.heads, n or max(ref.S, 8))
        self.ws = torch.full((self.wb,), 0x7F, dtype=torch.uint8, device="cuda")
        self.alive = []

    def ints(self, x):
        if x is None:
            return None
        t = self.torch.tensor(np.asarray(x).tolist(), dtype=self.torch.int32, device="cuda")
        self.alive.append(t)
        return t.data_ptr()

    def stream(self):
        return self.torch.cuda.current_stream()

    def extend(self, seqs, counts):
        self.nt.nt_kv8_extend(self.c, len(counts), self.ints(seqs), self.ints(counts), self.ws.data_ptr(), self.wb,
                              self.stream())

    def fork(self, src, dst, keep=None):
        self.nt.nt_kv8_fork(self.c, len(src), self.ints(src), self.ints(dst), self.ints(keep), self.ws.data_ptr(), self.wb,
                            self.stream())

    def free(self, seqs, keep=None):
        self.nt.nt_kv8_free(self.c, len(seqs), self.ints(seqs), self.ints(keep), self.stream())

    def append(self, k, v, begin, seqs=None, layer=0, freq=None, q=None, q_out=None):
        """torch k, v [rows, kv, hd] of any strides, q [rows, heads, hd]; begin None: a row each."""
        n = (len(begin) - 1) if begin is not None else (len(seqs) if seqs is not None else k.shape[0])
        assert k.stride() == v.stride()
        ptr = lambda t: None if t is None else t.data_ptr()   # noqa: E731
        self.nt.nt_kv8_append(self.c, layer, n, self.ints(seqs), self.ints(begin), k.shape[0],
                              "f16" if k.dtype == self.torch.float16 else "f32", k.data_ptr(), v.data_ptr(), k.stride(0),
                              k.stride(1), freq, 0 if q is None else q.shape[1], ptr(q), 0 if q is None else q.stride(0),
                              ptr(q_out), 0 if q_out is None else q_out.stride(0), self.stream())

    def read(self, k, v, begin, seqs=None, layer=0):
        n = (len(begin) - 1) if begin is not None else (len(seqs) if seqs is not None else k.shape[0])
        self.nt.nt_kv8_read(self.c, layer, n, self.ints(seqs), self.ints(begin), k.shape[0],
                            "f16" if k.dtype == self.torch.float16 else "f32", k.data_ptr(), v.data_ptr(), k.stride(0),
                            k.stride(1), self.stream())

    def select(self, q, top, first=0, last=0, seqs=None, ctx=None, layer=0):
        out = self.torch.full((q.shape[0], self.ref.n_kv, top), -7, dtype=self.torch.int32, device="cuda")
        self.nt.nt_kv8_select(self.c, layer, self.heads, q.shape[0], self.ints(seqs), self.ints(ctx), q.data_ptr(), q.stride(0),
                              top, first, last, out.data_ptr(), self.ws.data_ptr(), self.wb, self.stream())
        return out

    def attention(self, q, seqs=None, ctx=None, pages=None, layer=0, out=None, ws=None, stream=None):
        """q [n, heads, hd] (any row stride); pages: a torch tensor [n, kv, top]."""
        torch = self.torch
        out = torch.full((q.shape[0], self.heads, self.ref.hd), float("inf"), device="cuda") if out is None else out
        self.nt.nt_attention_kv8(self.c, layer, self.heads, q.shape[0], self.ints(seqs), self.ints(ctx),
                                 0 if pages is None else pages.shape[2], None if pages is None else pages.data_ptr(),
                                 q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0),
                                 (self.ws if ws is None else ws).data_ptr(), self.wb, stream or self.stream())
        return out

    def check(self, error=0):
        """The device's state is the model's."""
        self.torch.cuda.synchronize()
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.ref.table)
        np.testing.assert_array_equal(self.len.cpu().numpy(), self.ref.len)
        np.testing.assert_array_equal(self.refs.cpu().numpy(), self.ref.refs)
        got, want = self.pool.cpu().numpy(), self.ref.pool
        codes = self.ref.n_kv * 2 * self.ref.pl * self.ref.hd
        a, b = got[..., :codes], want[..., :codes]
        assert ((a == b) | ((a & 127 == 127) & (b & 127 == 127))).all()      # (a NaN has two codes)
        np.testing.assert_array_equal(got[..., codes:], want[..., codes:])
        assert int(self.error.cpu()[0]) == error


def rows(rng, n, kv, hd):
    x = rng.standard_normal((2, n, kv, hd)) * np.exp(rng.standard_normal((2, n, kv, 1)))
    return x.astype(np.float32)


def layout(torch, x, how, half=False):
    """[rows, kv, hd] k and v of x [2, rows, kv, hd] as a user may hold them."""
    t = torch.from_numpy(x).cuda()
    t = t.half() if half else t
    if how == "rows":            # a projection's rows
        return t[0], t[1]
    if how == "cache":           # [kv][position][dim]
        t = t.transpose(1, 2).contiguous().transpose(1, 2)
        return t[0], t[1]
    t = t.permute(1, 0, 2, 3).contiguous()   # K and V next to each other in every row
    return t[:, 0], t[:, 1]


def store(ref, x, begin, seqs, layer=0, freq=None):
    for i, s in enumerate(seqs):
        if begin[i + 1] > begin[i]:
            ref.append(layer, s, x[0, begin[i]:begin[i + 1]], x[1, begin[i]:begin[i + 1]], freq)


# -------------------------------------------------------------- append, read --

@pytest.mark.parametrize("how", ["rows", "cache", "both"])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("hd,kv,page_len", [(64, 1, 16), (64, 3, 64), (128, 2, 32), (128, 5, 128)])
def test_append_and_read(nt, hd, kv, page_len, half, how):
    import torch
    rng = np.random.default_rng(hd + kv)
    kept, new = [0, page_len - 1, 5, page_len, 3 * page_len + 7, 40], [2 * page_len + 3, 2, 1, page_len, 0, 17]
    n = sum(-(-(a + b) // page_len) for a, b in zip(kept, new))
    ref = R.RefCache(2, kv, hd, page_len, n + 2, 6, 8, fill=0xFF)
    ref.randomize(rng)
    ref.hold([a + b for a, b in zip(kept, new)], rng)
    begin = np.concatenate([[0], np.cumsum(new)])
    x = rows(rng, int(begin[-1]), kv, hd)
    if half:
        x = x.astype(np.float16).astype(np.float32)
    dev, freq = Dev(nt, ref), freqs(hd)
    k, v = layout(torch, x, how, half)
    store(ref, x, begin, range(6), layer=1, freq=freq)
    dev.append(k, v, begin, layer=1, freq=freq)
    dev.check()
    out = torch.full((2,) + tuple(k.shape), 77.0, device="cuda", dtype=k.dtype)
    dev.read(out[0], out[1], begin, layer=1)
    dev.check()
    for i in range(6):
        for g in range(kv):
            for got, want in zip(out, ref.kv(1, i, g)):
                want = want[len(want) - new[i]:].astype(np.float16 if half else np.float32)
                np.testing.assert_array_equal(got[begin[i]:begin[i + 1], g].cpu().numpy(), want)


def test_rows_one_at_a_time_with_growing_values(nt):
    """Token after token with values that grow: every page's exponent rises on the way and its codes are rounded again."""
    import torch
    rng = np.random.default_rng(3)
    ref = R.RefCache(1, 2, 64, 32, 8, 2, 4, fill=0xA5)
    ref.hold([0, 0])
    dev = Dev(nt, ref)
    for i in range(70):
        x = (rng.standard_normal((2, 2, 2, 64)) * 2.0 ** (i / 4 - 8)).astype(np.float32)
        ref.extend([0, 1], [1, 1])
        dev.extend([0, 1], [1, 1])
        store(ref, x, [0, 1, 2], [0, 1], freq=freqs(64))
        k, v = layout(torch, x, "rows")
        dev.append(k, v, None, freq=freqs(64))
    dev.check()


def test_a_page_begun_anew_forgets_its_exponent_and_bounds(nt):
    import torch
    rng = np.random.default_rng(4)
    ref = R.RefCache(1, 1, 64, 16, 4, 1, 4)
    ref.randomize(rng)
    ref.hold([20])
    dev = Dev(nt, ref)
    big, small = rows(rng, 20, 1, 64) * 1e6, rows(rng, 20, 1, 64) * 1e-6
    for x in (big, small):
        store(ref, x, [0, 20], [0])
        dev.append(*layout(torch, x, "rows"), [0, 20])
        dev.check()
    # back to the middle of a page: the scale stays, the rows behind are written anew
    ref.free([0], [10])
    dev.free([0], [10])
    ref.extend([0], [3])
    dev.extend([0], [3])
    x = rows(rng, 3, 1, 64)
    store(ref, x, [0, 3], [0])
    dev.append(*layout(torch, x, "rows"), [0, 3])
    dev.check()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("hd,kv,page_len,S", [(64, 11, 32, 2), (128, 9, 64, 2), (128, 3, 128, 2), (64, 1, 16, 2), (64, 11, 32, 40), (128, 9, 64, 40),
                                              (128, 3, 128, 60), (64, 20, 16, 50)])
def test_keys_between_two_codes(nt, hd, kv, page_len, S, half):
    """Keys half way between codes where the rotation leaves them (position 0), or far fewer bits long than their pair's other
    half, zeros of both signs: more of them than are put off, in pages begun, gone on with and ended in the middle; with few
    sequences a head in each CTA, with many several."""
    import torch
    rng = np.random.default_rng(40)
    n = page_len + 5
    ref = R.RefCache(2, kv, hd, page_len, 2 * S, S, 2)
    dev, freq = Dev(nt, ref), freqs(hd)
    half_way = (1 + (2 * rng.integers(0, 8, (2, S * n, kv, hd)) + 1) / 16) * 2.0 ** rng.integers(-6, 5, (2, S * n, kv, hd))
    x = (half_way * rng.choice([-1, 1], half_way.shape)).astype(np.float32)
    x[:, :, 0, 1::2] *= np.float32(2.0 ** -9)                  # (cos of a small angle is 1, and the sum nearly half way)
    x[0, :, kv // 2] = rng.choice([0.0, -0.0], (S * n, hd))
    x[0, rng.integers(0, S * n, n)] = -0.0
    k, v = layout(torch, x, "rows", half)
    for first, last in ((0, 1), (1, page_len - 3), (page_len - 3, n)):
        r = last - first
        dev.extend(range(S), [r] * S)
        ref.extend(list(range(S)), [r] * S)
        rows_of = (np.arange(S)[:, None] * n + np.arange(first, last)).reshape(-1)
        begin = [r * i for i in range(S + 1)]
        dev.append(k[rows_of].contiguous(), v[rows_of].contiguous(), begin, layer=1, freq=freq)
        store(ref, x[:, rows_of], begin, range(S), layer=1, freq=freq)
        dev.check()


@pytest.mark.parametrize("rotated", [False, True])
def test_values_that_cannot_be_held(nt, rotated):
    import torch
    rng = np.random.default_rng(5)
    ref = R.RefCache(1, 1, 64, 16, 4, 1, 4)
    ref.hold([40])
    x = rows(rng, 40, 1, 64)
    x[:, 3, 0, 7], x[:, 4, 0, 9], x[:, 20, 0, 1], x[:, 21, 0, 2] = np.nan, np.inf, -np.inf, 3e38
    x[:, 16:20] = 0
    x[:, 22], x[:, 23, 0, 5], x[:, 33] = 1e-42, R.MOST, 0
    x[:, 34:] *= 1e-33
    dev = Dev(nt, ref)
    freq = freqs(64) if rotated else None
    store(ref, x, [0, 40], [0], freq=freq)
    dev.append(*layout(torch, x, "rows"), [0, 40], freq=freq)
    dev.check()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("hd,heads", [(64, 1), (64, 7), (128, 5), (128, 64)])
def test_queries_are_rotated_beside_the_keys(nt, hd, heads, half):
    import torch
    rng = np.random.default_rng(6)
    lens, new = [5, 70, 300], [5, 1, 33]
    ref = R.RefCache(1, 1, hd, 64, 10, 3, 5)
    ref.hold(lens)
    begin = [0, 5, 6, 39]
    x, q = rows(rng, 39, 1, hd), rng.standard_normal((39, heads, hd)).astype(np.float32)
    if half:
        x, q = x.astype(np.float16).astype(np.float32), q.astype(np.float16).astype(np.float32)
    dev, freq = Dev(nt, ref), freqs(hd)
    store(ref, x, begin, range(3), freq=freq)
    pos = np.concatenate([np.arange(n - r, n) for n, r in zip(lens, new)])
    want = R.rotate(q, pos, freq)
    big = np.abs(q).reshape(39, heads, -1, 2).sum(-1).repeat(2, -1)
    k, v = layout(torch, x, "rows", half)
    base = torch.zeros(39, heads * hd + 8, device="cuda", dtype=k.dtype)
    tq = base[:, :heads * hd].view(39, heads, hd) if heads * hd % 8 else base[:, :heads * hd].unflatten(1, (heads, hd))
    tq.copy_(torch.from_numpy(q))
    out = torch.full((39, heads * hd + 4), 9.0, device="cuda")
    dev.append(k, v, begin, freq=freq, q=tq, q_out=out)
    dev.check()
    got = out.cpu().numpy()
    assert (got[:, heads * hd:] == 9).all()
    # one rounding of fp32 on either side, and 2^-45 of the products
    assert (np.abs(got[:, :heads * hd].reshape(q.shape) - want.astype(np.float64)) <= 2 * U * np.abs(want) + 2.0 ** -40 * big).all()
    if not half:   # in place
        dev.append(k, v, begin, freq=freq, q=tq, q_out=tq)
        np.testing.assert_array_equal(tq.cpu().numpy(), got[:, :heads * hd].reshape(q.shape))


@pytest.mark.parametrize("hd,heads,rows_each", [(64, 17, 1300), (128, 16, 1250), (128, 9, 100), (64, 24, 60)])
def test_queries_of_many_rows(nt, hd, heads, rows_each):
    """Rows enough for a warp to take 8 or 16 heads, the last ones not full."""
    import torch
    rng = np.random.default_rng(39)
    ref = R.RefCache(1, 1, hd, 128, 24, 2, 12)
    ref.hold([rows_each, rows_each + 7])
    dev, freq, n = Dev(nt, ref), freqs(hd), 2 * rows_each
    k = torch.zeros(n, 1, hd, device="cuda")
    q = torch.from_numpy(rng.standard_normal((n, heads, hd)).astype(np.float32)).cuda()
    out = torch.full((n + 1, heads * hd), 9.0, device="cuda")
    dev.append(k, k, [0, rows_each, n], freq=freq, q=q, q_out=out[:n])
    pos = np.concatenate([np.arange(rows_each), np.arange(7, rows_each + 7)])
    want = R.rotate(q.cpu().numpy(), pos, freq)
    big = np.abs(q.cpu().numpy()).reshape(n, heads, -1, 2).sum(-1).repeat(2, -1)
    # one rounding of fp32 on either side, and 2^-45 of the products
    assert (np.abs(out[:n].cpu().numpy().reshape(want.shape) - want.astype(np.float64)) <= 2 * U * np.abs(want) + 2.0 ** -40 * big).all()
    assert (out[n] == 9).all() and int(dev.error.cpu()[0]) == 0


@pytest.mark.parametrize("sign", [1, -1])
def test_rotation_at_far_positions(nt, sign):
    """Positions up to 2^31 - 257 without their pages: a table row whose last page is there is enough."""
    import torch
    rng = np.random.default_rng(7)
    n, M = (1 << 31) - 256, ((1 << 31) - 256) // 128
    freq = [sign * f for f in [1.0, 0.7, 1e-3, 2.0 ** 19] + freqs(64)[4:]]
    pool = torch.zeros(1, 1, nt.nt_kv8_pool_bytes(nt.make_kv8_cache(n_layers=1, n_kv_heads=1, head_dim=64, page_len=128, n_pages=1,
                                                                    max_seqs=1, max_pages=M))[0], dtype=torch.uint8, device="cuda")
    table = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    table[M - 1] = 0
    length, refs, error = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (n, 1, 0))
    c = nt.make_kv8_cache(n_layers=1, n_kv_heads=1, head_dim=64, page_len=128, n_pages=1, max_seqs=1, max_pages=M,
                          pool=pool.data_ptr(), table=table.data_ptr(), len=length.data_ptr(), refs=refs.data_ptr(),
                          error=error.data_ptr())
    x = torch.from_numpy(rng.standard_normal((3, 128, 64)).astype(np.float32)).cuda()
    out = torch.empty(128, 64, device="cuda")
    begin = torch.tensor([0, 128], dtype=torch.int32, device="cuda")
    nt.nt_kv8_append(c, 0, 1, None, begin.data_ptr(), 128, "f32", x[0].data_ptr(), x[1].data_ptr(), 64, 64, freq, 1,
                     x[2].data_ptr(), 64, out.data_ptr(), 64, torch.cuda.current_stream())
    assert int(error.cpu()[0]) == 0
    # the product in integers: freq is a dyadic number, the position whole, so the angle modulo 2 pi follows from 60 digits of pi
    from fractions import Fraction
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971693993751058209749446, 10 ** 61)
    q, got = x[2].cpu().numpy().astype(np.float64), out.cpu().numpy()
    for r in (0, 1, 64, 127):
        for i in range(32):
            turns = Fraction(n - 128 + r) * Fraction(freq[i]) / two_pi
            ang = 2 * np.pi * float(turns - int(turns))
            a, b = q[r, 2 * i], q[r, 2 * i + 1]
            want = np.array([a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)])
            # 2^-33 of a turn: 2 pi 2^-33 of the pair's length
            tol = U * np.abs(want) + 2 * np.pi * 2.0 ** -33 * np.hypot(a, b)
            assert (np.abs(got[r, 2 * i:2 * i + 2] - want) <= tol).all(), (r, i)


def test_rows_passed_over_are_flagged_and_left(nt):
    """A row range that does not fit, sequences out of range, shared and missing pages: flagged, nothing written."""
    import torch
    rng = np.random.default_rng(8)
    for case in ("len", "seq", "page", "shared", "back", "beyond"):
        ref = R.RefCache(1, 2, 64, 16, 6, 3, 3)
        ref.randomize(rng)
        ref.hold([16, 16, 20])
        dev = Dev(nt, ref)
        x = rows(rng, 6, 2, 64)
        q = torch.full((6, 1, 64), 5.0, device="cuda")
        seqs, begin, want, good = [0, 1, 2], [0, 2, 4, 6], 2, [0, 2]
        if case == "len":
            dev.len[1] = 1
            ref.len[1] = 1
        elif case == "seq":
            seqs, want = [0, 3, 2], 1
        elif case == "page":
            dev.table[1, 0] = ref.table[1, 0] = 6
            want = 4
        elif case == "shared":
            dev.refs[int(ref.table[1, 0])] = ref.refs[ref.table[1, 0]] = 2
            want = 4
        elif case == "back":
            begin, good = [0, 4, 2, 2], [0]
        else:
            begin, good = [0, 2, 4, 7], [0, 1]
        for i in good:
            ref.append(0, seqs[i], x[0, begin[i]:begin[i + 1]], x[1, begin[i]:begin[i + 1]], freqs(64))
        out = torch.full((6, 64), 3.0, device="cuda")
        dev.append(*layout(torch, x, "rows"), begin, seqs, freq=freqs(64), q=q, q_out=out)
        dev.check(want)
        moved = {r for i in good for r in range(begin[i], begin[i + 1])} | ({2, 3} if case in ("page", "shared") else set())
        assert {r for r in range(6) if (out[r] != 3).any()} == moved, case


# ------------------------------------------------------------------- pages --

def test_a_run_of_the_page_operators(nt):
    """Prompts, branches that share their pages, tokens on every branch, a branch dropped, the rest moved together."""
    import torch
    rng = np.random.default_rng(9)
    ref = R.RefCache(2, 2, 64, 32, 24, 6, 6)
    ref.randomize(rng)
    dev, freq = Dev(nt, ref, 8), freqs(64)
    steps = [("extend", [0, 1], [70, 33]), ("append", [0, 1], [70, 33]), ("fork", [0, 0, 1], [2, 3, 4], None),
             ("extend", [0, 2, 3, 4], [1, 5, 1, 2]), ("append", [0, 2, 3, 4], [1, 5, 1, 2]), ("free", [3], [40]), ("free", [1], None),
             ("fork", [2], [5], [64]), ("extend", [5, 3], [9, 2]), ("append", [5, 3], [9, 2])]
    for op, seqs, *rest in steps:
        if op == "append":
            begin = np.concatenate([[0], np.cumsum(rest[0])])
            for layer in range(2):
                x = rows(rng, int(begin[-1]), 2, 64)
                store(ref, x, begin, seqs, layer, freq)
                dev.append(*layout(torch, x, "rows"), begin, seqs, layer, freq)
        else:
            getattr(ref, op)(seqs, *rest)
            getattr(dev, op)(seqs, *rest)
        dev.check()
    table, refs, live = ref.compact()
    ref.table, ref.refs = table, refs
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    nt.nt_kv8_compact(dev.c, dev.table.data_ptr(), dev.refs.data_ptr(), n.data_ptr(), dev.ws.data_ptr(), dev.wb, dev.stream())
    dev.check()
    assert int(n.cpu()[0]) == live
    ref.copy_pages([0, 1], [live, live + 1])
    nt.nt_kv8_copy_pages(dev.c, 2, dev.ints([0, 1]), dev.ints([live, live + 1]), dev.stream())
    dev.check()
    for layer in range(2):
        check_attention(dev, rng, seqs=[0, 2, 3, 4, 5], layer=layer)


# --------------------------------------------------------------- attention --

def bound(parts, n, v_top):
    """What the fp32 steps allow (U = 2^-24).  Scores: the tensor cores align the 32 products of an instruction to the
    largest and drop what lies 2^-25 below, so each of up to 4 instructions loses at most 33 2^-25 of the largest |q k| and 2^-23
    of the sum so far (truncated); q itself is held to 2^-24: 80 U of sum |q| |k| covers them, and 8 U of |s| <= that the fp32
    factors and the exponential.  Weights: that twice (numerator and sum), 2^-22 of itself for the exponential and the sum.
    Outputs: the same losses in 4 instructions a tile and an fp32 addition a tile: (70 + n / 128) U of sum p |v|.  Weights are
    held to 2^-29 of the head's first tile's largest; those errors are independent and uniform: 6 sigma of n of them."""
    want, mag, dots, total = parts
    ds = 88 * U * dots
    return (2 * ds + (90 + n / 128) * U) * mag + 6 * 2.0 ** -29 / 3 ** 0.5 * n ** 0.5 * v_top / np.minimum(total, 1e9) + 1e-30


def check_attention(dev, rng, seqs=None, ctx=None, pages=None, layer=0, q=None):
    import torch
    ref, G = dev.ref, dev.heads // dev.ref.n_kv
    n = len(seqs) if seqs is not None else ref.S
    if q is None:
        q = rng.standard_normal((n, dev.heads, ref.hd)).astype(np.float32)
    tp = None if pages is None else torch.from_numpy(np.ascontiguousarray(pages)).int().cuda()
    got = dev.attention(torch.from_numpy(q).cuda(), seqs, ctx, tp, layer).cpu().numpy()
    worst = 0.0
    for i in range(n):
        s = seqs[i] if seqs is not None else i
        c = int(ref.len[s]) if ctx is None else ctx[i]
        for g in range(ref.n_kv):
            k, v = ref.kv(layer, s, g, c)
            if pages is not None:
                pos = np.concatenate([np.arange(j * ref.pl, min(c, (j + 1) * ref.pl)) for j in pages[i, g] if j >= 0] + [np.zeros(0, int)])
                k, v = k[pos.astype(int)], v[pos.astype(int)]
            h = slice(g * G, (g + 1) * G)
            parts = R.attend(q[i, h].astype(np.float64), k, v)
            tol = bound(parts, len(k), np.abs(v).max() if len(v) else 0)
            err = np.abs(got[i, h] - parts[0])
            assert (err <= tol).all(), (i, g, len(k), err.max(), (err / tol).max())
            worst = max(worst, float((err / tol).max()))
    return got, worst


@pytest.mark.parametrize("hd,page_len", [(64, 16), (64, 64), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("kv,heads", [(1, 1), (2, 4), (3, 9), (2, 14), (2, 16), (1, 16), (5, 20)])
def test_attention(nt, hd, page_len, kv, heads):
    """Every length at which something ends: pages, chunks of 16, tiles of 128, nothing at all."""
    rng = np.random.default_rng(10 + heads)
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 255, 300, 640]
    P = sum(-(-x // page_len) for x in lens) + 2
    ref = R.RefCache(1, kv, hd, page_len, P, len(lens), -(-max(lens) // page_len))
    ref.randomize(rng)
    ref.hold(lens, rng)
    check_attention(Dev(nt, ref, heads, len(lens)), rng)


@pytest.mark.parametrize("hd,kv,heads,page_len,lens", [
    (64, 2, 8, 16, [5000]), (128, 2, 16, 64, [9001]), (128, 1, 16, 32, [20011]), (64, 3, 21, 128, [3000, 1, 700, 2000]),
    (128, 8, 32, 64, [4161]), (128, 4, 4, 64, [1500] * 40), (128, 2, 8, 16, [int(x) for x in range(1, 2000, 37)])])
def test_attention_over_many_tiles(nt, hd, kv, heads, page_len, lens):
    rng = np.random.default_rng(11)
    P = sum(-(-x // page_len) for x in lens)
    ref = R.RefCache(1, kv, hd, page_len, P, len(lens), -(-max(lens) // page_len) + 3)
    ref.randomize(rng)
    ref.hold(lens, rng)
    dev = Dev(nt, ref, heads, len(lens))
    got, _ = check_attention(dev, rng)
    rng = np.random.default_rng(11)
    assert np.isfinite(got).all()


def rel_limit(k, q, n, spread):
    """What |got - want| / |want| over a head's outputs may be for values of mean zero that the weights' errors know nothing of:
    relative errors e of the weights move out = sum w V by sum w e (V - out), in the mean square by the root mean square of e
    times |out|.  e has
    - the scores' error: 2^-24 of sum |q||k| for q's six terms (four bits each); in each of the hd / 32 instructions 33 products
      that lose up to 2^-25 of the largest, half of it in the mean, and a sum truncated at 2^-23, which is half the final one in
      the mean; 4 U of |s| for the scale, the sum of the terms and the exponent, U of the exponent's argument,
    - 2^-22 of the exponential,
    - 2^-29 of the head's largest weight, 2^spread times that where the exponents of the tile's values are so far apart.
    A tile's sum is truncated in 4 instructions, at 2^-23 of itself each, and goes through at most n / 128 / 8 + 16 additions
    that round to nearest, each its own way."""
    hd = k.shape[1]
    s, big = k @ q / hd ** 0.5, (np.abs(k) * np.abs(q)).max(1) / hd ** 0.5
    w = np.exp(s - s.max())
    ds = U * (np.abs(k) @ np.abs(q)) / hd ** 0.5 + hd / 32 * (33 / 2 * 2.0 ** -25 * big + 2.0 ** -23 * np.abs(s) / 2)
    ds += 4 * U * np.abs(s) + U * np.abs(s - s.max())
    e = (ds * ds * w * w).sum() / (w * w).sum()
    return e ** 0.5 + 2.0 ** -22 + 2.0 ** (spread - 29) * (n / (w * w).sum()) ** 0.5 + 4 * 2.0 ** -23 + (n / 1024 + 16) ** 0.5 * U


def in_terms(q, terms):
    """q as so many e4m3 terms, each a sixteenth of the one before."""
    up = 2.0 ** (7 - np.floor(np.log2(np.abs(q).max())))
    rest, out = q * up, 0.0
    for i in range(terms):
        t = R.NUMBER[R.code(rest)]
        out, rest = out + t * 16.0 ** -i, (rest - t) * 16
    return out / up


# (kv heads, query heads, hd, page_len, columns of the table, lengths, size of q): a cluster per item, then tiles shared out
WHOLE = [
    (8, 64, 128, 64, 66, [4161], 1.0), (8, 128, 128, 32, 132, [4161], 1.0), (2, 4, 64, 16, 60, [900, 129, 1, 700], 1.0),
    (1, 2, 128, 128, 30, [3001], 2.0), (4, 64, 64, 64, 40, [2500], 1.0), (8, 32, 128, 64, 141, [9001], 1.0),
    (1, 8, 128, 64, 2049, [131077], 1.0), (1, 16, 128, 64, 2049, [131077], 1.0), (1, 4, 128, 32, 4097, [131077], 2.0),
    (1, 2, 128, 128, 1025, [131077], 1.0), (1, 8, 64, 16, 8193, [131077], 1.0), (1, 16, 64, 64, 2049, [131077, 40001], 1.0),
    (3, 12, 128, 64, 400, [20011, 2047, 25000, 1], 1.0)]


@pytest.mark.parametrize("kv,heads,hd,page_len,columns,lens,size", WHOLE)
def test_attention_as_a_whole_misses_nothing(nt, kv, heads, hd, page_len, columns, lens, size):
    """Weights of similar size, so that every position counts: a position left out anywhere, q in fewer terms or weights in fewer
    bits show at several times what is allowed."""
    import torch
    rng = np.random.default_rng([45, kv, heads, hd, lens[0]])
    P = sum(-(-x // page_len) for x in lens)
    ref = R.RefCache(1, kv, hd, page_len, P, len(lens), columns)
    c = rng.integers(0, 254, ref.pool.shape, np.uint8)
    ref.pool[:] = c + (c >= 127)
    at = [ref.exp_at(g, 0) for g in range(kv)]
    for a in at:
        ref.pool[..., a:a + 2] = rng.integers(-9, -6, ref.pool.shape[:2] + (2,)).astype(np.int8).view(np.uint8)
    ref.hold(lens, rng)
    q = (rng.standard_normal((len(lens), heads, hd)) * size).astype(np.float32)
    dev = Dev(nt, ref, heads)
    got = dev.attention(torch.from_numpy(q).cuda()).cpu().numpy()
    assert int(dev.error.cpu()[0]) == 0
    G, worst, seen = heads // kv, 0.0, {}
    for i, n in enumerate(lens):
        for g in range(kv):
            k, v = ref.kv(0, i, g)
            for h in range(g * G, (g + 1) * G):
                x = q[i, h].astype(np.float64)
                w = np.exp(k @ x / hd ** 0.5 - 2 * size)
                want, limit = w @ v / w.sum(), rel_limit(k, x, n, 2)
                norm = np.linalg.norm(want)
                rel = np.linalg.norm(got[i, h] - want) / norm
                assert rel <= limit, (n, h, rel, limit)
                worst = max(worst, rel / limit)
                if h % G == 0 and n > 2000:
                    for lost in (0, n // 3, n - 1):
                        assert np.linalg.norm((v[lost] - want) * w[lost] / (w.sum() - w[lost])) > 3 * limit * norm, (n, lost)
                    x3 = in_terms(x, 3)
                    w3 = np.exp(k @ x3 / hd ** 0.5 - 2 * size)
                    few = np.rint(w / w.max() * 2.0 ** 16)
                    for name, other in (("terms", w3 @ v / w3.sum()), ("bits", few @ v / few.sum())):
                        seen[name] = min(seen.get(name, np.inf), np.linalg.norm(other - want) / norm / limit)
    assert all(x > 2 for x in seen.values()), seen
    print(f"kv {kv} heads {heads} hd {hd} page {page_len} lengths {lens}: {worst:.2f} of the limit {limit:.1e}; {seen}")


def test_what_lies_behind_the_end_is_never_looked_at(nt):
    """The last page's other positions and all free pages hold NaN codes and the largest exponents."""
    rng = np.random.default_rng(12)
    for page_len in (16, 64, 128):
        lens = [1, 17, 100, 130, 260, 0]
        P = sum(-(-x // page_len) for x in lens) + 3
        ref = R.RefCache(1, 2, 64, page_len, P, 6, -(-260 // page_len))
        ref.randomize(rng)
        ref.hold(lens, rng)
        for p in range(P):
            if not ref.refs[p]:
                ref.pool[0, p] = 0xFF
        d = np.arange(64)
        for s, n in enumerate(lens):
            for t in range(n, ref.pages(n) * page_len):
                row = ref.pool[0, ref.table[s, t // page_len]]
                for g in range(2):
                    row[ref.k_at(g, t % page_len, d)] = 0x7F
                    row[ref.v_at(g, t % page_len, d)] = 0xFF
        got, _ = check_attention(Dev(nt, ref, 16), rng)
        assert np.isfinite(got).all()


def test_drafts_see_the_positions_up_to_their_own(nt):
    rng = np.random.default_rng(13)
    ref = R.RefCache(1, 2, 128, 64, 30, 3, 10)
    ref.randomize(rng)
    ref.hold([600, 130, 40], rng)
    seqs, ctx = [0] * 5 + [1] * 4 + [2, 2], [596, 597, 598, 599, 600, 127, 128, 129, 130, 0, 40]
    got, _ = check_attention(Dev(nt, ref, 8, 11), rng, seqs, ctx)
    assert (got[9] == 0).all()


@pytest.mark.parametrize("hd,kv,heads,page_len,longest,n", [
    (128, 2, 2, 16, 700, 60), (128, 2, 4, 64, 1500, 37), (64, 3, 9, 32, 900, 41), (128, 1, 4, 128, 6000, 23), (64, 2, 14, 16, 400, 30),
    (128, 4, 32, 64, 2000, 25), (64, 1, 16, 64, 3000, 9), (64, 1, 1, 16, 200, 3), (128, 8, 32, 64, 4000, 20)])
def test_entries_of_one_sequence_in_any_order(nt, hd, kv, heads, page_len, longest, n):
    """Runs of any length of the same sequence, lengths in any order, nothing at all among them."""
    rng = np.random.default_rng(29 + n)
    lens = [longest, 1, longest // 2, 130]
    P = sum(-(-x // page_len) for x in lens)
    ref = R.RefCache(1, kv, hd, page_len, P, 4, -(-longest // page_len))
    ref.randomize(rng)
    ref.hold(lens, rng)
    seqs, ctx = [], []
    while len(seqs) < n:
        s = int(rng.integers(4))
        for _ in range(int(rng.choice([1, 2, 5, 9]))):
            seqs.append(s)
            ctx.append(int(rng.choice([lens[s], max(0, lens[s] - int(rng.integers(6))), int(rng.integers(lens[s] + 1)), 0],
                                      p=[0.4, 0.3, 0.2, 0.1])))
    got, _ = check_attention(Dev(nt, ref, heads, n), rng, seqs[:n], ctx[:n])
    assert (got[np.array(ctx[:n]) == 0] == 0).all()


def test_a_missing_page_concerns_the_entries_that_see_it(nt):
    import torch
    rng = np.random.default_rng(30)
    for longest, bad_at in ((1000, 12), (1000, 0), (150, 8), (5000, 300)):
        ref = R.RefCache(1, 1, 64, 16, 400, 2, 320)
        ref.randomize(rng)
        ref.hold([longest, 40], rng)
        dev = Dev(nt, ref, 2, 8)
        dev.table[0, bad_at] = 400
        at = 16 * bad_at
        seqs, ctx = [0, 0, 0, 0, 1, 0, 0, 9], [longest, at, at + 1, max(0, at - 20), 40, longest // 2, min(longest, at + 16), 5]
        q = rng.standard_normal((8, 2, 64)).astype(np.float32)
        got = dev.attention(torch.from_numpy(q).cuda(), seqs, ctx).cpu().numpy()
        assert int(dev.error.cpu()[0]) == 1 | 4
        for i, (s, c) in enumerate(zip(seqs, ctx)):
            if s == 9 or (s == 0 and c > at):
                assert np.isnan(got[i]).all(), (longest, i)
                continue
            k, v = ref.kv(0, s, 0, c)
            parts = R.attend(q[i].astype(np.float64), k, v)
            assert (np.abs(got[i] - parts[0]) <= bound(parts, len(k), np.abs(v).max() if c else 0)).all(), (longest, i)


def test_a_value_that_is_no_number_concerns_the_entries_that_see_it(nt):
    import torch
    rng = np.random.default_rng(31)
    for hd, heads in ((128, 2), (64, 8)):
        ref = R.RefCache(1, 1, hd, 32, 20, 1, 20)
        ref.randomize(rng)
        ref.hold([300], rng)
        for pos, d in ((290, 5), (293, 60), (130, 7)):
            ref.pool[0, ref.table[0, pos // 32]][ref.v_at(0, pos % 32, d)] = 0xFF
        ref.pool[0, ref.table[0, 296 // 32]][ref.k_at(0, 296 % 32, 3)] = 0x7F
        ctx = [297, 290, 291, 294, 130, 131, 296, 295, 300, 0, 128]
        q = rng.standard_normal((len(ctx), heads, hd)).astype(np.float32)
        got = Dev(nt, ref, heads, len(ctx)).attention(torch.from_numpy(q).cuda(), [0] * len(ctx), ctx).cpu().numpy()
        for i, c in enumerate(ctx):
            nan = {d for pos, d in ((290, 5), (293, 60), (130, 7)) if pos < c}
            if c > 296:
                nan = set(range(hd))
            assert {int(d) for d in np.nonzero(np.isnan(got[i, 0]))[0]} == nan, (hd, c)


def test_strides_and_layers(nt):
    import torch
    rng = np.random.default_rng(14)
    ref = R.RefCache(3, 2, 64, 32, 12, 2, 8)
    ref.randomize(rng)
    ref.hold([200, 77], rng)
    dev = Dev(nt, ref, 6)
    q = rng.standard_normal((2, 6, 64)).astype(np.float32)
    want, _ = check_attention(dev, rng, layer=2, q=q)
    wide = torch.full((2, 6 * 64 + 20), float("nan"), device="cuda")
    wide[:, :384] = torch.from_numpy(q).cuda().flatten(1)
    out = torch.full((2, 6 * 64 + 12), 5.0, device="cuda")
    dev.attention(wide[:, :384].unflatten(1, (6, 64)), layer=2, out=out[:, :384].unflatten(1, (6, 64)))
    np.testing.assert_array_equal(out[:, :384].cpu().numpy(), want.reshape(2, -1))
    assert (out[:, 384:] == 5).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 30.0, 1e4, 1e15])
def test_scores_of_any_size(nt, scale):
    """From a flat softmax to one that a single position wins, whose values come out as they are held."""
    rng = np.random.default_rng(15)
    ref = R.RefCache(1, 1, 128, 64, 20, 1, 20)
    ref.randomize(rng)
    ref.hold([1100], rng)
    dev = Dev(nt, ref, 8)
    q = (rng.standard_normal((1, 8, 128)) * scale).astype(np.float32)
    if scale < 100:
        check_attention(dev, rng, q=q)
        return
    import torch
    got = dev.attention(torch.from_numpy(q).cuda()).cpu().numpy()[0]
    k, v = ref.kv(0, 0, 0)
    s = q[0].astype(np.float64) @ k.T / 128 ** 0.5
    top = np.sort(s, 1)
    assert (top[:, -1] - top[:, -2] > 40 + 200 * U * np.abs(s).max()).sum() >= 4      # a clear winner
    for h in range(8):
        if top[h, -1] - top[h, -2] > 40 + 200 * U * np.abs(s).max():
            np.testing.assert_allclose(got[h], v[s[h].argmax()], rtol=64 * U, atol=1e-12)


def test_exponents_of_every_size(nt):
    """Pages whose keys and values differ by many powers of two: the large ones decide, the small ones are not lost."""
    rng = np.random.default_rng(16)
    ref = R.RefCache(1, 1, 64, 16, 40, 3, 14)
    ref.randomize(rng)
    ref.hold([200, 200, 200], rng)
    for j in range(13):
        for s, (ke, ve) in enumerate([(-9, (-30, 0, 20)[j % 3]), (-9, -8 + 2 * j), (-12 + j % 5, 12 - 3 * j)]):
            row = ref.pool[0, ref.table[s, j]]
            row[ref.exp_at(0, 0)], row[ref.exp_at(0, 1)] = np.int8(ke).view(np.uint8), np.int8(ve).view(np.uint8)
    dev = Dev(nt, ref, 4)
    check_attention(dev, rng, q=(0.2 * rng.standard_normal((3, 4, 64))).astype(np.float32))


# (kv heads, query heads, hd, page_len, columns of the table, length): a cluster per item, then tiles shared out
APART = [(2, 4, 64, 16, 9, 129), (1, 8, 128, 32, 20, 600), (2, 32, 64, 64, 12, 700), (1, 2, 128, 64, 2, 128), (1, 2, 64, 128, 5, 600),
         (1, 8, 128, 16, 2000, 900), (2, 4, 64, 32, 1000, 3000), (1, 16, 128, 64, 800, 1500), (2, 2, 64, 16, 700, 128),
         (1, 5, 128, 128, 500, 1000)]


@pytest.mark.parametrize("gap", [3, 4, 5, 8, 12, 16, 24, 32, 60, 120])
@pytest.mark.parametrize("kv,heads,hd,page_len,columns,n", APART)
def test_pages_whose_values_differ_by_many_powers_of_two(nt, kv, heads, hd, page_len, columns, n, gap):
    """Every third page's values are 2^gap larger, some 2^(gap / 2), and their scores so far below the others' that they add less
    than e^-25: the outputs are the small values' mean, to fp32's accuracy.

    Allowed, relative to a head's outputs: the values have mean zero and the weights' errors know nothing of them, so relative
    errors e of the weights move out = sum w V by e |V| w, independent from position to position: in the mean square by the
    root mean square of e times |out|.  e is the scores' error, 12 U of their size |q||k| (24 bits of q, the losses of 4
    instructions, 2^-25 and 2^-23 of the largest product each, and the fp32 factors), 2^-22 of the exponential, and 2^-22 of
    the head's largest weight for the digits (2^-29 and exponents up to 7 apart), which is 2^-22 sqrt(n / sum w^2) of out, w
    relative to the largest; a sum of 128 loses 2^-23 of itself in each of 4 instructions and U in each fp32 addition."""
    import torch
    rng = np.random.default_rng([41, gap, hd, heads])
    held = -(-n // page_len)
    ref = R.RefCache(1, kv, hd, page_len, held + 1, 1, columns)
    ref.randomize(rng)
    ref.hold([n], rng)
    d, t = np.arange(hd), np.arange(page_len)[:, None]
    for j in range(held):
        row, up = ref.pool[0, ref.table[0, j]], gap if j % 3 == 1 else gap // 2 if j % 5 == 2 else 0
        for g in range(kv):
            c = R.code(rng.standard_normal((page_len, hd)) * 0.3 * (d > 0) + (d == 0) * (-8 if up else 0))
            row[ref.k_at(g, t, d)] = c
            row[ref.v_at(g, t, d)] = R.code(rng.standard_normal((page_len, hd)) * 100)
            row[ref.exp_at(g, 0)], row[ref.exp_at(g, 1)] = 0, np.int8(up - min(gap, 60)).view(np.uint8)
    q = rng.standard_normal((1, heads, hd)).astype(np.float32)
    q[..., 0] = (gap * 0.6931 + 25) / 8 * hd ** 0.5          # (e^-25 2^-gap)
    got = Dev(nt, ref, heads).attention(torch.from_numpy(q).cuda()).cpu().numpy()[0]
    G = heads // kv
    for h in range(heads):
        k, v = ref.kv(0, 0, h // G)
        x = q[0, h].astype(np.float64)
        s = k @ x / hd ** 0.5
        w = np.exp(s - s.max())
        want = R.attend(x[None], k, v)[0][0]
        dots = (np.abs(k) @ np.abs(x))[w > 1e-12].max() / hd ** 0.5
        e = 12 * U * dots + 2.0 ** -22 + 2.0 ** -22 * (n / (w * w).sum()) ** 0.5
        limit = e + 4 * 2.0 ** -23 + (n / 128 + 8) ** 0.5 * U
        rel = np.linalg.norm(got[h] - want) / np.linalg.norm(want)
        assert rel <= limit, (h, rel, limit)


@pytest.mark.parametrize("bits", [6.6, 11.5, 19.3, 22.4, 26.4, 29.2, 33.5, 45.3, 70.7, 95.2])
@pytest.mark.parametrize("kv,heads,hd,page_len,columns,n", [
    (1, 2, 128, 64, 20, 1200), (2, 16, 64, 16, 40, 600), (1, 16, 128, 32, 8, 250), (1, 4, 64, 128, 3, 300), (1, 8, 128, 64, 2048, 131072),
    (1, 4, 64, 16, 2000, 30000), (2, 32, 128, 128, 400, 5000)])
def test_many_low_weights_beside_a_large_one(nt, kv, heads, hd, page_len, columns, n, bits):
    """One position near the start has the largest score of all heads, the others' weights lie about 2^bits below, but their values
    are larger by as much as they are too few: the outputs are made of both parts, to fp32's accuracy.

    Allowed, relative to a head's outputs: the others' common score is off by 12 U of its size, their weights by 2^-22 for the
    exponential, and for the digits by 2^-25 where their values are more than 2^4 larger, else by 2^-29 of the largest weight,
    rounded each its own way (3 sigma of n uniform errors); twice that, since the outputs may be smaller than the sum of their two
    parts; a sum of 128 loses 2^-23 of itself in each of 4 instructions, and an fp32 addition U in the mean square, the
    sum of the weights as well."""
    import torch
    rng = np.random.default_rng([42, int(bits), hd, heads])
    held = -(-n // page_len)
    ref = R.RefCache(1, kv, hd, page_len, held, 1, columns)
    ref.hold([n], rng)
    up = int(np.clip(round(bits - np.log2(n)), -40, 90))
    d, t = np.arange(hd), np.arange(page_len)[:, None]
    for j in range(held):
        row = ref.pool[0, ref.table[0, j]]
        for g in range(kv):
            k = np.where(d == 0, -8.0, 0.1 * rng.standard_normal((page_len, hd)))
            v = 100 + 30 * rng.standard_normal((page_len, hd)) * (d % 2) - 200 * (d % 3 == 0)
            if j == 0:                                       # (no other position of its page: its values' exponent is its own)
                k[1:, 0], k[0] = -100, 0
                v[0] = 100 * rng.standard_normal(hd)
            row[ref.k_at(g, t, d)], row[ref.v_at(g, t, d)] = R.code(k), R.code(v)
            row[ref.exp_at(g, 0)], row[ref.exp_at(g, 1)] = 0, np.int8(up if j else 0).view(np.uint8)
    q = (0.1 * rng.standard_normal((1, heads, hd))).astype(np.float32)
    q[..., 0] = (bits + np.linspace(-0.7, 0.7, heads)) * 0.6931 / 8 * hd ** 0.5
    got = Dev(nt, ref, heads).attention(torch.from_numpy(q).cuda()).cpu().numpy()[0]
    G = heads // kv
    for h in range(heads):
        k, v = ref.kv(0, 0, h // G)
        x = q[0, h].astype(np.float64)
        want, alone = R.attend(x[None], k, v)[0][0], v[0]
        digits = 2.0 ** -25 if up > 4 else 3 * 2.0 ** (bits + 1 - 29) / (3 * n) ** 0.5
        limit = 2 * (12 * U * (bits + 1) * 0.6931 + 2.0 ** -22 + digits) + 8 * 2.0 ** -23 + 2 * (n / 128 + 8) ** 0.5 * U
        rel = np.linalg.norm(got[h] - want) / np.linalg.norm(want)
        assert rel <= limit, (h, rel, limit)
        assert up < 0 or np.linalg.norm(alone - want) > 1000 * limit * np.linalg.norm(want)


@pytest.mark.parametrize("larger", [8, 16, 24, 32])
@pytest.mark.parametrize("nats", [20, 50, 80])
@pytest.mark.parametrize("page_len,columns", [(16, 8), (32, 4), (64, 2), (16, 900), (32, 900), (64, 900)])
def test_large_values_with_low_weights_in_the_same_tile(nt, page_len, columns, nats, larger):
    """Two kinds of pages in one tile: the ones' scores lie 20 to 80 nats below, their values are 2^larger larger, so that they are
    everything, nothing or something between.  Limits as in test_many_low_weights_beside_a_large_one."""
    import torch
    rng = np.random.default_rng([43, nats, larger])
    hd, heads, n = 128, 8, 128
    ref = R.RefCache(1, 1, hd, page_len, n // page_len, 1, columns)
    ref.hold([n], rng)
    d, t = np.arange(hd), np.arange(page_len)[:, None]
    for j in range(n // page_len):
        row = ref.pool[0, ref.table[0, j]]
        row[ref.k_at(0, t, d)] = R.code(np.where(d == 0, -8.0 * (j % 2), 0.1 * rng.standard_normal((page_len, hd))))
        row[ref.v_at(0, t, d)] = R.code(100 + 30 * rng.standard_normal((page_len, hd)) - 200 * (d % (2 + j % 2) == 0))
        row[ref.exp_at(0, 0)], row[ref.exp_at(0, 1)] = 0, larger * (j % 2)
    q = (0.1 * rng.standard_normal((1, heads, hd))).astype(np.float32)
    q[..., 0] = (nats + np.linspace(-3, 3, heads)) / 8 * hd ** 0.5
    got = Dev(nt, ref, heads).attention(torch.from_numpy(q).cuda()).cpu().numpy()[0]
    k, v = ref.kv(0, 0, 0)
    for h in range(heads):
        want = R.attend(q[0, h][None].astype(np.float64), k, v)[0][0]
        limit = 2 * (12 * U * (nats + 4) + 2.0 ** -22 + 2.0 ** -25) + 8 * 2.0 ** -23 + 2 * 3 * U
        rel = np.linalg.norm(got[h] - want) / np.linalg.norm(want)
        assert rel <= limit, (h, rel, limit)


@pytest.mark.parametrize("up", [0, 4, 7])
@pytest.mark.parametrize("bits", [28.7, 29.4, 31.6])
@pytest.mark.parametrize("kv,heads,hd,page_len,n,entries", [(1, 8, 128, 64, 131072, 305), (1, 16, 64, 128, 36000, 400), (2, 4, 128, 16, 64000, 160),
                                                            (1, 2, 64, 32, 20000, 1)])
def test_many_weights_below_the_last_digit(nt, kv, heads, hd, page_len, n, entries, bits, up):
    """One large weight and n that lie 2^bits below it, less than the last digit, their values 2^up larger: their sum is in the
    outputs all the same.  (Several hundred entries, so that one CTA has a whole item: a part has a largest weight of its own.)

    Allowed, relative to a head's outputs: a weight below the last digit, 2^-28 of the largest, gets one or none, off by half of it in the
    mean square at most and each its own way, so that n of them move the outputs by sqrt(n) 2^-29 of a value, six times that in the
    worst case; the common score and the sums as in test_many_low_weights_beside_a_large_one."""
    import torch
    rng = np.random.default_rng([44, hd, up])
    held = -(-n // page_len)
    ref = R.RefCache(1, kv, hd, page_len, held, 1, held)
    ref.hold([n], rng)
    d, t = np.arange(hd), np.arange(page_len)[:, None]
    for j in range(held):
        row = ref.pool[0, ref.table[0, j]]
        for g in range(kv):
            row[ref.k_at(g, t, d)] = R.code(np.where((t == 0) & (j == 0) & (d == 0), 8.0, 0.0))
            row[ref.v_at(g, t, d)] = R.code(100 + 10 * rng.standard_normal((page_len, hd)))
            row[ref.exp_at(g, 0)], row[ref.exp_at(g, 1)] = 0, np.int8(up if j else 0).view(np.uint8)
    q = np.zeros((1, heads, hd), np.float32)
    q[..., 0] = (bits + np.linspace(0, 0.3, heads)) * 0.6931472 / 8 * hd ** 0.5
    got = Dev(nt, ref, heads, entries).attention(torch.from_numpy(q).cuda().repeat(entries, 1, 1), [0] * entries).cpu().numpy()
    for h in range(heads):
        k, v = ref.kv(0, 0, h // (heads // kv))
        want = R.attend(q[0, h][None].astype(np.float64), k, v)[0][0]
        digits = 6 * n ** 0.5 * 2.0 ** -29 * np.linalg.norm(v[page_len:]) / (n - page_len) ** 0.5 / np.linalg.norm(want)
        limit = digits + 2 * (12 * U * (bits + 1) * 0.6931 + 2.0 ** -22) + 8 * 2.0 ** -23 + 2 * (n / 128 + 8) ** 0.5 * U
        rel = np.linalg.norm(got[:, h] - want, axis=1).max() / np.linalg.norm(want)
        assert rel <= limit, (h, rel, limit)


def test_one_strong_position_far_from_the_start(nt):
    """The reference of the weights has to move: scores rise along the sequence, and one position outweighs the rest."""
    rng = np.random.default_rng(17)
    ref = R.RefCache(1, 1, 64, 64, 50, 2, 25)
    ref.hold([1500, 1500])
    k = (0.3 * rng.standard_normal((2, 1500, 1, 64))).astype(np.float32)
    k[0] += (np.arange(1500) / 300).astype(np.float32)[:, None, None]
    k[1, 1234] = 8
    v = rng.standard_normal((2, 1500, 1, 64)).astype(np.float32)
    for s in range(2):
        ref.append(0, s, k[s], v[s])
    check_attention(Dev(nt, ref, 3), rng, q=np.abs(rng.standard_normal((2, 3, 64))).astype(np.float32))


def test_nan_keys_values_and_queries(nt):
    rng = np.random.default_rng(18)
    ref = R.RefCache(1, 1, 64, 32, 40, 4, 10)
    ref.randomize(rng)
    ref.hold([300, 300, 300, 300], rng)
    ref.pool[0, ref.table[0, 3]][ref.k_at(0, 5, 9)] = 0x7F
    ref.pool[0, ref.table[1, 9]][ref.v_at(0, 5, 9)] = 0xFF
    import torch
    dev = Dev(nt, ref, 4)
    q = rng.standard_normal((4, 4, 64)).astype(np.float32)
    q[2, 1, 3] = np.nan
    got = dev.attention(torch.from_numpy(q).cuda()).cpu().numpy()
    assert np.isnan(got[0]).all()
    assert np.isnan(got[1, :, 9]).all() and np.isnan(got[1]).sum() == 4
    assert np.isnan(got[2, 1]).all() and np.isfinite(got[2, [0, 2, 3]]).all() and np.isfinite(got[3]).all()


def test_unreadable_entries_give_nan_and_flags(nt):
    import torch
    rng = np.random.default_rng(19)
    for case, want in (("seq", 1), ("len", 2), ("ctx", 2), ("page", 4), ("below", 4)):
        ref = R.RefCache(1, 2, 64, 32, 20, 3, 10)
        ref.randomize(rng)
        ref.hold([200, 150, 90], rng)
        dev = Dev(nt, ref, 4)
        seqs, ctx = [0, 1, 2], [200, 150, 90]
        if case == "seq":
            seqs[1] = 3
        elif case == "len":
            dev.len[1] = 10 * 32 + 1
        elif case == "ctx":
            ctx[1] = 151
        else:
            dev.table[1, 2] = 20 if case == "page" else -5
        q = rng.standard_normal((3, 4, 64)).astype(np.float32)
        got = dev.attention(torch.from_numpy(q).cuda(), seqs, ctx).cpu().numpy()
        assert np.isnan(got[1]).all() and np.isfinite(got[[0, 2]]).all(), case
        assert int(dev.error.cpu()[0]) == want


# ------------------------------------------------------------------ sparse --

@pytest.mark.parametrize("hd,kv,heads,page_len,top,first,last", [
    (64, 1, 1, 16, 1, 0, 0), (64, 2, 8, 16, 7, 1, 2), (128, 3, 9, 32, 4, 0, 1), (128, 1, 16, 64, 5, 2, 3), (64, 1, 7, 128, 3, 1, 0),
    (128, 2, 16, 16, 40, 1, 1)])
def test_select_and_attend(nt, hd, kv, heads, page_len, top, first, last):
    import torch
    rng = np.random.default_rng(20 + hd + top)
    lens = [0, 1, page_len * top, page_len * top + 1, 50 * page_len - 3, 33 * page_len, 9 * page_len + 1]
    P = sum(-(-x // page_len) for x in lens)
    ref = R.RefCache(1, kv, hd, page_len, P, len(lens), max(50, top + 1))
    ref.randomize(rng)
    ref.hold(lens, rng)
    dev = Dev(nt, ref, heads)
    q = rng.standard_normal((len(lens), heads, hd)).astype(np.float32)
    got = dev.select(torch.from_numpy(q).cuda(), top, first, last).cpu().numpy()
    G = heads // kv
    want = np.stack([[ref.select(0, s, g, q[s, g * G:(g + 1) * G], top, first, last) for g in range(kv)] for s in range(len(lens))])
    np.testing.assert_array_equal(got, want)
    check_attention(dev, rng, pages=got, q=q)
    dev.check()


def test_select_many_pages_with_many_ties(nt):
    """More pages than a CTA has threads, scores from few values: the lower pages win, wherever they stand."""
    import torch
    rng = np.random.default_rng(21)
    ref = R.RefCache(1, 1, 64, 16, 3000, 2, 3000)
    ref.hold([16 * 2500, 16 * 300 + 1], rng)
    for p in range(3000):
        ref.pool[0, p][ref.exp_at(0, 0)] = np.int8(rng.integers(-2, 1)).view(np.uint8)
        at = ref.exp_at(0, 0) + 16
        b = np.repeat(rng.integers(-2, 3, 2), 64)
        ref.pool[0, p][at:at + 128] = np.sort(b).astype(np.int8).view(np.uint8)
    dev = Dev(nt, ref, 2)
    q = np.ones((2, 2, 64), np.float32)
    q[:, 1] *= -0.5
    for top, first, last in ((1, 0, 0), (600, 1, 2), (1024, 0, 5), (2499, 3, 0)):
        got = dev.select(torch.from_numpy(q).cuda(), top, first, last).cpu().numpy()
        for s in range(2):
            np.testing.assert_array_equal(got[s, 0], ref.select(0, s, 0, q[s], top, first, last))


@pytest.mark.parametrize("pages", [300, 938, 2500, 4096, 5000, 9001])
def test_select_among_many_scores(nt, pages):
    """Scores that lie close together, so that the last bins hold few numbers each; more pages than a CTA holds in registers."""
    import torch
    rng = np.random.default_rng(32 + pages)
    ref = R.RefCache(1, 1, 64, 16, pages, 1, pages)
    ref.hold([16 * pages - 3], rng)
    at = ref.exp_at(0, 0)
    for p in range(pages):
        ref.pool[0, p][at] = np.int8(rng.integers(-7, -5)).view(np.uint8)
        ref.pool[0, p][at + 16:at + 144] = np.sort(rng.integers(-112, 113, (2, 64)), 0).reshape(-1).astype(np.int8).view(np.uint8)
    dev = Dev(nt, ref, 4)
    for k, spread in enumerate((1.0, 0.01, 30.0)):
        q = (rng.standard_normal((1, 4, 64)) * spread).astype(np.float32)
        if k == 1:
            q[0, :, 1:] = 0                                  # one dimension decides: many equal scores, and neighbours
        for top, first, last in ((1, 0, 0), (7, 1, 2), (64, 1, 4), (96, 0, 0), (255, 3, 3), (pages - 1, 0, 1)):
            got = dev.select(torch.from_numpy(q).cuda(), top, first, last).cpu().numpy()
            np.testing.assert_array_equal(got[0, 0], ref.select(0, 0, 0, q[0], top, first, last), err_msg=str((k, top)))


def test_select_with_ctx_lists_and_odd_queries(nt):
    import torch
    rng = np.random.default_rng(22)
    ref = R.RefCache(2, 2, 128, 16, 100, 2, 60)
    ref.randomize(rng)
    ref.hold([900, 600], rng)
    dev = Dev(nt, ref, 6, 6)
    seqs, ctx = [0, 0, 1, 0, 1, 1], [900, 333, 600, 1, 17, 599]
    q = rng.standard_normal((6, 6, 128)).astype(np.float32)
    q[0, 0, 0], q[1, 2, 5], q[2, :, 3], q[3] = np.nan, np.inf, -np.inf, 0
    q[4] *= np.float32(1e-42)
    q[5, :3], q[5, 3:] = q[5, :3] * np.float32(1e-20), q[5, 3:] * np.float32(1e30)
    got = dev.select(torch.from_numpy(q).cuda(), 5, 1, 1, seqs, ctx, layer=1).cpu().numpy()
    for i in range(6):
        for g in range(2):
            np.testing.assert_array_equal(got[i, g], ref.select(1, seqs[i], g, q[i, 3 * g:3 * g + 3], 5, 1, 1, ctx[i]))


def test_select_unreadable_entries(nt):
    import torch
    rng = np.random.default_rng(23)
    ref = R.RefCache(1, 1, 64, 16, 60, 3, 20)
    ref.randomize(rng)
    ref.hold([300, 300, 300], rng)
    ref.table[2, 4] = 60
    dev = Dev(nt, ref, 2)
    q = rng.standard_normal((3, 2, 64)).astype(np.float32)
    got = dev.select(torch.from_numpy(q).cuda(), 4, 1, 1, [0, 7, 2], None).cpu().numpy()
    assert (got[1] == -1).all() and int(dev.error.cpu()[0]) == 1 | 4
    for s in (0, 2):
        np.testing.assert_array_equal(got[s, 0], ref.select(0, s, 0, q[s], 4, 1, 1))


def test_empty_lists_among_others(nt):
    """Many entries whose lists are empty or end early, so that whole stretches of tiles have nothing to do."""
    rng = np.random.default_rng(28)
    ref = R.RefCache(1, 2, 64, 16, 60, 1, 60)
    ref.randomize(rng)
    ref.hold([900], rng)
    n, top = 400, 40
    pages = np.full((n, 2, top), -1, np.int32)
    for i in range(n):
        for g in range(2):
            m = int(rng.choice([0, 0, 0, 1, 9, 40]))
            pages[i, g, :m] = np.sort(rng.choice(57, m, replace=False))
    check_attention(Dev(nt, ref, 2, n), rng, [0] * n, pages=pages)


@pytest.mark.parametrize("lists,bad", [
    ([[0, 3, 9, -1]], False), ([[-1, -1, -1, -1]], False), ([[-1, 3, 9, -1]], True), ([[0, 0, 1, 2]], True), ([[3, 1, 2, 4]], True), ([[0, 1, 2, 13]], True),
    ([[0, 1, 1 << 30, -1]], True)])
def test_page_lists_of_the_caller(nt, lists, bad):
    """Ascending places within the sequence; anything else is NaN for that kv head and a flag, the others are untouched."""
    import torch
    rng = np.random.default_rng(24)
    ref = R.RefCache(1, 2, 64, 16, 30, 1, 20)
    ref.randomize(rng)
    ref.hold([13 * 16 - 5], rng)
    dev = Dev(nt, ref, 4)
    pages = np.array([[[1, 5, 12, -1]] + lists], np.int32)
    q = rng.standard_normal((1, 4, 64)).astype(np.float32)
    if not bad:
        check_attention(dev, rng, pages=pages, q=q)
        dev.check()
        return
    got = dev.attention(torch.from_numpy(q).cuda(), pages=torch.from_numpy(pages).cuda()).cpu().numpy()
    assert np.isnan(got[0, 2:]).all() and np.isfinite(got[0, :2]).all() and int(dev.error.cpu()[0]) == 4


def test_lists_longer_than_the_table_and_places_that_are_not_looked_at(nt):
    """n_select above the table's columns, in a selection and a caller's lists; what stands behind the first m places is nobody's."""
    import torch
    rng = np.random.default_rng(33)
    ref = R.RefCache(1, 2, 64, 32, 30, 3, 12)
    ref.randomize(rng)
    ref.hold([12 * 32, 77, 0], rng)
    dev = Dev(nt, ref, 6)
    q = rng.standard_normal((3, 6, 64)).astype(np.float32)
    got = dev.select(torch.from_numpy(q).cuda(), 70, 2, 3).cpu().numpy()
    for s in range(3):
        m = ref.pages(int(ref.len[s]))
        assert (got[s, :, :m] == np.arange(m)).all() and (got[s, :, m:] == -1).all()
    check_attention(dev, rng, pages=got, q=q)
    behind = got.copy()
    for s in range(3):
        behind[s, :, ref.pages(int(ref.len[s])):] = rng.integers(-5, 1 << 30, 70 - ref.pages(int(ref.len[s])))
    out = dev.attention(torch.from_numpy(q).cuda(), pages=torch.from_numpy(behind).cuda())
    assert torch.equal(out, dev.attention(torch.from_numpy(q).cuda(), pages=torch.from_numpy(got).cuda()))
    dev.check()


def test_pages_of_any_bytes(nt):
    """Pages that were never written hold anything: the selection stays a selection, and nothing beside the outputs is touched."""
    import torch
    rng = np.random.default_rng(34)
    ref = R.RefCache(1, 2, 64, 16, 700, 2, 600)
    ref.pool[:] = rng.integers(0, 256, ref.pool.shape)
    for p in range(0, 700, 3):   # exponents of which no number is made
        for g in range(2):
            ref.pool[0, p, ref.exp_at(g, 0):ref.exp_at(g, 0) + 2] = rng.choice([127, 128, 129], 2)
    ref.hold([16 * 600 - 1, 1500], rng)
    dev = Dev(nt, ref, 4)
    q = torch.from_numpy(rng.standard_normal((2, 4, 64)).astype(np.float32)).cuda()
    for top, first, last in ((1, 0, 0), (1, 0, 1), (60, 0, 0), (90, 3, 4)):
        out = torch.full((3, 2, 2, top), -7, dtype=torch.int32, device="cuda")
        nt.nt_kv8_select(dev.c, 0, 4, 2, None, None, q.data_ptr(), 256, top, first, last, out[1].data_ptr(), dev.ws.data_ptr(), dev.wb,
                         dev.stream())
        assert (out[0] == -7).all() and (out[2] == -7).all()
        for s in range(2):
            m = ref.pages(int(ref.len[s]))
            for row in out[1, s].cpu().numpy():
                assert (np.diff(row) > 0).all() and row[0] >= 0 and row[-1] < m
                assert set(range(first)) | set(range(m - last, m)) <= set(row.tolist())
        dev.attention(q, pages=out[1].contiguous())
    dev.attention(q)
    dev.check()


def test_more_entries_than_one_launch_takes(nt):
    """Over 512 entries, listed and not, dense and over selected pages; over 65535 (entry, kv head) pairs in a selection."""
    import torch
    rng = np.random.default_rng(35)
    S, hd = 700, 64
    lens = rng.integers(0, 40, S)
    lens[[3, 511, 512, 699]] = 190, 200, 0, 129
    ref = R.RefCache(1, 1, hd, 16, sum(-(-int(x) // 16) for x in lens), S, 13)
    ref.randomize(rng)
    ref.hold(lens, rng)
    dev = Dev(nt, ref, 2, 70000)
    check_attention(dev, rng)
    seqs = rng.integers(0, S, 1100)
    ctx = [int(rng.integers(0, lens[s] + 1)) for s in seqs]
    q = rng.standard_normal((1100, 2, hd)).astype(np.float32)
    check_attention(dev, rng, seqs, ctx, q=q)
    pages = dev.select(torch.from_numpy(q).cuda(), 3, 1, 1, seqs, ctx).cpu().numpy()
    for i in range(1100):
        np.testing.assert_array_equal(pages[i, 0], ref.select(0, seqs[i], 0, q[i], 3, 1, 1, ctx[i]))
    check_attention(dev, rng, seqs, ctx, pages, q=q)
    many = torch.arange(65536, device="cuda") % 1100
    for n in (65535, 65536):
        got = dev.select(torch.from_numpy(q).cuda()[many[:n]].contiguous(), 3, 1, 1, seqs[many[:n].cpu().numpy()], np.asarray(ctx)[many[:n].cpu().numpy()])
        assert torch.equal(got, torch.from_numpy(pages).cuda()[many[:n]])
    dev.check()


def test_offsets_beyond_32_bits(nt):
    """A pool of over 4 GB whose used pages lie at its end, in the last layer."""
    import torch
    rng = np.random.default_rng(36)
    small = R.RefCache(1, 8, 128, 64, 6, 2, 3)
    small.randomize(rng)
    small.hold([150, 65], rng)
    pages, layers = 10000, 4
    pool = torch.zeros(layers, pages, small.page_bytes, dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    pool[-1, pages - 6:] = torch.from_numpy(small.pool[0]).cuda()
    big = R.RefCache(1, 8, 128, 64, 1, 2, 3)
    big.shape.update(n_pages=pages, n_layers=layers)
    big.table = np.where(small.table >= 0, small.table + pages - 6, -1).astype(np.int32)
    big.len, big.refs = small.len, np.zeros(pages, np.int32)
    big.refs[big.table[big.table >= 0]] = 1
    dev, near = Dev(nt, big, 64), Dev(nt, small, 64)
    dev.pool = pool
    dev.c.pool = pool.data_ptr()
    q = torch.from_numpy(rng.standard_normal((2, 64, 128)).astype(np.float32)).cuda()
    assert torch.equal(dev.attention(q, layer=layers - 1), near.attention(q))
    chosen = dev.select(q, 1, 0, 0, layer=layers - 1)
    assert torch.equal(chosen, near.select(q, 1, 0, 0))
    assert torch.equal(dev.attention(q, pages=chosen, layer=layers - 1), near.attention(q, pages=chosen))
    x = rows(rng, 70, 8, 128)
    k, v = layout(torch, x, "rows")
    dev.append(k, v, [0, 5, 70], layer=layers - 1, freq=freqs(128))
    store(small, x, [0, 5, 70], [0, 1], freq=freqs(128))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(pool[-1, pages - 6:].cpu().numpy(), small.pool[0])
    back, want = [torch.zeros_like(k) for _ in range(4)], Dev(nt, small, 64)
    dev.read(*back[:2], [0, 5, 70], layer=layers - 1)
    want.read(*back[2:], [0, 5, 70])
    assert torch.equal(back[0], back[2]) and torch.equal(back[1], back[3]) and back[0].any()
    src, dst = torch.tensor([pages - 6, pages - 1], dtype=torch.int32).cuda(), torch.tensor([0, pages - 7], dtype=torch.int32).cuda()
    nt.nt_kv8_copy_pages(dev.c, 2, src.data_ptr(), dst.data_ptr(), dev.stream())
    for s, d in zip(src.tolist(), dst.tolist()):
        assert torch.equal(pool[:, s], pool[:, d])
    assert not pool[0].any() and int(dev.error.cpu()[0]) == 0


# ------------------------------------------------------- graphs and streams --

def test_a_decode_loop_in_one_graph(nt):
    """extend, append with the rotation, selection and both forms of attention captured once and replayed: the state and the
    outputs are those of the model, step by step."""
    import torch
    rng = np.random.default_rng(25)
    hd, kv, heads, top = 64, 2, 8, 4
    ref = R.RefCache(1, kv, hd, 16, 40, 2, 16)
    ref.hold([0, 0])
    dev, freq = Dev(nt, ref, heads), freqs(hd)
    x = rows(rng, 100, kv, hd)
    ref.extend([0, 1], [70, 30])
    dev.extend([0, 1], [70, 30])
    store(ref, x, [0, 70, 100], [0, 1], freq=freq)
    dev.append(*layout(torch, x, "rows"), [0, 70, 100], freq=freq)
    dev.check()
    k, v, q = (torch.zeros(2, m, hd, device="cuda") for m in (kv, kv, heads))
    qr, out, sparse = (torch.zeros(2, heads, hd, device="cuda") for _ in range(3))
    one, chosen = torch.ones(2, dtype=torch.int32, device="cuda"), torch.zeros(2, kv, top, dtype=torch.int32, device="cuda")
    ws2 = torch.zeros_like(dev.ws)

    def step():
        s = dev.stream()
        nt.nt_kv8_extend(dev.c, 2, None, one.data_ptr(), dev.ws.data_ptr(), dev.wb, s)
        dev.append(k, v, None, freq=freq, q=q, q_out=qr)
        nt.nt_attention_kv8(dev.c, 0, heads, 2, None, None, 0, None, qr.data_ptr(), heads * hd, out.data_ptr(), heads * hd,
                            dev.ws.data_ptr(), dev.wb, s)
        nt.nt_kv8_select(dev.c, 0, heads, 2, None, None, qr.data_ptr(), heads * hd, top, 1, 1, chosen.data_ptr(), ws2.data_ptr(),
                         dev.wb, s)
        nt.nt_attention_kv8(dev.c, 0, heads, 2, None, None, top, chosen.data_ptr(), qr.data_ptr(), heads * hd,
                            sparse.data_ptr(), heads * hd, ws2.data_ptr(), dev.wb, s)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(40):
        y, qs = rows(rng, 2, kv, hd), rng.standard_normal((2, heads, hd)).astype(np.float32)
        k.copy_(torch.from_numpy(y[0]))
        v.copy_(torch.from_numpy(y[1]))
        q.copy_(torch.from_numpy(qs))
        graph.replay()
        ref.extend([0, 1], [1, 1])
        store(ref, y, [0, 1, 2], [0, 1], freq=freq)
        dev.check()
        rot, got, got2, places = qr.cpu().numpy(), out.cpu().numpy(), sparse.cpu().numpy(), chosen.cpu().numpy()
        for s in range(2):
            for g in range(kv):
                h = slice(4 * g, 4 * g + 4)
                np.testing.assert_array_equal(places[s, g], ref.select(0, s, g, rot[s, h], top, 1, 1))
                kk, vv = ref.kv(0, s, g)
                pos = np.concatenate([np.arange(j * 16, min(len(kk), j * 16 + 16)) for j in places[s, g] if j >= 0])
                for o, a, b in ((got, kk, vv), (got2, kk[pos], vv[pos])):
                    parts = R.attend(rot[s, h].astype(np.float64), a, b)
                    assert (np.abs(o[s, h] - parts[0]) <= bound(parts, len(a), np.abs(b).max())).all()


def test_the_same_call_gives_the_same_bits_on_any_stream_and_beside_others(nt):
    import torch
    rng = np.random.default_rng(26)
    lens = [3000, 1, 500, 1777, 64, 900]
    ref = R.RefCache(1, 4, 128, 64, sum(-(-x // 64) for x in lens), 6, 47)
    ref.randomize(rng)
    ref.hold(lens, rng)
    dev = Dev(nt, ref, 32)
    q = torch.from_numpy(rng.standard_normal((6, 32, 128)).astype(np.float32)).cuda()
    want = dev.attention(q)
    streams = [torch.cuda.Stream() for _ in range(3)]
    wss, outs = [torch.zeros_like(dev.ws) for _ in streams], [torch.zeros_like(want) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, ws, o in zip(streams, wss, outs):
            dev.attention(q, out=o, ws=ws, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_two_graphs_that_share_a_workspace(nt):
    """One after the other on a stream: neither keeps anything in the workspace for its next replay."""
    import torch
    rng = np.random.default_rng(27)
    ref = R.RefCache(1, 2, 128, 32, 220, 2, 110)
    ref.randomize(rng)
    ref.hold([3300, 3000], rng)
    dev = Dev(nt, ref, 16)
    q = torch.from_numpy(rng.standard_normal((2, 16, 128)).astype(np.float32)).cuda()
    want = dev.attention(q)
    pages = dev.select(q, 7, 1, 1)
    want_sparse = dev.attention(q, pages=pages)
    torch.cuda.synchronize()
    graphs, outs, lists = [], [torch.zeros_like(want) for _ in range(2)], torch.zeros_like(pages)
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if i == 0:
                dev.attention(q, out=outs[0])
            else:
                nt.nt_kv8_select(dev.c, 0, 16, 2, None, None, q.data_ptr(), 2048, 7, 1, 1, lists.data_ptr(), dev.ws.data_ptr(),
                                 dev.wb, dev.stream())
                dev.attention(q, pages=lists, out=outs[1])
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], (want, want_sparse)[i])


FIRST_CALLS = """
import numpy as np, torch
import kv8_ref as R
from test_gpu_kv8 import Dev, freqs, layout, rows
from quantized_decode_dequant_gb300 import nt
rng = np.random.default_rng(37)
i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")

class Fixed(Dev):
    def ints(self, x):          # lists made before the capture
        return None if x is None else x.data_ptr()

def fresh(hd, page_len, heads):
    r = np.random.default_rng(38)
    ref = R.RefCache(2, 2, hd, page_len, 40, 4, 18)
    ref.randomize(r)
    ref.hold([17 * page_len + 3, 40, 0, 0], r)
    dev = Fixed(nt, ref, heads)
    dev.l = [i32(0, 1), i32(2, 3), i32(1, 1), i32(1), i32(3, 4), i32(38, 39), i32(0)]
    dev.x = [torch.zeros(2, heads, hd, device="cuda") for _ in range(4)]
    dev.back = [torch.zeros(2, 2, hd, device="cuda") for _ in range(2)]
    dev.chosen = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    return dev

def calls(dev, k, v, q):
    src, dst, one, drop, a, b, live = dev.l
    hd, heads = dev.ref.hd, dev.heads
    nt.nt_kv8_fork(dev.c, 2, src.data_ptr(), dst.data_ptr(), None, dev.ws.data_ptr(), dev.wb, dev.stream())
    nt.nt_kv8_extend(dev.c, 2, dst.data_ptr(), one.data_ptr(), dev.ws.data_ptr(), dev.wb, dev.stream())
    nt.nt_kv8_append(dev.c, 1, 2, dst.data_ptr(), None, 2, "f16" if k.dtype == torch.float16 else "f32", k.data_ptr(), v.data_ptr(),
                     2 * hd, hd, freqs(hd), heads, q.data_ptr(), heads * hd, dev.x[0].data_ptr(), heads * hd, dev.stream())
    nt.nt_kv8_read(dev.c, 1, 2, dst.data_ptr(), None, 2, "f32", dev.back[0].data_ptr(), dev.back[1].data_ptr(), 2 * hd, hd, dev.stream())
    dev.attention(dev.x[0], dst, layer=1, out=dev.x[1])
    nt.nt_kv8_select(dev.c, 1, heads, 2, dst.data_ptr(), None, dev.x[0].data_ptr(), heads * hd, 3, 1, 1, dev.chosen.data_ptr(),
                     dev.ws.data_ptr(), dev.wb, dev.stream())
    dev.attention(dev.x[0], dst, pages=dev.chosen, layer=1, out=dev.x[2])
    nt.nt_kv8_free(dev.c, 1, drop.data_ptr(), None, dev.stream())
    nt.nt_kv8_copy_pages(dev.c, 2, a.data_ptr(), b.data_ptr(), dev.stream())
    nt.nt_kv8_compact(dev.c, dev.table.data_ptr(), dev.refs.data_ptr(), live.data_ptr(), dev.ws.data_ptr(), dev.wb, dev.stream())

shapes = [(64, 16, 2, False), (64, 128, 32, True), (128, 64, 8, False), (128, 128, 16, True), (128, 16, 6, False)]
for hd, page_len, heads, half in shapes:
    x = rows(rng, 2, 2, hd)
    k, v = layout(torch, x, "rows", half)
    q = torch.from_numpy(rng.standard_normal((2, heads, hd)).astype(np.float32)).cuda().to(k.dtype)
    dev, dev2, side = fresh(hd, page_len, heads), fresh(hd, page_len, heads), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):        # every operator for the first time in this process
        calls(dev, k, v, q)
    graph.replay()
    torch.cuda.synchronize()
    calls(dev2, k, v, q)
    torch.cuda.synchronize()
    for a, b in zip((dev.pool, dev.table, dev.len, dev.refs, dev.error, dev.chosen, *dev.x, *dev.back),
                    (dev2.pool, dev2.table, dev2.len, dev2.refs, dev2.error, dev2.chosen, *dev2.x, *dev2.back)):
        assert torch.equal(a, b)
    assert int(dev.error) == 0 and all(torch.isfinite(y).all() and y.any() for y in dev.x[:3])
print("captured")
"""


def test_first_calls_of_a_process_inside_a_capture(nt):
    """What a kernel is set up with at its first launch does not disturb a capture."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=os.path.dirname(here), env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
