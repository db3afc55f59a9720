"""CPU: the 4-bit cache's format on hand-made blocks, its plain model, and every refusal that the library makes on the host."""
import numpy as np
import pytest

import kv4_ref as R
from quantized_decode_dequant_gb300 import nt


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()
    return nt.lib()


# ------------------------------------------------------------------- format --

def test_scale_has_six_mantissa_bits_and_is_near_a_seventh_of_the_maximum():
    rng = np.random.default_rng(0)
    for std in (1e-4, 0.02, 1.0, 300.0):
        for _ in range(200):
            x = (rng.standard_normal(32) * std).astype(np.float32)
            d = R.scale_of(x)
            assert int(d.view(np.uint16)) & 15 == 0
            if d >= 2.0 ** -14:
                # f16's rounding is half of 2^-10, six bits' half of 2^-6 of the leading bit
                assert abs(float(d) - np.abs(x).max() / 7) <= (2.0 ** -7 + 2.0 ** -10) * float(d)


def test_hand_made_blocks():
    x = np.zeros(32, np.float32)
    x[:8] = [7, -7, 3, -3, 0.5, -0.5, 0.49, 1.5]             # scale exactly 1
    d = R.scale_of(x)
    assert float(d) == 1.0
    assert list(R.codes_of(x, d)[:8]) == [15, 1, 11, 5, 9, 7, 8, 10]
    assert float(R.scale_of(np.zeros(32))) == 0 and (R.codes_of(np.zeros(32), np.float16(0)) == 8).all()
    for v in (np.nan, np.inf, -np.inf, 6400.0, 3e38):
        x[5] = v
        assert np.isnan(R.scale_of(x)), v
    x[5] = 7 * 896.0
    assert float(R.scale_of(x)) == 896.0
    # the smallest scale is 2^-20; 6.5 / 7 of 2^-21 is 7.4 units of f16, rounds to 7, and has no bit left
    assert float(R.scale_of(np.full(32, 7 * 2.0 ** -20))) == 2.0 ** -20
    assert float(R.scale_of(np.full(32, 6.5 * 2.0 ** -21))) == 0


def test_values_and_the_products_on_the_way_are_exact_in_f16():
    """Every scale up to 896: 64 + q, 72 d and d (q - 8) are f16 numbers, so one fused multiply-add (64 + q) d - 72 d
    gives the value without rounding."""
    bits = np.arange(0, 0x6301, 16, dtype=np.uint16)
    d = bits.view(np.float16).astype(np.float64)
    for x in [72 * d] + [d * (q - 8) for q in range(16)]:
        np.testing.assert_array_equal(x.astype(np.float16).astype(np.float64), x)


def test_model_put_and_get():
    rng = np.random.default_rng(1)
    for hd in (64, 128):
        c = R.RefCache(2, 3, hd, 32, 4, 1, 2, fill=0xA5)
        seen = {}
        for at in rng.permutation(32):
            for g in range(3):
                k, v = rng.standard_normal((2, hd)).astype(np.float32)
                c.put(1, 2, g, at, k, v)
                seen[at, g] = [R.values(*R.quantize(k)), R.values(*R.quantize(v))]
        for (at, g), want in seen.items():
            for a, b in zip(c.get(1, 2, g, at), want):
                np.testing.assert_array_equal(a, b)
        assert (c.pool[0] == 0xA5).all() and (c.pool[1, [0, 1, 3]] == 0xA5).all()


# ----------------------------------------------------------------- refusals --

GOOD = dict(n_layers=2, n_kv_heads=2, head_dim=64, page_len=32, n_pages=10, max_seqs=4, max_pages=5, pool=1 << 20,
            table=1 << 12, len=1 << 13, refs=1 << 14, error=1 << 15)


def cache(**kw):
    return nt.make_kv4_cache(**dict(GOOD, **kw))


def status(f, *a):
    with pytest.raises(nt.NtError) as ei:
        f(*a)
    assert str(ei.value)
    return ei.value.status


def test_sizes(built):
    page, pool = nt.nt_kv4_pool_bytes(cache())
    assert page == 2 * 2 * 18 * 64 and pool == page * 10 * 2
    assert nt.nt_kv4_workspace_bytes(cache(), 8, 4) > 0
    for kw in (dict(n_layers=0), dict(n_layers=65536), dict(n_kv_heads=0), dict(n_kv_heads=65536), dict(page_len=0),
               dict(page_len=24), dict(page_len=272), dict(n_pages=0), dict(max_seqs=0), dict(max_seqs=65537),
               dict(max_pages=0), dict(max_pages=1 << 27, page_len=16)):
        assert status(nt.nt_kv4_pool_bytes, cache(**kw)) == nt.NT_E_INVAL, kw
    for hd in (0, 32, 96, 256):
        assert status(nt.nt_kv4_pool_bytes, cache(head_dim=hd)) == nt.NT_E_UNSUPPORTED
    assert status(nt.nt_kv4_workspace_bytes, cache(), 3, 4) == nt.NT_E_INVAL
    assert status(nt.nt_kv4_workspace_bytes, cache(), 8, -1) == nt.NT_E_INVAL
    assert status(nt.nt_kv4_workspace_bytes, cache(), 0, 1) == nt.NT_E_INVAL
    lib = nt.lib()
    assert lib.nt_kv4_pool_bytes(None, None, None) == nt.NT_E_INVAL
    assert lib.nt_kv4_workspace_bytes(cache(), 8, 4, None) == nt.NT_E_INVAL


A, B, WS, Q, O = 1 << 24, (1 << 24) + 4096, 1 << 25, 1 << 28, 1 << 29   # addresses that meet nothing (never dereferenced)


def calls(c=None, **kw):
    """Every operator with valid arguments but for those given."""
    c = c or cache()
    wb = nt.nt_kv4_workspace_bytes(cache(), 8, 4)
    a = dict(n=2, seq=A, count=B, ws=WS, wb=wb, layer=0, rows=3, type="f32", k=Q, v=O, rs=128, hs=64, heads=8, q=Q, qs=512,
             out=O, os=512, keep=None, table_out=A, refs_out=B, live=B + 4096)
    a.update(kw)
    g = lambda *names: [a[x] for x in names]   # noqa: E731
    return {
        "extend": lambda: nt.nt_kv4_extend(c, *g("n", "seq", "count", "ws", "wb")),
        "fork": lambda: nt.nt_kv4_fork(c, *g("n", "seq", "count", "keep", "ws", "wb")),
        "free": lambda: nt.nt_kv4_free(c, *g("n", "seq", "keep")),
        "copy_pages": lambda: nt.nt_kv4_copy_pages(c, *g("n", "seq", "count")),
        "compact": lambda: nt.nt_kv4_compact(c, *g("table_out", "refs_out", "live", "ws", "wb")),
        "append": lambda: nt.nt_kv4_append(c, *g("layer", "n", "seq", "count", "rows", "type", "k", "v", "rs", "hs")),
        "read": lambda: nt.nt_kv4_read(c, *g("layer", "n", "seq", "count", "rows", "type", "k", "v", "rs", "hs")),
        "attention": lambda: nt.nt_attention_kv4(c, *g("layer", "heads", "n", "seq", "q", "qs", "out", "os", "ws", "wb")),
    }


ALL = ["extend", "fork", "free", "copy_pages", "compact", "append", "read", "attention"]
ROWS, LISTS = ["append", "read"], ["extend", "fork", "free", "copy_pages"]


@pytest.mark.parametrize("ops,kw", [
    (["extend", "fork", "compact", "attention"], dict(ws=0)), (["extend", "fork", "compact", "attention"], dict(ws=WS + 8)),
    (["extend", "fork", "compact", "attention"], dict(wb=8)),
    (["extend", "fork", "compact", "attention"], dict(ws=GOOD["pool"])),
    (["extend", "fork", "compact", "attention"], dict(ws=GOOD["table"] + 16)),
    (["extend", "fork", "free", "copy_pages", "append", "read", "attention"], dict(n=-1)),
    (["extend", "fork", "free", "append"], dict(n=5)), (["copy_pages"], dict(n=11)),
    (["read", "attention"], dict(n=5, seq=None)), (["fork", "copy_pages"], dict(seq=None)),
    (["extend", "fork", "copy_pages"], dict(count=None)),
    (["extend", "fork", "free", "copy_pages", "append", "read", "attention"], dict(seq=A + 2)),
    (["extend", "fork", "copy_pages", "append", "read"], dict(count=B + 1)), (["fork", "free"], dict(keep=A + 3)),
    (["extend", "fork", "free", "copy_pages", "append", "read"], dict(seq=GOOD["len"])),
    (["extend", "fork"], dict(count=WS + 16)),
    (["append", "read", "attention"], dict(layer=-1)), (["append", "read", "attention"], dict(layer=2)),
    (ROWS, dict(rows=-1)), (ROWS, dict(type="q8_0")), (ROWS, dict(k=0)), (ROWS, dict(v=O + 8)), (ROWS, dict(rs=130)),
    (ROWS, dict(hs=-64)), (ROWS, dict(rs=132, type="f16")), (ROWS, dict(k=GOOD["pool"])), (ROWS, dict(rs=1 << 50)),
    (ROWS, dict(rows=(1 << 31) - 1, rs=0)), (ROWS, dict(rows=(1 << 30) + 16, rs=0)),
    (["read"], dict(v=Q)), (["read"], dict(rs=64)), (["read"], dict(hs=32)), (["read"], dict(hs=0)), (["read"], dict(rs=0)),
    (["read"], dict(v=Q + 256, rs=128)), (["read"], dict(seq=Q + 64)), (["read"], dict(count=O)),
    (["attention"], dict(heads=3)), (["attention"], dict(heads=0)), (["attention"], dict(qs=508)),
    (["attention"], dict(os=514)), (["attention"], dict(qs=510)), (["attention"], dict(q=0)), (["attention"], dict(q=Q + 4)),
    (["attention"], dict(out=0)), (["attention"], dict(out=Q + 2048)), (["attention"], dict(out=GOOD["pool"])),
    (["attention"], dict(out=WS)), (["attention"], dict(q=WS)), (["attention"], dict(n=65537)),
    (["attention"], dict(seq=O + 4)), (["attention"], dict(qs=1 << 50)),
    (["compact"], dict(table_out=0)), (["compact"], dict(refs_out=B + 2)), (["compact"], dict(live=0)),
    (["compact"], dict(table_out=GOOD["table"] + 4)), (["compact"], dict(refs_out=GOOD["refs"] + 4)),
    (["compact"], dict(refs_out=GOOD["table"])), (["compact"], dict(live=GOOD["len"])), (["compact"], dict(live=A)),
    (["compact"], dict(table_out=B)), (["compact"], dict(refs_out=WS)),
])
def test_refused_arguments(built, ops, kw):
    for op in ops:
        assert status(calls(**kw)[op]) == nt.NT_E_INVAL, (op, kw)


@pytest.mark.parametrize("kw,want", [
    (dict(pool=0), nt.NT_E_INVAL), (dict(pool=(1 << 20) + 8), nt.NT_E_INVAL), (dict(table=0), nt.NT_E_INVAL),
    (dict(len=2), nt.NT_E_INVAL), (dict(refs=0), nt.NT_E_INVAL), (dict(error=0), nt.NT_E_INVAL),
    (dict(n_pages=0), nt.NT_E_INVAL), (dict(page_len=8), nt.NT_E_INVAL), (dict(head_dim=96), nt.NT_E_UNSUPPORTED)])
def test_refused_caches(built, kw, want):
    for op in ALL:
        assert status(calls(cache(**kw))[op]) == want, (op, kw)


def test_unsupported_groups(built):
    assert status(calls(heads=6)["attention"]) == nt.NT_E_UNSUPPORTED
    assert status(calls(heads=64)["attention"]) == nt.NT_E_UNSUPPORTED


def test_empty_calls_launch_nothing(built):
    for op in LISTS + ROWS + ["attention"]:
        calls(n=0)[op]()
    for op in ROWS:
        calls(rows=0)[op]()


def test_rows_that_interleave_are_not_taken_for_overlapping(built):
    """K and V next to each other in one projection's rows: their ranges overlap, their elements do not.  The call gets as
    far as a later check."""
    lib = nt.lib()
    with pytest.raises(nt.NtError) as ei:
        nt.nt_kv4_read(cache(), 0, 2, A, Q + 4, 3, "f32", Q, Q + 512, 256, 64)   # dev_begin inside the output
    assert "another buffer" in str(ei.value)
    assert lib.nt_last_error()


def _meet(begin_k, begin_v, rows, kv, hd, es, rs, hs):
    """Whether two (row, kv head) vectors of K and V, or of one of them, share bytes: every pair of them."""
    at = np.add.outer(np.arange(rows) * rs, np.arange(kv) * hs).reshape(-1) * es
    at = np.sort(np.concatenate([begin_k + at, begin_v + at]))
    return bool((np.diff(at) < hd * es).any())


def test_read_refuses_exactly_the_outputs_that_overlap(built):
    """Strides of every kind, small ones and few rows among them (a row stride plays no part with a single row)."""
    rng = np.random.default_rng(3)
    seen = [0, 0]
    for _ in range(4000):
        half, rows, kv = bool(rng.integers(2)), int(rng.choice([1, 1, 2, 3, 5])), int(rng.choice([1, 2, 3]))
        es = 2 if half else 4
        unit = 16 // es
        rs, hs = (int(rng.choice([0, unit, 3 * unit, 5 * unit, 40, 64, 72, 64 * kv, 128 * kv, 64 * kv + unit, 64 * rows])) for _ in "rh")
        apart = int(rng.choice([16, 80, 64 * es, 64 * es * kv, 64 * es * kv * rows, 128 * es, 1 << 16, 64 * es - 16])) * int(rng.choice([-1, 1]))
        want = _meet(Q, Q + apart, rows, kv, 64, es, rs, hs)
        seen[want] += 1
        c = cache(n_kv_heads=kv)
        # a list inside the outputs is refused after their own overlap: either message, no launch
        with pytest.raises(nt.NtError) as ei:
            nt.nt_kv4_read(c, 0, 1, A, Q, rows, "f16" if half else "f32", Q, Q + apart, rs, hs)
        assert ("rows of the outputs" in str(ei.value)) == want, (half, rows, kv, rs, hs, apart)
    assert min(seen) > 500


def test_rows_calls_whose_grid_would_pass_2_to_the_31(built):
    """65535 kv heads: 65535 units of 16 rows and two an entry are one too many."""
    rows = (65535 - 5) * 16
    for op in ROWS:
        with pytest.raises(nt.NtError) as ei:
            calls(cache(n_kv_heads=65535), rows=rows, rs=64, hs=64 * rows, type="f32")[op]()
        assert ei.value.status == nt.NT_E_INVAL and "2^32 - 2^17" in str(ei.value)
