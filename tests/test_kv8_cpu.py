"""CPU: the 8-bit cache's format on hand-made values, its plain model, and every refusal that the library makes on the host."""
import numpy as np
import pytest

import kv8_ref as R
from quantized_decode_dequant_gb300 import nt


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()
    return nt.lib()


# ------------------------------------------------------------------- format --

def test_codes_of_hand_made_numbers():
    assert R.NUMBER[0x7E] == 448 and R.NUMBER[0x08] == 2.0 ** -6 and R.NUMBER[1] == 2.0 ** -9 and R.NUMBER[0xB8] == -1
    x = [0, 1, -1, 448, -448, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 1.0625, 1.1875, 17, 19, np.nan, 447, 2.0 ** -10 + 1e-9]
    want = [0, 0x38, 0xB8, 0x7E, 0xFE, 1, 0, 2, 0x38, 0x3A, 0x58, 0x5A, 0x7F, 0x7E, 1]
    assert list(R.code(x)) == want
    np.testing.assert_array_equal(R.code(R.NUMBER[np.arange(127)]), np.arange(127))


def test_codes_are_those_of_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * np.exp(rng.standard_normal(20000) * 3)).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(R.code(x), want)


def test_exponents():
    for top, e in ((448, 0), (448.0001, 1), (224, -1), (1.0, -8), (7 / 8, -9), (0.875001, -8), (0, -100), (1e-40, -100),
                   (R.MOST, 100), (np.nan, -100), (np.inf, -100), (R.MOST * 1.001, -100)):
        assert R.exponent(np.array([top, 0.0])) == e, top


def test_appending_in_pieces_is_appending_at_once_where_the_first_piece_has_the_largest_value():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 30, 2, 64)).astype(np.float32)
    k[0, :, 3], v[0, :, 5] = 9.0, -8.0
    k[16, :, 3], v[16, :, 5] = 9.0, -8.0
    pools = []
    for cuts in ((0, 30), (0, 1, 2, 17, 29, 30)):
        c = R.RefCache(1, 2, 64, 16, 4, 1, 4, fill=0xA5)
        c.hold([30])
        for a, b in zip(cuts, cuts[1:]):
            c.len[0] = b
            c.append(0, 0, k[a:b], v[a:b])
        pools.append(c.pool.copy())
    np.testing.assert_array_equal(*pools)


def test_a_growing_scale_keeps_the_values_within_its_steps_and_the_bounds_true():
    rng = np.random.default_rng(2)
    c = R.RefCache(1, 1, 64, 32, 1, 1, 1)
    c.hold([32])
    rows = [(rng.standard_normal((1, 1, 64)) * 2.0 ** (i / 3)).astype(np.float32) for i in range(32)]
    for i, x in enumerate(rows):
        c.len[0] = i + 1
        c.append(0, 0, x, -x)
    k, v = c.kv(0, 0, 0)
    row = c.pool[0, 0]
    e = c.page_kv(row, 0)[2][0]
    for i, x in enumerate(rows):
        # a code rounded twice: half a step of its size (2^-4), and half of the smallest step 2^(e - 9) for each rounding
        np.testing.assert_allclose(k[i], x[0, 0], rtol=2.0 ** -4, atol=2 * 2.0 ** (e - 10) + 1e-30)
        np.testing.assert_allclose(v[i], -x[0, 0], rtol=2.0 ** -4, atol=2 * 2.0 ** (e - 10) + 1e-30)
    lo, hi = c.bounds(row, 0) * 2.0 ** (e + 2)
    assert (lo <= k.min(0)).all() and (hi >= k.max(0)).all()


def test_selection_by_hand():
    c = R.RefCache(1, 1, 64, 16, 8, 1, 8)
    c.hold([16 * 7 + 3])
    x = np.zeros((16 * 7 + 3, 1, 64), np.float32)
    for j, peak in enumerate([1, 5, 2, 5, 3, 0.1, 4, 0.2]):
        x[16 * j, 0, 0] = peak
    c.append(0, 0, x, x)
    q = np.zeros((2, 64))
    q[0, 0], q[1, 0] = 1.0, 0.5
    assert list(c.select(0, 0, 0, q, 3, 0, 0)) == [1, 3, 6]
    assert list(c.select(0, 0, 0, q, 3, 1, 1)) == [0, 1, 7]         # the lower of two equal ones
    assert list(c.select(0, 0, 0, -q, 2, 0, 0)) == [0, 1]           # nothing below zero anywhere: every bound is 0
    assert list(c.select(0, 0, 0, q, 10, 0, 0)) == list(range(8)) + [-1, -1]


# ----------------------------------------------------------------- refusals --

GOOD = dict(n_layers=2, n_kv_heads=2, head_dim=64, page_len=32, n_pages=10, max_seqs=4, max_pages=5, pool=1 << 20,
            table=1 << 12, len=1 << 13, refs=1 << 14, error=1 << 15)


def cache(**kw):
    return nt.make_kv8_cache(**dict(GOOD, **kw))


def status(f, *a):
    with pytest.raises(nt.NtError) as ei:
        f(*a)
    assert str(ei.value)
    return ei.value.status


def test_sizes(built):
    page, pool = nt.nt_kv8_pool_bytes(cache())
    assert page == 2 * (2 * 32 * 64 + 16 + 128) and pool == page * 10 * 2
    assert nt.nt_kv8_workspace_bytes(cache(), 8, 4) > 0
    for kw in (dict(n_layers=0), dict(n_layers=65536), dict(n_kv_heads=0), dict(n_kv_heads=65536), dict(page_len=0),
               dict(page_len=-16), dict(n_pages=0), dict(max_seqs=0), dict(max_seqs=65537), dict(max_pages=0),
               dict(max_pages=1 << 27, page_len=16)):
        assert status(nt.nt_kv8_pool_bytes, cache(**kw)) == nt.NT_E_INVAL, kw
    for kw in [dict(head_dim=x) for x in (0, 32, 96, 256)] + [dict(page_len=x) for x in (8, 24, 48, 256)]:
        assert status(nt.nt_kv8_pool_bytes, cache(**kw)) == nt.NT_E_UNSUPPORTED
    assert status(nt.nt_kv8_workspace_bytes, cache(), 3, 4) == nt.NT_E_INVAL
    assert status(nt.nt_kv8_workspace_bytes, cache(), 8, -1) == nt.NT_E_INVAL
    assert status(nt.nt_kv8_workspace_bytes, cache(), 0, 1) == nt.NT_E_INVAL
    lib = nt.lib()
    assert lib.nt_kv8_pool_bytes(None, None, None) == nt.NT_E_INVAL
    assert lib.nt_kv8_workspace_bytes(cache(), 8, 4, None) == nt.NT_E_INVAL


def test_workspace_of_any_number_of_sequences(built):
    """No call takes more than 65536 sequences, so more need no more; the largest sizes do not wrap round."""
    for kw in (dict(), dict(n_kv_heads=256, page_len=16, max_pages=(1 << 27) - 16), dict(n_kv_heads=65535, page_len=16, max_pages=(1 << 27) - 16)):
        c = cache(**kw)
        most = nt.nt_kv8_workspace_bytes(c, c.n_kv_heads, 65536)
        assert most >= 65536 * c.n_kv_heads * c.max_pages * 4
        for n in (65537, 1 << 20, 1 << 28, (1 << 31) - 1):
            assert nt.nt_kv8_workspace_bytes(c, c.n_kv_heads, n) == most
        assert nt.nt_kv8_workspace_bytes(c, c.n_kv_heads, 1000) < most


A, B, CTX, WS, Q, O, K, V = (1 << 24, (1 << 24) + 4096, (1 << 24) + 8192, 1 << 25, 1 << 28, 1 << 29, 1 << 30, 1 << 31)
FREQ = [1.0 / (i + 1) for i in range(32)]


def calls(c=None, **kw):
    """Every operator with valid arguments but for those given (addresses that meet nothing, never dereferenced)."""
    c = c or cache()
    wb = nt.nt_kv8_workspace_bytes(cache(), 8, 4)
    a = dict(n=2, seq=A, count=B, ws=WS, wb=wb, layer=0, rows=3, type="f32", k=K, v=V, rs=128, hs=64, heads=8, q=Q, qs=512,
             out=O, os=512, keep=None, table_out=A, refs_out=B, live=B + 4096, freq=FREQ, ctx=CTX, top=4, first=1, last=1,
             chosen=CTX + 4096, sel=4, pages=CTX + 4096)
    a.update(kw)
    g = lambda *names: [a[x] for x in names]   # noqa: E731
    return {
        "extend": lambda: nt.nt_kv8_extend(c, *g("n", "seq", "count", "ws", "wb")),
        "fork": lambda: nt.nt_kv8_fork(c, *g("n", "seq", "count", "keep", "ws", "wb")),
        "free": lambda: nt.nt_kv8_free(c, *g("n", "seq", "keep")),
        "copy_pages": lambda: nt.nt_kv8_copy_pages(c, *g("n", "seq", "count")),
        "compact": lambda: nt.nt_kv8_compact(c, *g("table_out", "refs_out", "live", "ws", "wb")),
        "append": lambda: nt.nt_kv8_append(c, *g("layer", "n", "seq", "count", "rows", "type", "k", "v", "rs", "hs", "freq",
                                                 "heads", "q", "qs", "out", "os")),
        "read": lambda: nt.nt_kv8_read(c, *g("layer", "n", "seq", "count", "rows", "type", "k", "v", "rs", "hs")),
        "select": lambda: nt.nt_kv8_select(c, *g("layer", "heads", "n", "seq", "ctx", "q", "qs", "top", "first", "last",
                                                 "chosen", "ws", "wb")),
        "attention": lambda: nt.nt_attention_kv8(c, *g("layer", "heads", "n", "seq", "ctx", "sel", "pages", "q", "qs", "out",
                                                       "os", "ws", "wb")),
    }


ALL = ["extend", "fork", "free", "copy_pages", "compact", "append", "read", "select", "attention"]
ROWS, LISTS, ATT = ["append", "read"], ["extend", "fork", "free", "copy_pages"], ["select", "attention"]


@pytest.mark.parametrize("ops,kw", [
    (["extend", "fork", "compact"] + ATT, dict(ws=0)), (["extend", "fork", "compact"] + ATT, dict(ws=WS + 8)),
    (["extend", "fork", "compact"] + ATT, dict(wb=8)), (["extend", "fork", "compact"] + ATT, dict(ws=GOOD["pool"])),
    (["extend", "fork", "compact"] + ATT, dict(ws=GOOD["table"] + 16)),
    (LISTS + ROWS + ATT, dict(n=-1)), (["extend", "fork", "free", "append"], dict(n=5)), (["copy_pages"], dict(n=11)),
    (["read"] + ATT, dict(n=5, seq=None)), (["fork", "copy_pages"], dict(seq=None)),
    (["extend", "fork", "copy_pages"], dict(count=None)), (LISTS + ROWS + ATT, dict(seq=A + 2)),
    (["extend", "fork", "copy_pages", "append", "read"], dict(count=B + 1)), (["fork", "free"], dict(keep=A + 3)),
    (LISTS + ROWS, dict(seq=GOOD["len"])), (["extend", "fork"], dict(count=WS + 16)),
    (ROWS + ATT, dict(layer=-1)), (ROWS + ATT, dict(layer=2)),
    (ROWS, dict(rows=-1)), (ROWS, dict(type="q8_0")), (ROWS, dict(k=0)), (ROWS, dict(v=V + 8)), (ROWS, dict(rs=130)),
    (ROWS, dict(hs=-64)), (ROWS, dict(rs=132, type="f16")), (ROWS, dict(k=GOOD["pool"])), (ROWS, dict(rs=1 << 50)),
    (ROWS, dict(rows=(1 << 31) - 1, rs=0)),
    (["read"], dict(v=K)), (["read"], dict(rs=64)), (["read"], dict(hs=32)), (["read"], dict(hs=0)), (["read"], dict(rs=0)),
    (["read"], dict(v=K + 256, rs=128)), (["read"], dict(seq=K + 64)), (["read"], dict(count=V)),
    (["append"], dict(freq=None)), (["append"], dict(freq=FREQ[:-1] + [float("nan")])),
    (["append"], dict(freq=FREQ[:-1] + [float("inf")])), (["append"], dict(freq=FREQ[:-1] + [-1.1e6])),
    (["append"], dict(q=0)), (["append"], dict(q=Q + 8)), (["append"], dict(out=0)), (["append"], dict(out=O + 4)),
    (["append"], dict(heads=0)), (["append"], dict(heads=65536, qs=1 << 23, os=1 << 23)), (["append"], dict(qs=508)),
    (["append"], dict(os=508)), (["append"], dict(os=514)), (["append"], dict(qs=514)), (["append"], dict(qs=516, type="f16")),
    (["append"], dict(out=Q + 1024)), (["append"], dict(out=Q, os=516)), (["append"], dict(out=Q, type="f16")),
    (["append"], dict(out=K)), (["append"], dict(out=V + 64)), (["append"], dict(out=GOOD["pool"])),
    (["append"], dict(out=GOOD["len"])), (["append"], dict(q=GOOD["pool"])), (["append"], dict(seq=O)),
    (["append"], dict(count=O + 4)), (["append"], dict(qs=1 << 50)),
    (ATT, dict(heads=3)), (ATT, dict(heads=0)), (ATT, dict(qs=508)), (["attention"], dict(os=514)), (ATT, dict(qs=510)),
    (ATT, dict(q=0)), (ATT, dict(q=Q + 4)), (["attention"], dict(out=0)), (["attention"], dict(out=Q + 2048)),
    (["attention"], dict(out=GOOD["pool"])), (["attention"], dict(out=WS)), (ATT, dict(q=WS)), (ATT, dict(n=65537)),
    (["attention"], dict(seq=O + 4)), (["attention"], dict(ctx=O + 4)), (["attention"], dict(pages=O + 8)), (ATT, dict(qs=1 << 50)),
    (ATT, dict(ctx=CTX + 2)), (["attention"], dict(pages=None)), (["attention"], dict(sel=0)), (["attention"], dict(sel=-1)),
    (["attention"], dict(sel=65537)), (["attention"], dict(pages=WS)), (["attention"], dict(pages=CTX + 1)),
    (["select"], dict(top=0)), (["select"], dict(top=65537)), (["select"], dict(first=-1)), (["select"], dict(last=-1)),
    (["select"], dict(first=3, last=2)), (["select"], dict(chosen=0)), (["select"], dict(chosen=CTX + 2)),
    (["select"], dict(chosen=WS)), (["select"], dict(chosen=Q)), (["select"], dict(chosen=CTX)), (["select"], dict(chosen=A)),
    (["select"], dict(chosen=GOOD["refs"])),
    (["compact"], dict(table_out=0)), (["compact"], dict(refs_out=B + 2)), (["compact"], dict(live=0)),
    (["compact"], dict(table_out=GOOD["table"] + 4)), (["compact"], dict(refs_out=GOOD["table"])),
    (["compact"], dict(live=A)), (["compact"], dict(table_out=B)), (["compact"], dict(refs_out=WS)),
])
def test_refused_arguments(built, ops, kw):
    for op in ops:
        assert status(calls(**kw)[op]) == nt.NT_E_INVAL, (op, kw)


@pytest.mark.parametrize("kw,want", [
    (dict(pool=0), nt.NT_E_INVAL), (dict(pool=(1 << 20) + 8), nt.NT_E_INVAL), (dict(table=0), nt.NT_E_INVAL),
    (dict(len=2), nt.NT_E_INVAL), (dict(refs=0), nt.NT_E_INVAL), (dict(error=0), nt.NT_E_INVAL),
    (dict(n_pages=0), nt.NT_E_INVAL), (dict(page_len=0), nt.NT_E_INVAL), (dict(page_len=48), nt.NT_E_UNSUPPORTED),
    (dict(head_dim=96), nt.NT_E_UNSUPPORTED)])
def test_refused_caches(built, kw, want):
    for op in ALL:
        if "head_dim" in kw and op == "append":
            continue                                         # the binding asks for the frequencies of that head_dim first
        assert status(calls(cache(**kw))[op], ) == want, (op, kw)


def test_too_many_query_heads(built):
    for op in ATT:
        assert status(calls(heads=34, qs=34 * 64, os=34 * 64)[op]) == nt.NT_E_UNSUPPORTED


def test_empty_calls_launch_nothing(built):
    for op in LISTS + ROWS + ATT:
        calls(n=0)[op]()
    for op in ROWS:
        calls(rows=0)[op]()


def test_the_binding_refuses_another_number_of_frequencies(built):
    with pytest.raises(ValueError):
        calls(freq=FREQ[:-1])["append"]()
