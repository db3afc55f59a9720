"""Cases of the paged 8-bit K/V cache operators: append with the position rotation, attention, and attention over the
pages that a cheap score selects.

Each case names one pass through an operator.  With ``own`` false ``run`` computes the plain form (elementary torch
operations in fp32, in fp64 where 32 bits lose what matters); with ``own`` true it makes the library calls.  Both read
and write the same page pool.

The cache.  A page holds ``page_len`` (16, 32, 64 or 128) positions of one layer:
  for every kv head  K codes [page_len / 8][hd / 16][8][16], V codes [page_len / 16][hd][16]   (e4m3 bytes)
  then for every kv head  K exponent, V exponent (int8), 14 bytes unused, lo int8 [hd], hi int8 [hd]
K code (t / 8, d / 16, t % 8, d % 16) and V code (t / 16, d, t % 16) are dimension d of position t; a value is
code * 2^exponent, one exponent for the K and one for the V of a page and kv head.  lo and hi bound the page's keys per
dimension, in units of 2^(K exponent + 2).

Scale: the smallest exponent from -100 on that brings the page's largest magnitude to at most 448, and never smaller
than the page had while it fills up: where rows are added that need a larger one, the codes held are rounded again.
"""
import math

import torch

own = False

DEV = "cuda"
EMIN, EMAX = -100, 100
THETA = 500000.0


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the tiny two-layer model's decode step: the latency of one call
        dict(name="append 1 token", op="append", heads=8, kv=2, hd=64, page_len=16, n=1, rows=1, kept=37, half=False),
        # one new token of each of 16 sequences, in the middle of their pages, with the queries of 64 heads
        dict(name="append 16 tokens", op="append", heads=64, kv=8, hd=128, page_len=64, n=16, rows=1, kept=700, half=False),
        # five drafted tokens of each of 56 sequences, far into their contexts
        dict(name="append 56 drafts of 5", op="append", heads=32, kv=8, hd=128, page_len=32, n=56, rows=5, kept=2009,
             half=False),
        # two prompts whose f16 keys and values come as [kv head][position][dimension]; their queries go elsewhere
        dict(name="append 2 x 20k f16", op="append", heads=0, kv=8, hd=128, page_len=64, n=2, rows=20011, kept=0, half=True),
        # the decode step of the tiny model
        dict(name="attention 1 short", op="attention", heads=8, kv=2, hd=64, page_len=16, n=1, longest=37, ragged=False,
             drafts=1),
        # one 70B-shaped layer at the flagship decode step's context
        dict(name="attention 1 x 4k", op="attention", heads=64, kv=8, hd=128, page_len=64, n=1, longest=4161, ragged=False,
             drafts=1),
        # the same layer over a very long document
        dict(name="attention 1 x 131k", op="attention", heads=64, kv=8, hd=128, page_len=64, n=1, longest=131077,
             ragged=False, drafts=1),
        # 8B-shaped layer, many samples of different lengths, one of them just begun (empty)
        dict(name="attention 56 ragged", op="attention", heads=32, kv=8, hd=128, page_len=32, n=56, longest=9001, ragged=True,
             drafts=1),
        # a speculative draft of 5 tokens is verified for 4 sequences: every token sees the positions up to its own
        dict(name="attention 4 x 5 drafts", op="attention", heads=32, kv=8, hd=128, page_len=64, n=4, longest=6007,
             ragged=True, drafts=5),
        # fewer pages than would be selected: everything is attended
        dict(name="sparse 1 short", op="sparse", heads=8, kv=2, hd=64, page_len=16, n=1, longest=101, ragged=False, top=8,
             first=1, last=2),
        # a very long document, of which each token looks at 64 pages of 64 positions
        dict(name="sparse 1 x 131k", op="sparse", heads=64, kv=8, hd=128, page_len=64, n=1, longest=131077, ragged=False,
             top=64, first=1, last=2),
        # 24 long conversations, 32 pages each
        dict(name="sparse 24 x 30k", op="sparse", heads=32, kv=8, hd=128, page_len=32, n=24, longest=30011, ragged=True,
             top=96, first=1, last=4),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "sparse"])
    hd, kv, page_len = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32, 64, 128])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op == "append":
        n = _spread(rng, 1, 64)
        rows = _spread(rng, 1, max(2, 16000 // n))
        return dict(op=op, heads=kv * group if rows * n < 1000 else 0, kv=kv, hd=hd, page_len=page_len, n=n, rows=rows,
                    kept=rng.choice([0, _spread(rng, 1, 3000)]), half=rng.random() < 0.4)
    row = 2 * kv * hd                                # cache bytes of one position
    n = _spread(rng, 1, 64)
    most = min(131072, 200_000_000 // (row * n))
    if op == "attention":
        drafts = rng.choice([1, 1, 1, 2, 5])
        return dict(op=op, heads=kv * group, kv=kv, hd=hd, page_len=page_len, n=n,
                    longest=max(drafts, _spread(rng, 1, max(1, most // drafts))), ragged=rng.random() < 0.6, drafts=drafts)
    top, first, last = _spread(rng, 4, 128), rng.choice([0, 1]), rng.choice([1, 2])
    return dict(op=op, heads=kv * group, kv=kv, hd=hd, page_len=page_len, n=n, longest=_spread(rng, 1, most),
                ragged=rng.random() < 0.6, top=top, first=first, last=last)


def _lens(case):
    """Lengths of the sequences: the longest first; ragged ones spread evenly, the fourth of many empty."""
    n, longest = case["n"], case["longest"]
    if not case["ragged"]:
        return [longest] * n
    least = case.get("drafts", 1)
    return [0 if i == 3 and n > 4 and least == 1 else least + int((longest - least) * (1 - (i * 0.6180339887) % 1))
            for i in range(n)]


def _entries(case):
    """(sequence, positions seen) of every query: the last drafts of each sequence, the first of them first."""
    d = case.get("drafts", 1)
    return [(i, x - d + 1 + j) if x else (i, 0) for i, x in enumerate(_lens(case)) for j in range(d)]


def _rows(case):
    """New rows of each sequence: the last one takes one fewer where there are several."""
    return [case["rows"] - (1 if i and i == case["n"] - 1 and case["rows"] > 1 else 0) for i in range(case["n"])]


def _back(case):
    """Older positions in the page that the new rows begin in: their codes may be rounded again."""
    return case["kept"] % case["page_len"]


def work(case):
    kv, hd, p = case["kv"], case["hd"], case["page_len"]
    if case["op"] == "append":
        rows, es = sum(_rows(case)), 2 if case["half"] else 4
        both = rows + case["n"] * _back(case)
        pages = sum(-(-(_back(case) + r) // p) for r in _rows(case))
        q = rows * case["heads"] * hd
        return dict(bytes=2 * rows * kv * hd * (es + 1) + 2 * both * kv * hd * (es + 1) + pages * kv * (2 * hd + 2) + q * (es + 4),
                    flops=3 * (rows * kv * hd + q))
    if case["op"] == "attention":
        d = case["drafts"]
        total, seen = sum(_lens(case)), sum(c for _, c in _entries(case))
        pages = sum(-(-x // p) for x in _lens(case))
        return dict(bytes=total * 2 * kv * hd + pages * (2 * kv + 4) + 2 * case["n"] * d * case["heads"] * hd * 4,
                    flops=4 * seen * case["heads"] * hd)
    pages = sum(-(-x // p) for x in _lens(case))
    read = seen = 0
    for x in _lens(case):
        m = min(case["top"], -(-x // p))
        seen += m * p - (-x % p)
    read = seen * 2 * kv * hd + pages * (kv * (2 * hd + 1) + 4)
    return dict(bytes=read + 2 * case["n"] * case["heads"] * hd * 4 + case["n"] * kv * case["top"] * 4,
                flops=4 * seen * case["heads"] * hd + 2 * pages * case["heads"] * hd)


# ----------------------------------------------------- pages, in torch --

def _page_bytes(case):
    return case["kv"] * (2 * case["page_len"] * case["hd"] + 2 * case["hd"] + 16)


def _exponent(top):
    """Smallest exponent from EMIN on with top <= 448 * 2^exponent; int32."""
    m, x = torch.frexp(top)
    return torch.where(top > 0, x - 9 + (m > 0.875).int(), torch.full_like(x, EMIN)).clamp(min=EMIN).int()


def _held(x):
    """Whether fp32 values can be held (the others are stored as NaN)."""
    return x.abs() <= 448 * 2.0 ** EMAX


def _codes(x, e):
    """Codes of fp32 values for exponents e (both of one shape): e4m3, rounded to nearest even."""
    y = (x.double() * torch.exp2(-e.double())).float()
    return torch.where(_held(x), y, torch.full_like(y, float("nan"))).to(torch.float8_e4m3fn)


def _parts(pool, case):
    """Views of pages [..., bytes]: K codes [..., kv, p/8, hd/16, 8, 16], V codes [..., kv, p/16, hd, 16] (e4m3),
    exponents [..., kv, 16] and bounds [..., kv, 2, hd] (int8)."""
    kv, hd, p = case["kv"], case["hd"], case["page_len"]
    codes = pool[..., :kv * 2 * p * hd].unflatten(-1, (kv, 2, p * hd)).view(torch.float8_e4m3fn)
    meta = pool[..., kv * 2 * p * hd:].unflatten(-1, (kv, 16 + 2 * hd)).view(torch.int8)
    return (codes[..., 0, :].unflatten(-1, (p // 8, hd // 16, 8, 16)), codes[..., 1, :].unflatten(-1, (p // 16, hd, 16)),
            meta[..., :16], meta[..., 16:].unflatten(-1, (2, hd)))


def _values(pool, case):
    """K and V of pages [..., bytes] as fp32 [..., kv, positions, hd]."""
    k, v, e, _ = _parts(pool, case)
    k = k.float().transpose(-3, -2).flatten(-2).flatten(-3, -2)
    v = v.float().transpose(-2, -1).flatten(-3, -2)
    scale = torch.exp2(e[..., :2].float())
    return k * scale[..., 0, None, None], v * scale[..., 1, None, None]


def _bounds(k):
    """lo and hi of keys in units of their exponent [..., positions, hd]; a NaN counts as unbounded."""
    nan = torch.isnan(k).any(-2)
    lo, hi = torch.floor(k.amin(-2) / 4), torch.ceil(k.amax(-2) / 4)
    return torch.where(nan, torch.full_like(lo, -127), lo), torch.where(nan, torch.full_like(hi, 127), hi)


def _random_pool(case, pages, gen):
    """Pages of K and V as a prompt leaves them: K with a few strong channels and a direction of its own for each page."""
    kv, hd, p = case["kv"], case["hd"], case["page_len"]
    out = torch.zeros(pages, _page_bytes(case), dtype=torch.uint8, device=DEV)
    chans = torch.where(torch.rand(hd, device=DEV, generator=gen) < 0.06, 4.0, 0.8)
    step = max(1, (1 << 26) // (kv * p * hd))
    for a in range(0, pages, step):
        part = out[a:a + step]
        shape = (part.shape[0], kv, p, hd)
        k = torch.randn(shape, device=DEV, generator=gen) * chans
        k += 0.5 * torch.randn(shape[:2] + (1, hd), device=DEV, generator=gen)
        v = torch.randn(shape, device=DEV, generator=gen)
        kc, vc, e, b = _parts(part, case)
        ke, ve = _exponent(k.abs().amax((-1, -2))), _exponent(v.abs().amax((-1, -2)))
        kq, vq = _codes(k, ke[..., None, None].expand(shape)), _codes(v, ve[..., None, None].expand(shape))
        kc.copy_(kq.unflatten(-1, (hd // 16, 16)).unflatten(-3, (p // 8, 8)).transpose(-3, -2))
        vc.copy_(vq.unflatten(-2, (p // 16, 16)).transpose(-2, -1))
        e[..., 0], e[..., 1] = ke.to(torch.int8), ve.to(torch.int8)
        lo, hi = _bounds(kq.float())
        b[..., 0, :], b[..., 1, :] = lo.to(torch.int8), hi.to(torch.int8)
    return out


# ---------------------------------------------------------------- prepare --

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _frequencies(hd):
    """Radians per position of each pair of dimensions."""
    return [THETA ** (-2.0 * i / hd) for i in range(hd // 2)]


def _tables(lens, page_len, spare, host):
    """Page tables of sequences whose pages lie anywhere in the pool, the number of pages and the reference counts."""
    held = [-(-x // page_len) for x in lens]
    pages = sum(held) + spare
    order = torch.randperm(pages, generator=host).int()
    table = torch.full((len(lens), max(1, max(held))), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(held):
        table[i, :m] = order[at:at + m]
        at += m
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[order[:at].long()] = 1
    return table.to(DEV), refs.to(DEV), pages


def prepare(case, seed):
    gen, host = torch.Generator(DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
    op, kv, hd, page_len = case["op"], case["kv"], case["hd"], case["page_len"]
    st = dict(case=case)
    if op == "append":
        rows = _rows(case)
        lens = [case["kept"] + r for r in rows]             # the rows' pages are there already
        st["table"], st["refs"], pages = _tables(lens, page_len, 2, host)
        st["pool"], st["len"] = _random_pool(case, pages, gen), _ints(lens)
        st["rows"], st["read"] = sum(rows), sum(rows) + case["n"] * _back(case)
        st["begin"] = torch.nn.functional.pad(_ints(rows).cumsum(0).int(), (1, 0))
        st["begin_read"] = torch.nn.functional.pad(_ints([r + _back(case) for r in rows]).cumsum(0).int(), (1, 0))
        st["freq"] = _frequencies(hd)
        x = torch.randn(2, kv, sum(rows), hd, device=DEV, generator=gen) * torch.exp(0.7 * torch.randn(hd, device=DEV, generator=gen))
        # f16: [kv head][position][dimension]; fp32: rows as the projections write them
        kind = torch.float16 if case["half"] else torch.float32
        st["k"], st["v"] = x.to(kind) if case["half"] else x.transpose(1, 2).contiguous().transpose(1, 2)
        shape = (2, kv, st["read"], hd) if case["half"] else (2, st["read"], kv, hd)
        out = torch.empty(shape, dtype=kind, device=DEV)
        st["ko"], st["vo"] = out if case["half"] else out.transpose(1, 2)
        st["q"] = torch.randn(sum(rows), case["heads"], hd, device=DEV, generator=gen).to(kind)
        st["qo"] = torch.empty(sum(rows), case["heads"], hd, device=DEV)
    else:
        lens, entries = _lens(case), _entries(case)
        st["table"], st["refs"], pages = _tables(lens, page_len, 3, host)
        st["pool"], st["len"] = _random_pool(case, pages, gen), _ints(lens)
        st["seq"] = st["ctx"] = None
        if case.get("drafts", 1) > 1:
            st["seq"], st["ctx"] = _ints([s for s, _ in entries]), _ints([c for _, c in entries])
        st["q"] = torch.randn(len(entries), case["heads"], hd, device=DEV, generator=gen)
        st["out"] = torch.empty_like(st["q"])
        if op == "sparse":
            st["chosen"] = torch.empty(len(entries), kv, case["top"], dtype=torch.int32, device=DEV)
    if own:   # the handle and workspace that a program keeps beside its cache
        from quantized_decode_dequant_gb300 import nt
        st["error"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        st["cache"] = nt.make_kv8_cache(
            n_layers=1, n_kv_heads=kv, head_dim=hd, page_len=page_len, n_pages=pages, max_seqs=st["table"].shape[0],
            max_pages=st["table"].shape[1], pool=st["pool"].data_ptr(), table=st["table"].data_ptr(),
            len=st["len"].data_ptr(), refs=st["refs"].data_ptr(), error=st["error"].data_ptr())
        n = st["q"].shape[0] if op != "append" else case["n"]
        st["ws"] = torch.empty(nt.nt_kv8_workspace_bytes(st["cache"], case["heads"] or kv, n), dtype=torch.uint8, device=DEV)
    return st


# -------------------------------------------------------------------- run --

def run(st):
    return {"append": _append, "attention": _attention, "sparse": _sparse}[st["case"]["op"]](st)


def _rotate(x, pos, hd):
    """fp32 [rows, heads, hd]: pairs (2 i, 2 i + 1) rotated by position times frequency i."""
    angle = pos.double().unsqueeze(1) * torch.tensor(_frequencies(hd), dtype=torch.float64, device=DEV)
    c, s = torch.cos(angle).unsqueeze(1), torch.sin(angle).unsqueeze(1)
    a, b = x.double().unflatten(-1, (-1, 2)).unbind(-1)
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2).float()


def _append(st):
    """Rows of keys, rotated by their positions, and values into the last positions of their sequences; queries rotated
    beside them; then those positions, with the older ones of their first page, read back.  The exponents and bounds of
    all pages come along."""
    case, k, v = st["case"], st["k"], st["v"]
    kv, hd, n, p, heads = case["kv"], case["hd"], case["n"], case["page_len"], case["heads"]
    _, _, exps, bounds = _parts(st["pool"], case)
    if own:
        from quantized_decode_dequant_gb300 import nt
        s, kind = torch.cuda.current_stream(), "f16" if case["half"] else "f32"
        nt.nt_kv8_append(st["cache"], 0, n, None, st["begin"].data_ptr(), st["rows"], kind, k.data_ptr(), v.data_ptr(),
                         k.stride(1), k.stride(0), st["freq"], heads, st["q"].data_ptr() if heads else None, heads * hd,
                         st["qo"].data_ptr() if heads else None, heads * hd, s)
        ko, vo = st["ko"], st["vo"]
        nt.nt_kv8_read(st["cache"], 0, n, None, st["begin_read"].data_ptr(), st["read"], kind, ko.data_ptr(), vo.data_ptr(),
                       ko.stride(1), ko.stride(0), s)
        return ko, vo, st["qo"], exps[..., :2], bounds
    row = torch.arange(st["rows"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(st["begin"], row, right=True) - 1
    first = st["len"][seq] - (st["begin"][seq + 1] - st["begin"][seq])            # the sequence's first new position
    pos = (st["len"][seq] - (st["begin"][seq + 1] - row)).long()
    slot = pos // p
    page = st["table"][seq, slot].long()
    kf, vf = _rotate(k.transpose(0, 1), pos, hd), v.transpose(0, 1).float()       # rows, kv, hd
    qo = _rotate(st["q"], pos, hd)
    # pages touched: which they are, and whether older positions are in them
    pages, at = torch.unique(page, return_inverse=True)
    old = torch.zeros(len(pages), dtype=torch.int64, device=DEV).index_put_((at,), (first - slot * p).clamp(0, p - 1).long())
    kc, vc, e, b = (x[pages] for x in _parts(st["pool"], case))
    codes = [kc.transpose(-3, -2).flatten(-2).flatten(-3, -2), vc.transpose(-2, -1).flatten(-3, -2)]   # page, kv, p, hd
    for i, x in enumerate((kf, vf)):
        top = torch.where(_held(x), x.abs(), torch.zeros_like(x)).amax(-1)        # rows, kv
        need = torch.full((len(pages), kv), EMIN, dtype=torch.int32, device=DEV).scatter_reduce_(
            0, at.unsqueeze(1).expand(-1, kv), _exponent(top), "amax")
        was = e[..., i].int()
        now = torch.where(old.unsqueeze(1) > 0, torch.maximum(need, was), need)
        grown = torch.exp2((was - now).float()).unsqueeze(-1)
        again = (codes[i].float() * grown.unsqueeze(-1)).to(torch.float8_e4m3fn)
        held = (torch.arange(p, device=DEV) < old.unsqueeze(1))[:, None, :, None]
        codes[i] = torch.where(held, again.view(torch.uint8), codes[i].view(torch.uint8))
        new = _codes(x, now[at].unsqueeze(-1).expand(x.shape)).view(torch.uint8)
        codes[i][at, :, pos % p] = new
        e[..., i] = now.to(torch.int8)
        if i == 0:
            nan = torch.isnan(new.view(torch.float8_e4m3fn).float())
            y = new.view(torch.float8_e4m3fn).float()
            lo, hi = torch.floor(y / 4), torch.ceil(y / 4)
            lo, hi = torch.where(nan, torch.full_like(lo, -127), lo), torch.where(nan, torch.full_like(hi, 127), hi)
            where = at[:, None, None].expand(-1, kv, hd)
            empty = torch.full((len(pages), kv, hd), 1000.0, device=DEV)
            lo = empty.clone().scatter_reduce_(0, where, lo, "amin")
            hi = (-empty).scatter_reduce_(0, where, hi, "amax")
            lo0, hi0 = b[..., 0, :].float(), b[..., 1, :].float()
            lo0 = torch.where(lo0 == -127, lo0, torch.floor(lo0 * grown))
            hi0 = torch.where(hi0 == 127, hi0, torch.ceil(hi0 * grown))
            has = (old > 0)[:, None, None]
            b[..., 0, :] = torch.where(has, torch.minimum(lo0, lo), lo).to(torch.int8)
            b[..., 1, :] = torch.where(has, torch.maximum(hi0, hi), hi).to(torch.int8)
    kp, vp, ep, bp = _parts(st["pool"], case)
    kp.view(torch.uint8)[pages] = codes[0].unflatten(-1, (hd // 16, 16)).unflatten(-3, (p // 8, 8)).transpose(-3, -2)
    vp.view(torch.uint8)[pages] = codes[1].unflatten(-2, (p // 16, 16)).transpose(-2, -1)
    ep[pages], bp[pages] = e, b
    # back
    row = torch.arange(st["read"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(st["begin_read"], row, right=True) - 1
    pos = (st["len"][seq] - (st["begin_read"][seq + 1] - row)).long()
    page = torch.searchsorted(pages, st["table"][seq, pos // p].long())
    scale = torch.exp2(e[page].float())                                           # rows, kv, 16
    ko, vo = (c.view(torch.float8_e4m3fn)[page, :, pos % p].float() * scale[..., i, None] for i, c in enumerate(codes))
    return ko.transpose(0, 1).to(k.dtype), vo.transpose(0, 1).to(k.dtype), qo, exps[..., :2], bounds


def _seen(st):
    """Table rows and lengths of the queries' sequences."""
    seq = torch.arange(st["len"].numel(), device=DEV) if st["seq"] is None else st["seq"].long()
    return st["table"][seq].long(), (st["len"][seq] if st["ctx"] is None else st["ctx"]).long()


def _softmax_v(q, k, v, live):
    """q [..., group, hd], k and v [..., positions, hd], live [..., 1, positions]; zeros where nothing is live."""
    s = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    s = s.masked_fill(~live, float("-inf"))
    w = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    v = v.masked_fill(~live.transpose(-1, -2), 0)                                  # what lies past the end is no number
    return (w @ v) / w.sum(-1, keepdim=True).clamp(min=1e-30)


def _attention(st):
    """out = softmax(q K^T / sqrt(hd)) V over the positions that a query sees; zeros where there is none."""
    case, q, out = st["case"], st["q"], st["out"]
    heads, kv, hd, n = case["heads"], case["kv"], case["hd"], st["q"].shape[0]
    if own:
        from quantized_decode_dequant_gb300 import nt
        nt.nt_attention_kv8(st["cache"], 0, heads, n, None if st["seq"] is None else st["seq"].data_ptr(),
                            None if st["ctx"] is None else st["ctx"].data_ptr(), 0, None, q.data_ptr(), heads * hd,
                            out.data_ptr(), heads * hd, st["ws"].data_ptr(), st["ws"].numel(), torch.cuda.current_stream())
        return out
    table, seen = _seen(st)
    k, v = _values(st["pool"][table.clamp(min=0)], case)                           # n, max_pages, kv, p, hd
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))
    live = torch.arange(k.shape[2], device=DEV) < seen.view(n, 1, 1, 1)
    return _softmax_v(q.view(n, kv, heads // kv, hd), k, v, live).view(n, heads, hd)


def _scores(q, bounds, exps):
    """Upper bounds of the group's scores on each page: q rounded to whole numbers up to 63 by a power of two, times lo
    or hi, whichever gives more, summed over dimensions and heads.  q [n, kv, group, hd], bounds [n, pages, kv, 2, hd]."""
    m, x = torch.frexp(q.abs().amax((-1, -2)))
    f = (x - 6 + (m > 0.984375).int()).double()
    w = torch.round(q.double() * torch.exp2(-f)[..., None, None])                  # whole numbers: every sum is exact
    up, down = w.clamp(min=0).sum(2).float(), w.clamp(max=0).sum(2).float()        # n, kv, hd
    s = (bounds[..., 1, :].float() * up.unsqueeze(1)).sum(-1) + (bounds[..., 0, :].float() * down.unsqueeze(1)).sum(-1)
    return s.transpose(1, 2) * torch.exp2(exps[..., 0].float()).transpose(1, 2)    # n, kv, pages


def _sparse(st):
    """Every query's group of heads chooses `top` pages: the first and last ones and those of the highest scores (ties to
    the lower page), and attends to their positions.  The choice, ascending with -1 behind, is an output too."""
    case, q, out, chosen = st["case"], st["q"], st["out"], st["chosen"]
    heads, kv, hd, p, n, top = case["heads"], case["kv"], case["hd"], case["page_len"], q.shape[0], case["top"]
    if own:
        from quantized_decode_dequant_gb300 import nt
        s, ws, wb = torch.cuda.current_stream(), st["ws"].data_ptr(), st["ws"].numel()
        nt.nt_kv8_select(st["cache"], 0, heads, n, None, None, q.data_ptr(), heads * hd, top, case["first"], case["last"],
                         chosen.data_ptr(), ws, wb, s)
        nt.nt_attention_kv8(st["cache"], 0, heads, n, None, None, top, chosen.data_ptr(), q.data_ptr(), heads * hd,
                            out.data_ptr(), heads * hd, ws, wb, s)
        return chosen, out
    table, seen = _seen(st)
    qg = q.view(n, kv, heads // kv, hd)
    _, _, exps, bounds = _parts(st["pool"], case)
    at = table.clamp(min=0)
    score = _scores(qg, bounds[at], exps[at])
    pages = ((seen + p - 1) // p).view(n, 1, 1)
    place = torch.arange(table.shape[1], device=DEV)
    always = (place < case["first"]) | (place >= pages - case["last"])
    score = score.masked_fill(always, float("inf")).masked_fill(place >= pages, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    order = torch.where(torch.arange(order.shape[-1], device=DEV) < pages, order, torch.full_like(order, 1 << 40))
    order = torch.sort(order, -1).values
    order = torch.nn.functional.pad(order, (0, top - order.shape[-1]), value=1 << 40)
    some = order < (1 << 40)
    chosen = torch.where(some, order, torch.full_like(order, -1)).int()
    page = at.unsqueeze(1).expand(-1, kv, -1).gather(2, order.masked_fill(~some, 0))          # n, kv, top
    head = torch.arange(kv, device=DEV).view(1, kv, 1)
    kc, vc, ex, _ = _parts(st["pool"], case)
    scale = torch.exp2(ex[page, head].float())
    k = kc.view(torch.uint8)[page, head].view(torch.float8_e4m3fn).float().transpose(-3, -2).flatten(-2).flatten(-3, -2)
    v = vc.view(torch.uint8)[page, head].view(torch.float8_e4m3fn).float().transpose(-2, -1).flatten(-3, -2)
    k, v = (k * scale[..., 0, None, None]).flatten(2, 3), (v * scale[..., 1, None, None]).flatten(2, 3)
    pos = (order * p).unsqueeze(-1) + torch.arange(p, device=DEV)
    live = (some.unsqueeze(-1) & (pos < seen.view(n, 1, 1, 1))).flatten(2).unsqueeze(2)
    return chosen, _softmax_v(qg, k, v, live).view(n, heads, hd)


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """From the definitions in 64 bits, position by position of the layout."""
    st = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "sparse": _exact_sparse}[case["op"]](case, st)


def _byte_values():
    """The number that each e4m3 byte stands for."""
    out = []
    for b in range(256):
        e, m, s = b >> 3 & 15, b & 7, -1.0 if b & 128 else 1.0
        out.append(float("nan") if b & 127 == 127 else s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)))
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _read64(case, st, seq, pos, g, raw=False):
    """K and V of positions of a sequence and kv head [positions, hd] in 64 bits (raw: without the exponents)."""
    hd, p, kv, pool, size = case["hd"], case["page_len"], case["kv"], st["pool"].flatten(), _page_bytes(case)
    d = torch.arange(hd, device=DEV)
    base = st["table"][seq].long()[pos // p] * size
    t = (pos % p).unsqueeze(1)
    head = (base + g * 2 * p * hd).unsqueeze(1)
    k = pool[head + t // 8 * (8 * hd) + d // 16 * 128 + t % 8 * 16 + d % 16].long()
    v = pool[head + p * hd + t // 16 * (16 * hd) + d * 16 + t % 16].long()
    table = _byte_values()
    meta = base + kv * 2 * p * hd + g * (16 + 2 * hd)
    ke, ve = (pool[meta + i].view(torch.int8).double().unsqueeze(1) for i in range(2))
    if raw:
        return table[k], table[v], ke, ve
    return table[k] * 2.0 ** ke, table[v] * 2.0 ** ve


def _e4m3(x):
    """Numbers up to 448 rounded to the nearest that e4m3 holds, ties to even, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _need(x):
    """Smallest exponent from -100 on for values in 64 bits."""
    e = torch.ceil(torch.log2(x.abs().max().clamp(min=1e-300) / 448))
    while 448 * 2.0 ** float(e) < float(x.abs().max()):
        e += 1
    while float(e) > EMIN and 448 * 2.0 ** (float(e) - 1) >= float(x.abs().max()):
        e -= 1
    return max(float(e), float(EMIN))


def _exact_append(case, st):
    """What the rows read back hold: the scale of each page from all it gets, older codes rounded a second time."""
    kv, hd, p, kept = case["kv"], case["hd"], case["page_len"], case["kept"]
    few = sum(_rows(case)) * kv <= 4000                    # page by page: the large ones would take too long
    freq = torch.tensor(_frequencies(hd), dtype=torch.float64, device=DEV)

    def turned(x, pos):
        a = pos.double().view(-1, 1, 1) * freq
        y = torch.view_as_complex(x.double().reshape(x.shape[:-1] + (hd // 2, 2)).contiguous()) * torch.polar(torch.ones_like(a), a)
        return torch.view_as_real(y).reshape(x.shape)

    row0, qs, ko, vo = 0, [], [], []
    for i, r in enumerate(_rows(case)):
        pos = torch.arange(kept, kept + r, device=DEV)
        qs.append(turned(st["q"][row0:row0 + r], pos))
        if few:
            k = turned(st["k"][:, row0:row0 + r].transpose(0, 1), pos).float().double()    # rows, kv, hd: an fp32 key is what is held
            v = st["v"][:, row0:row0 + r].transpose(0, 1).double()
            for j in range(kept // p, (kept + r - 1) // p + 1):
                new = (pos >= j * p) & (pos < (j + 1) * p)
                older = torch.arange(j * p, max(j * p, min(kept, (j + 1) * p)), device=DEV)
                for g in range(kv):
                    rk, rv, ke, ve = _read64(case, st, i, older, g, raw=True)
                    for fresh, held, was, out in ((k[new, g], rk, ke, ko), (v[new, g], rv, ve, vo)):
                        e = _need(fresh)
                        if len(older):
                            e = max(e, float(was[0]))
                            held = _e4m3(held * 2.0 ** (was - e))
                        out.append((torch.cat([held, _e4m3(fresh * 2.0 ** -e)]) * 2.0 ** e).unsqueeze(0))
        row0 += r
    q = torch.cat(qs)
    if not few:
        return None, None, q, None, None

    def together(parts):
        return torch.cat([torch.cat(parts[at:at + kv]) for at in range(0, len(parts), kv)], 1)

    return together(ko), together(vo), q, None, None


def _attend64(case, st, entry, g, seq, pos):
    group, hd = case["heads"] // case["kv"], case["hd"]
    k, v = _read64(case, st, seq, pos, g)
    return torch.softmax(st["q"][entry, g * group:(g + 1) * group].double() @ k.T / math.sqrt(hd), -1) @ v


def _exact_attention(case, st):
    group = case["heads"] // case["kv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for i, (seq, n) in enumerate(_entries(case)):
        for g in range(case["kv"] if n else 0):
            out[i, g * group:(g + 1) * group] = _attend64(case, st, i, g, seq, torch.arange(n, device=DEV))
    return out


def _exact_sparse(case, st):
    """The pages chosen are whole numbers: they come out of the integers' definition, head by head."""
    group, hd, p, kv, top = case["heads"] // case["kv"], case["hd"], case["page_len"], case["kv"], case["top"]
    pool, size = st["pool"].flatten(), _page_bytes(case)
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    chosen = torch.full((case["n"], kv, top), -1, dtype=torch.int32, device=DEV)
    for i, n in enumerate(_lens(case)):
        m = -(-n // p)
        for g in range(kv if n else 0):
            q = st["q"][i, g * group:(g + 1) * group].double()
            f = math.floor(math.log2(float(q.abs().max()) / 63)) - 1
            while 63 * 2.0 ** f < float(q.abs().max()):
                f += 1
            w = torch.round(q / 2.0 ** f)
            meta = st["table"][i, :m].long() * size + kv * 2 * p * hd + g * (16 + 2 * hd)
            d = torch.arange(2 * hd, device=DEV)
            b = pool[meta.unsqueeze(1) + 16 + d].view(torch.int8).double()
            e = pool[meta].view(torch.int8).double()
            s = sum(torch.maximum(w[h] * b[:, :hd], w[h] * b[:, hd:]).sum(1) for h in range(group)) * 2.0 ** e
            j = torch.arange(m, device=DEV)
            s[(j < case["first"]) | (j >= m - case["last"])] = float("inf")
            pick = torch.sort(torch.sort(-s, stable=True).indices[:top]).values
            chosen[i, g, :len(pick)] = pick.int()
            pos = (pick.unsqueeze(1) * p + torch.arange(p, device=DEV)).flatten()
            out[i, g * group:(g + 1) * group] = _attend64(case, st, i, g, i, pos[pos < n])
    return chosen, out
