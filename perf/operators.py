"""Cases of the paged 4-bit K/V cache operators: attention over it, append and read, and the page operators.

Each case names one pass through an operator.  With ``own`` false ``run`` computes the plain form (elementary torch
operations in fp32); with ``own`` true it makes the library calls.  Both read and write the same page pool.

The cache.  A page holds ``page_len`` positions (a multiple of 16) of one layer: for every kv head the 16-position
chunks one after the other.  With NG = head_dim / 32, one chunk is
  K codes  [i 2][n 8][tg 4][j NG] words of 4 bytes: the 4-bit codes of position 8 i + n, dimensions 32 j + 8 tg + 0..7
  V codes  [r 2][gi 8][tg 4][j NG] words: low half position 8 r + 2 tg, high half the next one, each the codes of
           dimensions 32 j + 4 gi + 0..3
  K scales [position 16][j NG] f16
  V scales [r 2][tg 4][j NG][2] f16: positions 8 r + 2 tg and the next one
with the lowest code in the lowest bits.  A value is d (q - 8), d the scale of its 32 dimensions, q its code.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the decode step of the tiny two-layer model: latency of one call
        dict(name="attention 1 short", op="attention", heads=8, kv=2, hd=64, page_len=16, n=1, longest=37, ragged=False),
        # one 70B-shaped layer, batch 1, a few thousand positions: the flagship decode step's context
        dict(name="attention 1 x 4k", op="attention", heads=64, kv=8, hd=128, page_len=64, n=1, longest=4161, ragged=False),
        # one 70B-shaped layer over a very long document
        dict(name="attention 1 x 131k", op="attention", heads=64, kv=8, hd=128, page_len=64, n=1, longest=131077,
             ragged=False),
        # 8B-shaped layer, many samples of different lengths, one of them just begun (empty)
        dict(name="attention 56 ragged", op="attention", heads=32, kv=8, hd=128, page_len=32, n=56, longest=9001,
             ragged=True),
        # one new token of each of 16 sequences, read back
        dict(name="store 16 tokens", op="store", kv=8, hd=128, page_len=64, n=16, rows=1, kept=700, half=False),
        # an f16 cache ([kv head][position][dimension], as the f16 attention reads it) taken over into 4 bits
        dict(name="store 2 x 20k f16", op="store", kv=8, hd=128, page_len=64, n=2, rows=20011, kept=0, half=True),
        # a few pages of the tiny model
        dict(name="copy 3 pages", op="copy", kv=2, hd=64, page_len=16, layers=2, pages=12, moved=3),
        # pages of all 80 layers of the 70B shape
        dict(name="copy 24 pages x 80", op="copy", kv=8, hd=128, page_len=64, layers=80, pages=64, moved=24),
        # two branches of one speculative draft are dropped and drawn anew
        dict(name="branch 2", op="branch", kv=2, hd=64, page_len=16, layers=2, parents=1, branches=2, longest=45),
        # 8 prompts, 5 samples each, 32 layers
        dict(name="branch 8 x 5", op="branch", kv=8, hd=128, page_len=64, layers=32, parents=8, branches=5, longest=2999),
        # a small cache after one sequence left
        dict(name="compact 40 pages", op="compact", kv=2, hd=64, page_len=16, layers=2, pages=40, live=20, moved=6),
        # a large cache, two thirds free, before the rest of the memory is given away
        dict(name="compact 420 x 32", op="compact", kv=8, hd=128, page_len=64, layers=32, pages=420, live=140, moved=60),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "store", "copy", "branch", "compact"])
    hd, kv, page_len = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 48, 64, 128])
    row = kv * (hd + hd // 8)                       # cache bytes of one position
    if op == "attention":
        n = _spread(rng, 1, 64)
        longest = _spread(rng, 1, min(131072, 100_000_000 // (row * n)))
        return dict(op=op, heads=kv * rng.choice([1, 2, 4, 8, 16]), kv=kv, hd=hd, page_len=page_len, n=n, longest=longest,
                    ragged=rng.random() < 0.6)
    if op == "store":
        n = _spread(rng, 1, 64)
        return dict(op=op, kv=kv, hd=hd, page_len=page_len, n=n, rows=_spread(rng, 1, max(2, 20000 // n)),
                    kept=rng.choice([0, _spread(rng, 1, 2000)]), half=rng.random() < 0.4)
    layers = _spread(rng, 1, 80)
    most = max(4, 300_000_000 // (row * page_len * layers))   # pages whose bytes in all layers come to 300 MB
    if op == "copy":
        moved = _spread(rng, 1, max(1, min(400, most // 3)))
        return dict(op=op, kv=kv, hd=hd, page_len=page_len, layers=layers, pages=2 * moved + rng.randint(0, 9), moved=moved)
    if op == "branch":
        parents, branches = _spread(rng, 1, 8), _spread(rng, 1, 8)
        pages = max(1, min(60, most // parents - branches - 2))
        return dict(op=op, kv=kv, hd=hd, page_len=page_len, layers=max(1, layers // 2), parents=parents, branches=branches,
                    longest=_spread(rng, 1, pages * page_len))
    live = _spread(rng, 1, max(2, min(2000, most // 3)))
    return dict(op=op, kv=kv, hd=hd, page_len=page_len, layers=layers, pages=2 * live + rng.randint(0, 9), live=live,
                moved=rng.randint(0, live))


def _lens(case):
    """Lengths of the sequences of a case: the longest first; ragged ones spread evenly, the fourth of them empty."""
    n, longest = case.get("n") or case["parents"], case["longest"]
    if not case.get("ragged", "parents" in case):
        return [longest] * n
    return [0 if i == 3 and "n" in case else 1 + int((longest - 1) * (1 - (i * 0.6180339887) % 1)) for i in range(n)]


def _chunk_bytes(case):
    return 16 * case["hd"] + 2 * case["hd"]


def _page_bytes(case):
    return case["kv"] * case["page_len"] // 16 * _chunk_bytes(case)


def work(case):
    pos = case["kv"] * (case["hd"] + case["hd"] // 8)      # cache bytes of a position
    if case["op"] == "attention":
        total = sum(_lens(case))
        tables = sum(-(-x // case["page_len"]) for x in _lens(case)) * 4
        return dict(bytes=total * pos + 2 * case["n"] * case["heads"] * case["hd"] * 4 + tables,
                    flops=4 * total * case["heads"] * case["hd"])
    if case["op"] == "store":
        rows = sum(_rows(case))
        values = 2 * rows * case["kv"] * case["hd"] * (2 if case["half"] else 4)
        return dict(bytes=2 * values + 2 * rows * pos, flops=0)
    if case["op"] == "branch":
        tails = case["branches"] * sum(x % case["page_len"] != 0 for x in _lens(case))
        pages = (case["branches"] + 1) * sum(-(-(x + 1) // case["page_len"]) for x in _lens(case))
        return dict(bytes=2 * tails * case["layers"] * _page_bytes(case) + 16 * pages, flops=0)
    tables = 16 * case["live"] if case["op"] == "compact" else 0
    return dict(bytes=2 * case["moved"] * case["layers"] * _page_bytes(case) + tables + 4 * case["pages"], flops=0)


def _rows(case):
    """New rows of each sequence: the last one takes one fewer where there are several."""
    return [case["rows"] - (1 if i and i == case["n"] - 1 and case["rows"] > 1 else 0) for i in range(case["n"])]


# ----------------------------------------------------- pages, in torch --

def _quantize(x):
    """fp32 [..., hd] -> (codes uint8 [..., hd], scales f16 [..., hd / 32]): 4-bit codes and the scale of each 32."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    h = (top / 7).half()
    d = ((h.view(torch.int16).int() + 8) & 0xFFF0).to(torch.int16).view(torch.float16)
    bad = ~(torch.isfinite(b).all(-1) & (d <= 896))
    d = torch.where(bad, torch.full_like(d, float("nan")), d)
    flat = (bad | (d == 0)).unsqueeze(-1)
    r = torch.where(flat, torch.zeros_like(b), b / torch.where(flat, torch.ones_like(b[..., :1]), d.float().unsqueeze(-1)))
    t = torch.trunc(r)
    t = t + torch.sign(r) * ((r - t).abs() >= 0.5)          # half away from zero
    return (t + 8).clamp(0, 15).to(torch.uint8).flatten(-2), d


def _nibbles(q):
    """Codes, an even number of them last, to bytes: the first of two in the low half."""
    q = q.unflatten(-1, (-1, 2))
    return q[..., 0] | (q[..., 1] << 4)


def _pack(kq, kd, vq, vd):
    """Codes and scales [..., 16, hd] of whole chunks to chunk bytes [..., chunk]."""
    ng = kd.shape[-1]
    k = kq.unflatten(-1, (ng, 4, 8)).transpose(-3, -2)                                   # 16, tg, j, 8
    v = vq.unflatten(-1, (ng, 8, 4)).unflatten(-4, (2, 4, 2))                            # r, tg, half, j, gi, 4
    v = v.permute(*range(v.dim() - 6), -6, -2, -5, -3, -4, -1)                           # r, gi, tg, j, half, 4
    vd = vd.unflatten(-2, (2, 4, 2)).transpose(-2, -1)                                   # r, tg, j, half
    return torch.cat([_nibbles(k).flatten(-4), _nibbles(v).flatten(-6), kd.contiguous().view(torch.uint8).flatten(-2),
                      vd.contiguous().view(torch.uint8).flatten(-4)], -1)


def _unpack(chunks, hd):
    """Chunk bytes [..., chunk] to fp32 K and V [..., 16, hd]."""
    ng, code = hd // 32, 8 * hd

    def codes(part, *shape):
        part = part.unflatten(-1, shape)
        return torch.stack([part & 15, part >> 4], -1).flatten(-2)

    k = codes(chunks[..., :code], 16, 4, ng, 4).transpose(-3, -2).flatten(-3)
    v = codes(chunks[..., code:2 * code], 2, 8, 4, ng, 4).unflatten(-1, (2, 4))          # r, gi, tg, j, half, 4
    v = v.permute(*range(v.dim() - 6), -6, -4, -2, -3, -5, -1).flatten(-3).flatten(-4, -2)
    s = chunks[..., 2 * code:].contiguous().view(torch.float16)
    kd = s[..., :16 * ng].unflatten(-1, (16, ng))
    vd = s[..., 16 * ng:].unflatten(-1, (2, 4, ng, 2)).transpose(-2, -1).flatten(-4, -2)

    def values(q, d):
        return ((q.float() - 8).unflatten(-1, (ng, 32)) * d.float().unsqueeze(-1)).flatten(-2)

    return values(k, kd), values(v, vd)


def _random_pool(case, layers, pages, gen):
    """Pages of normal K and V, K with a few strong channels, as trained keys have."""
    shape = (layers * pages, case["kv"], case["page_len"] // 16, 16, case["hd"])
    chans = torch.where(torch.rand(case["hd"], device=DEV, generator=gen) < 0.06, 4.0, 0.8)
    out = torch.empty(layers * pages, _page_bytes(case), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (case["kv"] * case["page_len"] * case["hd"]))
    for a in range(0, layers * pages, step):
        part = (min(step, layers * pages - a),) + shape[1:]
        k = torch.randn(part, device=DEV, generator=gen) * chans
        v = torch.randn(part, device=DEV, generator=gen)
        out[a:a + step] = _pack(*_quantize(k), *_quantize(v)).flatten(1)
    return out.view(layers, pages, -1)


def _random_bytes(case, layers, pages, gen):
    """Pages for operators that move them whole: random bytes, finite scales left aside."""
    n = layers * pages * _page_bytes(case) // 8
    return torch.randint(-(1 << 61), 1 << 61, (n,), device=DEV, generator=gen).view(torch.uint8).view(layers, pages, -1)


# ---------------------------------------------------------------- prepare --

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tables(lens, page_len, pages, max_pages, order):
    """Page tables of sequences that take their pages from `order`, and the reference counts."""
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    at = 0
    for i, x in enumerate(lens):
        m = -(-x // page_len)
        table[i, :m] = order[at:at + m]
        at += m
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[order[:at].long()] = 1
    return table.to(DEV), refs.to(DEV)


def prepare(case, seed):
    gen, host = torch.Generator(DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
    op, kv, hd, page_len = case["op"], case["kv"], case["hd"], case["page_len"]
    layers = case.get("layers", 1)
    st = dict(case=case)
    if op == "attention":
        lens = _lens(case)
        max_pages = max(1, -(-max(lens) // page_len))
        pages = sum(-(-x // page_len) for x in lens) + 3
        st["table"], st["refs"] = _tables(lens, page_len, pages, max_pages, torch.randperm(pages, generator=host).int())
        st["pool"], st["len"] = _random_pool(case, 1, pages, gen), _ints(lens)
        st["q"] = torch.randn(case["n"], case["heads"], hd, device=DEV, generator=gen)
        st["out"] = torch.empty_like(st["q"])
    elif op == "store":
        rows, n = _rows(case), case["n"]
        lens = [case["kept"] + r for r in rows]             # the rows' pages are there already
        max_pages = -(-max(lens) // page_len)
        pages = sum(-(-x // page_len) for x in lens) + 2
        st["table"], st["refs"] = _tables(lens, page_len, pages, max_pages, torch.randperm(pages, generator=host).int())
        st["pool"], st["len"] = torch.zeros(1, pages, _page_bytes(case), dtype=torch.uint8, device=DEV), _ints(lens)
        st["rows"] = sum(rows)
        st["begin"] = torch.nn.functional.pad(_ints(rows).cumsum(0).int(), (1, 0))
        x = torch.randn(2, kv, sum(rows), hd, device=DEV, generator=gen) * torch.exp(torch.randn(hd, device=DEV, generator=gen))
        # f16: an existing cache's order, [kv head][position][dimension]; fp32: rows as the projections write them
        x = x.half() if case["half"] else x.transpose(1, 2).contiguous().transpose(1, 2)
        st["k"], st["v"] = x[0], x[1]
        st["ko"], st["vo"] = torch.empty_like(x[0]), torch.empty_like(x[1])
    elif op == "copy":
        st["pool"] = _random_bytes(case, layers, case["pages"], gen)
        order = torch.randperm(case["pages"], generator=host).int()
        st["src"], st["dst"] = order[:case["moved"]].to(DEV), order[case["moved"]:2 * case["moved"]].to(DEV)
        st["table"], st["len"] = _ints([[-1]]), _ints([0])
        st["refs"] = torch.ones(case["pages"], dtype=torch.int32, device=DEV)
    elif op == "branch":
        lens, b = _lens(case), case["branches"]
        p, grown = len(lens), [x + 1 for x in lens]
        max_pages = -(-max(grown) // page_len)
        pages = sum(-(-x // page_len) for x in grown) + 2 * p * b + 3
        order = torch.randperm(pages, generator=host).int()
        table, st["refs"] = _tables(lens + [0] * (p * b), page_len, pages, max_pages, order)
        st["table"], st["len"] = table, _ints(lens + [0] * (p * b))
        st["pool"] = _random_bytes(case, layers, pages, gen)
        st["all"] = _ints(list(range(p + p * b)))
        st["keep"] = _ints(lens + [0] * (p * b))              # parents back to their prompts, branches dropped
        st["src"] = _ints([i for i in range(p) for _ in range(b)])
        st["dst"] = _ints([p + i for i in range(p * b)])
        st["one"] = torch.ones(p + p * b, dtype=torch.int32, device=DEV)
    elif op == "compact":
        pages, live, moved = case["pages"], case["live"], case["moved"]
        low, high = torch.randperm(live, generator=host), live + torch.randperm(pages - live, generator=host)
        used = torch.cat([low[moved:], high[:moved]])[torch.randperm(live, generator=host)].int()
        st["pool"] = _random_bytes(case, layers, pages, gen)
        n = 1 + live // 9                                       # sequences that hold the live pages
        held = [live // n + (i < live % n) for i in range(n)]
        st["table"], st["refs"] = _tables([h * page_len for h in held], page_len, pages, max(held) + 2, used)
        st["len"] = _ints([h * page_len - i % page_len for i, h in enumerate(held)])
        st["table_out"], st["refs_out"] = torch.empty_like(st["table"]), torch.empty_like(st["refs"])
        st["live"] = torch.empty(1, dtype=torch.int32, device=DEV)
    else:
        raise ValueError(op)
    if own:   # the handle and workspace that a program keeps beside its cache
        from quantized_decode_dequant_gb300 import nt
        st["error"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        st["cache"] = nt.make_kv4_cache(
            n_layers=layers, n_kv_heads=kv, head_dim=hd, page_len=page_len, n_pages=st["pool"].shape[1],
            max_seqs=st["table"].shape[0], max_pages=st["table"].shape[1], pool=st["pool"].data_ptr(),
            table=st["table"].data_ptr(), len=st["len"].data_ptr(), refs=st["refs"].data_ptr(),
            error=st["error"].data_ptr())
        n = max(st["table"].shape[0], case.get("moved", 0))
        st["ws"] = torch.empty(nt.nt_kv4_workspace_bytes(st["cache"], case.get("heads", kv), n), dtype=torch.uint8,
                               device=DEV)
    return st


# -------------------------------------------------------------------- run --

def run(st):
    return {"attention": _attention, "store": _store, "copy": _copy, "branch": _branch, "compact": _compact}[
        st["case"]["op"]](st)


def _attention(st):
    """out = softmax(q K^T / sqrt(hd)) V over each sequence's cached positions; zeros where there is none."""
    case, q, out = st["case"], st["q"], st["out"]
    heads, kv, hd, n = case["heads"], case["kv"], case["hd"], case["n"]
    if own:
        from quantized_decode_dequant_gb300 import nt
        nt.nt_attention_kv4(st["cache"], 0, heads, n, None, q.data_ptr(), heads * hd, out.data_ptr(), heads * hd,
                            st["ws"].data_ptr(), st["ws"].numel(), torch.cuda.current_stream())
        return out
    pages = st["pool"][0][st["table"].long().clamp(min=0)]                       # n, max_pages, bytes
    k, v = _unpack(pages.unflatten(-1, (kv, case["page_len"] // 16, _chunk_bytes(case))), hd)
    k, v = (x.permute(0, 2, 1, 3, 4, 5).flatten(2, 4) for x in (k, v))           # n, kv, positions, hd
    s = q.view(n, kv, heads // kv, hd) @ k.transpose(-1, -2) / math.sqrt(hd)
    off = torch.arange(k.shape[2], device=DEV) >= st["len"].view(n, 1, 1, 1)
    s = s.masked_fill(off, float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    v = v.masked_fill(off.transpose(-1, -2), 0)                                   # what lies past the end is no number
    return ((p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)).view(n, heads, hd)


def _store(st):
    """Quantise rows into the last positions of their sequences, then read the same positions back."""
    case, k, v = st["case"], st["k"], st["v"]
    kv, hd, n, page_len = case["kv"], case["hd"], case["n"], case["page_len"]
    if own:
        from quantized_decode_dequant_gb300 import nt
        s, kind = torch.cuda.current_stream(), "f16" if case["half"] else "f32"
        nt.nt_kv4_append(st["cache"], 0, n, None, st["begin"].data_ptr(), st["rows"], kind, k.data_ptr(), v.data_ptr(),
                         k.stride(1), k.stride(0), s)
        ko, vo = st["ko"], st["vo"]
        nt.nt_kv4_read(st["cache"], 0, n, None, st["begin"].data_ptr(), st["rows"], kind, ko.data_ptr(), vo.data_ptr(),
                       ko.stride(1), ko.stride(0), s)
        return ko, vo
    row = torch.arange(st["rows"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(st["begin"], row, right=True) - 1
    pos = (st["len"][seq] - (st["begin"][seq + 1] - row)).long()
    page, at = st["table"][seq, pos // page_len].long(), pos % page_len
    chunk, t = at // 16, at % 16
    ng, code = hd // 32, 8 * hd
    (kq, kd), (vq, vd) = (_quantize(x.transpose(0, 1).float()) for x in (k, v))    # rows, kv, hd
    chunks = st["pool"][0].unflatten(-1, (kv, page_len // 16, _chunk_bytes(case)))
    kc = chunks[..., :code].unflatten(-1, (16, 4, ng, 4))
    vc = chunks[..., code:2 * code].unflatten(-1, (2, 8, 4, ng, 2, 2))
    kc[page, :, chunk, t] = _nibbles(kq.unflatten(-1, (ng, 4, 8)).transpose(-3, -2))
    vc[page, :, chunk, t // 8, :, t % 8 // 2, :, t % 2] = _nibbles(vq.unflatten(-1, (ng, 8, 4)).transpose(-3, -2))
    ks = chunks[..., 2 * code:2 * code + 32 * ng].unflatten(-1, (16, ng, 2))
    vs = chunks[..., 2 * code + 32 * ng:].unflatten(-1, (2, 4, ng, 2, 2))
    ks[page, :, chunk, t] = kd.contiguous().view(torch.uint8).unflatten(-1, (ng, 2))
    vs[page, :, chunk, t // 8, t % 8 // 2, :, t % 2] = vd.contiguous().view(torch.uint8).unflatten(-1, (ng, 2))
    # back: the codes and scales of each row out of its chunk
    kb, vb = kc[page, :, chunk, t], vc[page, :, chunk, t // 8, :, t % 8 // 2, :, t % 2]
    kb, vb = (torch.stack([b & 15, b >> 4], -1).flatten(-2).transpose(-3, -2).flatten(-3) for b in (kb, vb))
    kd = ks[page, :, chunk, t].contiguous().flatten(-2).view(torch.float16)
    vd = vs[page, :, chunk, t // 8, t % 8 // 2, :, t % 2].contiguous().flatten(-2).view(torch.float16)

    def values(q, d):
        x = ((q.float() - 8).unflatten(-1, (ng, 32)) * d.float().unsqueeze(-1)).flatten(-2)
        return x.transpose(0, 1).to(k.dtype)

    return values(kb, kd), values(vb, vd)


def _copy(st):
    """Page dst[i] becomes a copy of page src[i] in every layer.  The pool is returned as 8-byte words."""
    if own:
        from quantized_decode_dequant_gb300 import nt
        nt.nt_kv4_copy_pages(st["cache"], st["src"].numel(), st["src"].data_ptr(), st["dst"].data_ptr(),
                             torch.cuda.current_stream())
    else:
        words = st["pool"].view(torch.int64)
        words[:, st["dst"].long()] = words[:, st["src"].long()]
    return st["pool"].view(torch.int64)


def _branch(st):
    """Sequences give back what lies behind `keep`; the branches start anew as copies of their parents (full pages shared,
    the partly filled one copied); every sequence gets room for one more position."""
    pool, table, length, refs = st["pool"], st["table"], st["len"], st["refs"]
    if own:
        from quantized_decode_dequant_gb300 import nt
        s, ws, wb = torch.cuda.current_stream(), st["ws"].data_ptr(), st["ws"].numel()
        c = st["cache"]
        nt.nt_kv4_free(c, st["all"].numel(), st["all"].data_ptr(), st["keep"].data_ptr(), s)
        nt.nt_kv4_fork(c, st["src"].numel(), st["src"].data_ptr(), st["dst"].data_ptr(), None, ws, wb, s)
        nt.nt_kv4_extend(c, st["all"].numel(), st["all"].data_ptr(), st["one"].data_ptr(), ws, wb, s)
        return table, length, refs, pool.view(torch.int64)
    size, words = st["case"]["page_len"], pool.view(torch.int64)
    place = torch.arange(table.shape[1], device=DEV)
    # give back
    dropped = (place >= (st["keep"].unsqueeze(1) + size - 1) // size) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -dropped.flatten().int())
    table.masked_fill_(dropped, -1)
    length.copy_(st["keep"])
    # branch
    src, dst = st["src"].long(), st["dst"].long()
    n = length[src].long()
    whole, tail = n // size, n % size != 0
    free = torch.argsort(refs != 0, stable=True)                                  # free pages, the lowest first
    new = free[(tail.cumsum(0) - 1).clamp(min=0)]
    row = table[src]
    old = row.gather(1, whole.clamp(max=table.shape[1] - 1).unsqueeze(1)).squeeze(1).long()
    shared = place < whole.unsqueeze(1)
    refs.index_add_(0, row.clamp(min=0).flatten().long(), shared.flatten().int())
    refs.index_add_(0, new, tail.int())
    rows = torch.where(shared, row, torch.where((place == whole.unsqueeze(1)) & tail.unsqueeze(1), new.int().unsqueeze(1), -1))
    table[dst] = rows.int()
    length[dst] = n.int()
    at = torch.nonzero(tail).squeeze(1)
    words[:, new[at]] = words[:, old[at]]
    # one more position: a fresh page where the last is full, or a copy of one that others hold too
    n = length.long()
    last = (n // size).clamp(max=table.shape[1] - 1)
    old = table.gather(1, last.unsqueeze(1)).squeeze(1).long()
    copied = (n % size != 0) & (refs[old.clamp(min=0)] > 1)
    fresh = (n % size == 0) | copied
    free = torch.argsort(refs != 0, stable=True)
    new = torch.where(fresh, free[(fresh.cumsum(0) - 1).clamp(min=0)], old)
    refs.index_add_(0, old.clamp(min=0), -copied.int())
    refs.index_add_(0, new, fresh.int())
    table.scatter_(1, last.unsqueeze(1), new.int().unsqueeze(1))
    at = torch.nonzero(copied).squeeze(1)
    words[:, new[at]] = words[:, old[at]]
    length.add_(1)
    return table, length, refs, words


def _compact(st):
    """The live pages move below the number of live pages, into the holes there; the tables follow.  The tables before
    are kept beside the new ones, so a pass can be made again."""
    pool, table, refs = st["pool"], st["table"], st["refs"]
    if own:
        from quantized_decode_dequant_gb300 import nt
        nt.nt_kv4_compact(st["cache"], st["table_out"].data_ptr(), st["refs_out"].data_ptr(), st["live"].data_ptr(),
                          st["ws"].data_ptr(), st["ws"].numel(), torch.cuda.current_stream())
        return st["table_out"], st["refs_out"], st["live"], pool.view(torch.int64)
    used = refs > 0
    live = used.sum()
    place = torch.arange(refs.numel(), device=DEV)
    src, dst = (torch.nonzero(m).squeeze(1) for m in (used & (place >= live), ~used & (place < live)))
    to = place.clone()
    to[src] = dst
    words = pool.view(torch.int64)
    words[:, dst] = words[:, src]
    st["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), -1))
    out = st["refs_out"].copy_(refs)
    out[dst], out[src] = refs[src], 0
    st["live"].copy_(live)
    return st["table_out"], out, st["live"], words


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """Attention and the stored values from their definitions in 64 bits; the page operators move whole numbers."""
    if case["op"] not in ("attention", "store"):
        return None
    st = prepare(case, seed)
    return _exact_attention(case, st) if case["op"] == "attention" else _exact_store(case, st)


def _exact_attention(case, st):
    heads, kv, hd, page_len, ng = case["heads"], case["kv"], case["hd"], case["page_len"], case["hd"] // 32
    pool = st["pool"].flatten()
    e = torch.arange(hd, device=DEV)
    out = torch.zeros(case["n"], heads, hd, dtype=torch.float64, device=DEV)
    for i, n in enumerate(_lens(case)):
        for g in range(kv if n else 0):
            t = torch.arange(n, device=DEV)
            page = st["table"][i].long()[t // page_len]
            chunk = (page * _page_bytes(case) + (g * (page_len // 16) + t % page_len // 16) * _chunk_bytes(case)).unsqueeze(1)
            p = (t % 16).unsqueeze(1)                       # position within its chunk
            # K: code number m = e % 8 of word (p, (e / 8) % 4, e / 32)
            byte = chunk + 4 * ((p * 4 + e // 8 % 4) * ng + e // 32) + e % 8 // 2
            k = (pool[byte].long() >> (4 * (e % 2))) & 15
            d = chunk + 16 * hd + 2 * (p * ng + e // 32)
            kf = (k - 8).double() * _half_at(pool, d)
            # V: code number 4 (p % 2) + e % 4 of word (p / 8, (e / 4) % 8, (p / 2) % 4, e / 32)
            word = ((p // 8 * 8 + e // 4 % 8) * 4 + p // 2 % 4) * ng + e // 32
            byte = chunk + 8 * hd + 4 * word + 2 * (p % 2) + e % 4 // 2
            v = (pool[byte].long() >> (4 * (e % 2))) & 15
            d = chunk + 16 * hd + 32 * ng + 2 * (((p // 2) * ng + e // 32) * 2 + p % 2)
            vf = (v - 8).double() * _half_at(pool, d)
            rows = slice(g * (heads // kv), (g + 1) * (heads // kv))
            s = st["q"][i, rows].double() @ kf.T / math.sqrt(hd)
            out[i, rows] = torch.softmax(s, -1) @ vf
    return out


def _half_at(pool, at):
    """The f16 numbers at byte addresses, in 64 bits."""
    b = pool[at].int() | (pool[at + 1].int() << 8)
    return b.to(torch.int16).view(torch.float16).double()


def _exact_store(case, st):
    def one(x):
        b = x.double().reshape(*x.shape[:-1], -1, 32)
        top = torch.max(torch.abs(b), -1, keepdim=True).values
        # the scale: top / 7 rounded to fp32, to f16, then to six bits behind the leading one (never below 2^-20)
        d = (top / 7).float().half().double()
        step = torch.exp2(torch.floor(torch.log2(d.clamp(min=2.0 ** -14))) - 6)
        d = torch.floor(d / step + 0.5) * step
        ratio = (b / torch.where(d > 0, d, torch.ones_like(d))).float().double()     # one fp32 division
        q = torch.where(ratio < 0, -torch.floor(0.5 - ratio), torch.floor(ratio + 0.5)).clamp(-8, 7)
        return torch.where(d > 0, q * d, torch.zeros_like(b)).reshape(x.shape)

    return one(st["k"]), one(st["v"])
