"""What is measured of the paged 8-bit cache: attention that reads it, the append that writes it, and the
operations on its pages.

A cache is four pools indexed by page: codes ``k_pages``/``v_pages`` [num_pages, Hkv, page_size, D]
(float8_e4m3fn or int8) and fp32 ``k_scales``/``v_scales`` [num_pages, Hkv, page_size / 16], one scale
for each block of 16 tokens and head; a code stands for code * scale.  ``table`` int32 [slots,
pages_per_seq] lists each sequence's pages in key order, ``seqlens`` int32 [slots] its length, ``refs``
int32 [num_pages] how many sequences hold a page.
"""
import math

import torch

own = False

BLOCK = 16                                      # tokens that share a scale
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FLOAT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the smallest call: one short chat of a small model, one token: latency is all there is
        dict(name="attend one token, len 37", kind="attend", B=1, Nq=1, Hkv=2, G=4, D=64, page=16, longest=37, even=True,
             codes="e4m3", dtype="bf16", shared=0),
        # a serving batch of ragged lengths, one token each (the decode benchmark's heads and capacity)
        dict(name="attend batch 64 ragged 8192", kind="attend", B=64, Nq=1, Hkv=8, G=4, D=128, page=16, longest=8192, even=False,
             codes="e4m3", dtype="bf16", shared=0),
        # few sequences with a very long context (the sharded decode benchmark's length): one long axis
        dict(name="attend 4 x 131072", kind="attend", B=4, Nq=1, Hkv=8, G=4, D=128, page=64, longest=131072, even=True,
             codes="int8", dtype="fp16", shared=0),
        # drafted tokens verified together, odd group of heads, odd lengths
        dict(name="attend verify 5 tokens", kind="attend", B=16, Nq=5, Hkv=4, G=7, D=128, page=32, longest=4099, even=False,
             codes="int8", dtype="fp16", shared=0),
        # chunks of prompts behind a cached prefix that the sequences share
        dict(name="attend chunk 1024 of 16384", kind="attend", B=2, Nq=1024, Hkv=8, G=4, D=128, page=16, longest=16384, even=True,
             codes="e4m3", dtype="bf16", shared=8192),
        # a decode step's new rows, one for each sequence, into blocks that are partly filled
        dict(name="append decode step, 64 rows", kind="append", B=64, Nt=1, even=True, Hkv=8, D=128, page=16, before=8000,
             codes="e4m3", dtype="bf16"),
        # whole prompts of ragged lengths into empty sequences
        dict(name="append prompts 8 x 2048", kind="append", B=8, Nt=2048, even=False, Hkv=8, D=128, page=64, before=0,
             codes="e4m3", dtype="bf16"),
        # accepted drafts: a few rows each, odd sizes, blocks that are partly filled, the other type
        dict(name="append 7 drafted rows", kind="append", B=33, Nt=7, even=False, Hkv=5, D=64, page=32, before=1000,
             codes="int8", dtype="fp16"),
        # a beam step of a few sequences: dropped, forked again, and one sequence admitted
        dict(name="pages turnover, 8 forks", kind="turnover", forks=8, admit=1, layers=1, Hkv=8, D=128, page=16, longest=1000,
             pages=2048),
        # the same of a large batch with long tables, in a pool of several layers
        dict(name="pages turnover, 192 forks", kind="turnover", forks=192, admit=32, layers=4, Hkv=8, D=128, page=64, longest=8192,
             pages=16384),
        # a small pool squeezed
        dict(name="pages compact 512", kind="compact", slots=8, layers=1, Hkv=2, D=64, page=16, pages=512, live=0.5),
        # a pool of a few GB, three quarters full, before its tail is given back
        dict(name="pages compact 16384", kind="compact", slots=64, layers=2, Hkv=8, D=128, page=64, pages=16384, live=0.75),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "append", "turnover", "compact"])
    codes, dtype = rng.choice(["e4m3", "int8"]), rng.choice(["bf16", "fp16"])
    heads = dict(Hkv=rng.choice([1, 2, 3, 4, 5, 8]), D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]))
    if kind == "attend":
        c = dict(kind=kind, **heads, G=rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), codes=codes, dtype=dtype, shared=0, even=rng.random() < 0.3)
        c["Nq"] = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 1024)])
        c["B"] = _log(rng, 1, 64) if c["Nq"] < 10 else rng.randint(1, 4)
        c["longest"] = _log(rng, 1, 131072)
        top = {w["name"]: work(w) for w in listed()}
        while work(c)["bytes"] > top["attend 4 x 131072"]["bytes"] or work(c)["flops"] > top["attend chunk 1024 of 16384"]["flops"] \
                or c["B"] * c["Nq"] * c["Hkv"] * c["G"] * c["longest"] > 1 << 30:
            c["longest"] = c["longest"] * 2 // 3
            if c["longest"] < 64:
                c["Nq"] = c["Nq"] // 2 + 1
        if c["Nq"] > 9 and c["longest"] > 1000:
            c["shared"] = c["longest"] // 2 // c["page"] * c["page"]
        return c
    if kind == "append":
        c = dict(kind=kind, **heads, B=_log(rng, 1, 64), Nt=_log(rng, 1, 2048), even=rng.random() < 0.5, before=rng.choice([0, _log(rng, 1, 8000)]),
                 codes=codes, dtype=dtype)
        c["Nt"] = max(1, min(c["Nt"], 16384 // c["B"]))
        return c
    if kind == "turnover":
        c = dict(kind=kind, forks=_log(rng, 1, 192), admit=rng.randint(1, 32), layers=rng.randint(1, 4), longest=_log(rng, 40, 8192), **heads)
        more = rng.randint(2, 4) * (c["forks"] + 2 * c["admit"] + 4) * 4
    else:
        c = dict(kind=kind, slots=rng.randint(1, 64), layers=rng.randint(1, 2), pages=_log(rng, 64, 16384), live=rng.choice([0.0, 0.1, 0.5, 0.75, 0.95, 1.0]),
                 **heads)
        c["slots"] = min(c["slots"], c["pages"])
    if kind == "turnover":
        c["pages"] = more + (8 + c["admit"]) * (c["longest"] // c["page"] + 2)
    while c["pages"] * c["layers"] * c["Hkv"] * c["D"] * c["page"] > 1 << 31:
        c["layers"], c["page"] = max(1, c["layers"] - 1), max(16, c["page"] // 2)
        if kind == "turnover":
            c["pages"] = more + (8 + c["admit"]) * (c["longest"] // c["page"] + 2)
    return c


# ---------------------------------------------------------------------------------------------------
# inputs

def _lengths(c, top, low=1):
    """Lengths of a batch: all `top`, or spread from `low` to it; the same for every seed, as the case's cost is."""
    B = c["B"]
    return [top if c["even"] or B == 1 else low + (top - low) * ((i * 37 + 11) % B) // (B - 1) for i in range(B)]


def _pages_of(n, page):
    return -(-n // page)


def _values(g, shape, dtype):
    """Rows as a projection gives them: about normal, channels of unlike size, now and then a token that stands out."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.7 * torch.randn(shape[-1], generator=g, device="cuda"))
    far = torch.rand(shape[:-1], generator=g, device="cuda") > 0.995
    x *= torch.where(far, 9.0, 1.0).unsqueeze(-1)
    return x.to(dtype)


def _to_codes(x, codes):
    """Codes and scales of whole blocks x [..., rows, D], as an earlier append has left them."""
    top = x.float().unflatten(-2, (-1, BLOCK)).abs().amax((-1, -2))
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp_min(2.0 ** -100) / QMAX[codes])))
    y = x.float() / scale.repeat_interleave(BLOCK, -1).unsqueeze(-1)
    y = y.clamp(-QMAX[codes], QMAX[codes])
    return (y.to(CODE[codes]) if codes == "e4m3" else torch.round(y).to(torch.int8)), scale


def _pools(c, g, pages):
    """Pools of random codes and scales, a part of the pages at a time."""
    Hkv, D, page = c["Hkv"], c["D"], c["page"]
    code = lambda: torch.empty((pages, Hkv, page, D), dtype=CODE[c["codes"]], device="cuda")  # noqa: E731
    scale = lambda: torch.empty((pages, Hkv, page // BLOCK), dtype=torch.float32, device="cuda")  # noqa: E731
    got = [code(), code(), scale(), scale()]
    step = max(1, (1 << 27) // (Hkv * page * D))
    for i in (0, 1):
        for at in range(0, pages, step):
            n = min(step, pages - at)
            x, s = _to_codes(_values(g, (n, Hkv, page, D), torch.float32), c["codes"])
            got[i][at:at + n], got[2 + i][at:at + n] = x, s
    return got


def _prepare_attend(c, g):
    B, Nq, Hkv, G, D, page = c["B"], c["Nq"], c["Hkv"], c["G"], c["D"], c["page"]
    lens = _lengths(c, c["longest"])
    common = c["shared"] // page
    need = [max(0, _pages_of(n, page) - common) for n in lens]
    pages = common + sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(1, _pages_of(max(lens), page)) + 1), -1, dtype=torch.int32, device="cuda")
    at = common
    for b, n in enumerate(need):
        m = min(common, _pages_of(lens[b], page))
        table[b, :m] = order[:m]
        table[b, common:common + n] = order[at:at + n]
        at += n
    kp, vp, ks, vs = _pools(c, g, pages)
    return dict(c, q=_values(g, (B, Nq, Hkv * G, D), FLOAT[c["dtype"]]), k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs, table=table,
                seqlens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def _append_lens(c):
    new = _lengths(c, c["Nt"], 0)
    before = [max(0, c["before"] - (i * 29) % 64) if c["before"] else 0 for i in range(c["B"])]
    return before, new


def _prepare_append(c, g):
    B, Hkv, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    before, new = _append_lens(c)
    # only the pages that this call reaches are given places of their own: the others of a sequence share page 0
    first = [n // page for n in before]
    last = [_pages_of(n + m, page) for n, m in zip(before, new)]
    pages = 1 + sum(max(0, z - a) for a, z in zip(first, last))
    order = (1 + torch.randperm(pages - 1, generator=g, device="cuda")).to(torch.int32) if pages > 1 else torch.zeros(0, dtype=torch.int32, device="cuda")
    table = torch.zeros((B, max(1, max(last))), dtype=torch.int32, device="cuda")
    at = 0
    for b, (a, z) in enumerate(zip(first, last)):
        if z > a:
            table[b, a:z] = order[at:at + z - a]
            at += z - a
    kp, vp, ks, vs = _pools(c, g, pages)
    k, v = (_values(g, (B, c["Nt"], Hkv, D), FLOAT[c["dtype"]]) for _ in range(2))
    return dict(c, k=k, v=v, k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs, table=table,
                seqlens=torch.tensor([n + m for n, m in zip(before, new)], dtype=torch.int32, device="cuda"),
                new=torch.tensor(new, dtype=torch.int32, device="cuda"))


def _page_pools(c, g):
    """The pools of a model's layers, as bytes and scales: what is in them is any bits to these operations."""
    Hkv, D, page, pages = c["Hkv"], c["D"], c["page"], c["pages"]
    pools = []
    for _ in range(c["layers"]):
        pools += [torch.randint(-128, 128, (pages, Hkv, page, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
        pools += [torch.rand((pages, Hkv, page // BLOCK), generator=g, device="cuda") for _ in range(2)]
    return pools


def _turnover_lens(c):
    """(lengths of the parents, of the forks' parents by index, of the admitted sequences)."""
    parents = [max(1, c["longest"] - 41 * i) for i in range(8)]
    return parents, [i % 8 for i in range(c["forks"])], [1 + (c["page"] * 3 + 5 * i) % (4 * c["page"]) for i in range(c["admit"])]


def _prepare_turnover(c, g):
    """Parents in the first slots, their forks behind them, then the admitted ones: the state that one pass leaves behind
    when it begins with it, so that every pass does the same work."""
    page, pages = c["page"], c["pages"]
    parents, of, admitted = _turnover_lens(c)
    n_par = sum(_pages_of(n, page) for n in parents)
    # the parents' pages are spread over the pool's first part, holes between them
    spread = min(pages, 2 * n_par)
    own_pages = torch.randperm(spread, generator=g, device="cuda")[:n_par].to(torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[own_pages.long()] = 1
    free = torch.nonzero(refs == 0).flatten().to(torch.int32)
    slots = 8 + c["forks"] + c["admit"]
    cols = _pages_of(max(parents + admitted), page) + 1
    table = torch.full((slots, cols), -1, dtype=torch.int32, device="cuda")
    at = taken = 0
    for i, n in enumerate(parents):
        m = _pages_of(n, page)
        table[i, :m] = own_pages[at:at + m]
        at += m
    for i, p in enumerate(of):
        full = parents[p] // page
        table[8 + i, :full] = table[p, :full]
        refs.index_add_(0, table[p, :full].long(), torch.ones(full, dtype=torch.int32, device="cuda"))
        if parents[p] % page:
            table[8 + i, full] = free[taken]
            taken += 1
    for i, n in enumerate(admitted):
        m = _pages_of(n, page)
        table[8 + c["forks"] + i, :m] = free[taken:taken + m]
        taken += m
    refs[free[:taken].long()] = 1
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pools = _page_pools(c, g)
    return dict(c, table=table, refs=refs, pools=pools, seqlens=ints(parents + [parents[p] for p in of] + admitted),
                drop=ints(list(range(8, slots))), src=ints(of), dst=ints(list(range(8, 8 + c["forks"]))),
                enter=ints(list(range(8 + c["forks"], slots))), add=ints(admitted))


def _compact_lens(c):
    live = int(c["pages"] * c["live"])
    per = [live // c["slots"] + (i < live % c["slots"]) for i in range(c["slots"])]
    return live, [max(0, n * c["page"] - (7 * i) % c["page"]) for i, n in enumerate(per)]


def _prepare_compact(c, g):
    page, pages, slots = c["page"], c["pages"], c["slots"]
    live, lens = _compact_lens(c)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((slots, max(1, _pages_of(max(lens), page))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(lens):
        m = _pages_of(n, page)
        table[i, :m] = order[at:at + m]
        at += m
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:live].long()] = 1
    return dict(c, table=table, refs=refs, pools=_page_pools(c, g), seqlens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"attend": _prepare_attend, "append": _prepare_append, "turnover": _prepare_turnover, "compact": _prepare_compact}[case["kind"]](case, g)


# ---------------------------------------------------------------------------------------------------
# plain forms

def _rows(pages, scales, table):
    """The cached rows of each sequence in key order, [B, Hkv, keys, D], in 32 bits."""
    at = table.clamp_min(0).long()
    x = pages.view(torch.int8)[at].view(pages.dtype).float() * scales[at].repeat_interleave(BLOCK, -1).unsqueeze(-1)
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    q = s["q"]
    B, Nq, Hq, D = q.shape
    Hkv = s["Hkv"]
    K, V = _rows(s["k_pages"], s["k_scales"], s["table"]), _rows(s["v_pages"], s["v_scales"], s["table"])
    n = s["seqlens"].long().view(B, 1, 1, 1)
    key = torch.arange(K.shape[2], device="cuda")
    V = torch.where((key < s["seqlens"].long().view(B, 1, 1)).unsqueeze(-1), V, 0.0)
    qs = q.float().view(B, Nq, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = (qs @ K.transpose(2, 3)) * (1.0 / math.sqrt(D))
    token = torch.arange(Nq, device="cuda").repeat_interleave(Hq // Hkv).view(-1, 1)
    x = torch.where(key <= n - Nq + token, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    o = (x @ V) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).squeeze(-1)
    back = lambda t: t.unflatten(2, (Nq, Hq // Hkv))  # noqa: E731
    return {"o": back(o).permute(0, 2, 1, 3, 4).reshape(B, Nq, Hq, D).to(q.dtype), "lse": back(lse).transpose(2, 3).reshape(B, Hq, Nq)}


def _power(top, qmax):
    """The smallest power of two s with top <= qmax s, at least 2^-126."""
    m, e = torch.frexp(torch.where(top > 0, top, 1.0))
    e = e + torch.where(m > math.frexp(qmax)[0], 1, 0) - math.frexp(qmax)[1]
    e = torch.where(top > 0, e, -126).clamp_min(-126)
    return torch.exp2(e.double()).float()


def _plain_append_one(s, x, pages, scales):
    page, codes, D = s["page"], s["codes"], s["D"]
    B, Nt = x.shape[:2]
    end, new = s["seqlens"].long(), s["new"].long()
    first = (end - new) // BLOCK * BLOCK                                 # first row of the first block that is written
    span = (Nt + 2 * BLOCK - 2) // BLOCK * BLOCK                         # rows of the blocks that Nt new ones can reach
    key = first.view(B, 1) + torch.arange(span, device="cuda")
    is_new = (key >= (end - new).view(B, 1)) & (key < end.view(B, 1))
    is_old = key < (end - new).view(B, 1)
    written = is_new.unflatten(1, (-1, BLOCK)).any(2)                    # [B, blocks]
    at = s["table"].long().gather(1, (key // page).clamp_max(s["table"].shape[1] - 1))
    row = key % page
    block, blk = at[:, ::BLOCK], row[:, ::BLOCK] // BLOCK
    old_scale = scales[block, :, blk]                                    # [B, blocks, Hkv]
    bits = pages.view(torch.int8)
    held = bits[at, :, row]
    old = held.view(pages.dtype).float()                                      # [B, span, Hkv, D]
    given = x.float().gather(1, (key - (end - new).view(B, 1)).clamp(0, Nt - 1).view(B, span, 1, 1).expand(-1, -1, *x.shape[2:]))
    given = torch.where(is_new.view(B, span, 1, 1), given, 0.0)
    has_old = is_old.unflatten(1, (-1, BLOCK)).any(2).unsqueeze(-1)
    scale = _power(given.unflatten(1, (-1, BLOCK)).abs().amax((2, 4)), QMAX[codes])
    scale = torch.where(has_old, torch.maximum(scale, old_scale), scale)
    by = lambda t: t.repeat_interleave(BLOCK, 1).unsqueeze(-1)  # noqa: E731
    y = torch.where(is_new.view(B, span, 1, 1), given / by(scale), old * by(old_scale / scale)).clamp(-QMAX[codes], QMAX[codes])
    y = y.to(torch.float8_e4m3fn) if codes == "e4m3" else torch.round(y).to(torch.int8)
    keep = ~(is_new | (is_old & written.repeat_interleave(BLOCK, 1)))
    # rows that are left as they were are written back as they were
    y = torch.where(keep.view(B, span, 1, 1), held, y.view(torch.int8))
    some = torch.nonzero(~keep, as_tuple=True)
    bits[at[some], :, row[some]] = y[some]
    some = torch.nonzero(written, as_tuple=True)
    scales[block[some], :, blk[some]] = scale[some]


def _plain_append(s):
    _plain_append_one(s, s["k"], s["k_pages"], s["k_scales"])
    _plain_append_one(s, s["v"], s["v_pages"], s["v_scales"])
    return {n: s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales")}


def _free_list(refs):
    """The free pages from the lowest on (then -1), without waiting for their number."""
    free = refs == 0
    place = torch.where(free, torch.cumsum(free, 0) - 1, refs.numel())
    out = torch.full((refs.numel() + 1,), -1, dtype=torch.int32, device="cuda")
    return out.scatter_(0, place, torch.arange(refs.numel(), dtype=torch.int32, device="cuda"))


def _plain_turnover(s):
    table, refs, seqlens, page = s["table"], s["refs"], s["seqlens"], s["page"]
    col = torch.arange(table.shape[1], device="cuda")
    count = lambda n: (n.long() + page - 1) // page  # noqa: E731
    # free
    drop = s["drop"].long()
    held = col < count(seqlens[drop]).view(-1, 1)
    gone = torch.where(held, table[drop], 0).long().flatten()
    refs.index_add_(0, gone, -held.flatten().int())
    table[drop], seqlens[drop] = -1, 0
    # fork
    src, dst = s["src"].long(), s["dst"].long()
    n = seqlens[src].long()
    partial = n % page != 0
    fresh = _free_list(refs)[torch.where(partial, torch.cumsum(partial, 0) - 1, refs.numel())]
    row = table[src]
    full = col < (n // page).view(-1, 1)
    refs.index_add_(0, torch.where(full, row, 0).long().flatten(), full.flatten().int())
    last = (n // page).view(-1, 1)
    origin = row.gather(1, last.clamp_max(table.shape[1] - 1)).flatten().long()
    table[dst] = torch.where(full, row, torch.where((col == last) & partial.view(-1, 1), fresh.view(-1, 1), -1))
    seqlens[dst] = seqlens[src]
    pick = torch.nonzero(partial).flatten()
    to, frm = fresh[pick].long(), origin[pick]
    refs[to] = 1
    for pool in s["pools"]:
        pool[to] = pool[frm]
    # extend
    enter, add = s["enter"].long(), s["add"].long()
    a, z = count(seqlens[enter]), count(seqlens[enter].long() + add)
    start = torch.cumsum(z - a, 0) - (z - a)
    new = (col >= a.view(-1, 1)) & (col < z.view(-1, 1))
    rank = torch.where(new, start.view(-1, 1) + col - a.view(-1, 1), refs.numel())
    got = _free_list(refs)[rank]
    table[enter] = torch.where(new, got, table[enter])
    refs.index_add_(0, torch.where(new, got, 0).long().flatten(), new.flatten().int())
    seqlens[enter] += s["add"]
    return {"table": table, "refs": refs, "seqlens": seqlens, "pools": [p if p.is_floating_point() else p.view(torch.int8) for p in s["pools"]]}


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    live = refs > 0
    n_live = live.sum(dtype=torch.int32)
    page = torch.arange(refs.numel(), device="cuda")
    movers, holes = torch.nonzero(live & (page >= n_live)).flatten(), torch.nonzero(~live & (page < n_live)).flatten()
    remap = torch.where(live, page, -1).to(torch.int32)
    remap[movers] = holes.to(torch.int32)
    new_refs = torch.where(page < n_live, refs, 0)
    new_refs[holes] = refs[movers]
    held = torch.arange(table.shape[1], device="cuda") < ((s["seqlens"].long() + s["page"] - 1) // s["page"]).view(-1, 1)
    new_table = torch.where(held, remap[torch.where(held, table, 0).long()], table)
    for pool in s["pools"]:
        pool[holes] = pool[movers]
    return {"table": new_table, "refs": new_refs, "remap": remap, "n_live": n_live.view(1), "pools": list(s["pools"])}


# ---------------------------------------------------------------------------------------------------
# a pass

def run(s):
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "turnover": _plain_turnover, "compact": _plain_compact}[s["kind"]](s)
    import exact_tiled_attention_47_b200 as fa
    if s["kind"] == "attend":
        o, lse = fa.attend_kv8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"], s["seqlens"])
        return {"o": o, "lse": lse}
    if s["kind"] == "append":
        fa.append_kv8(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"], s["seqlens"], s["new"])
        return {n: s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales")}
    if s["kind"] == "turnover":
        fa.free_pages(s["table"], s["seqlens"], s["refs"], s["page"], s["drop"])
        fa.fork_pages(s["table"], s["seqlens"], s["refs"], s["page"], s["src"], s["dst"], s["pools"])
        fa.extend_pages(s["table"], s["seqlens"], s["refs"], s["page"], s["add"], s["enter"])
        return {"table": s["table"], "refs": s["refs"], "seqlens": s["seqlens"], "pools": list(s["pools"])}
    table, refs, remap, n_live = fa.compact_pages(s["table"], s["seqlens"], s["refs"], s["page"], s["pools"])
    return {"table": table, "refs": refs, "remap": remap, "n_live": n_live, "pools": list(s["pools"])}


# ---------------------------------------------------------------------------------------------------
# what a pass cannot do without

def _page_bytes(c):
    return c["layers"] * 2 * c["Hkv"] * (c["page"] * c["D"] + c["page"] // BLOCK * 4)


def work(case):
    c = case
    if c["kind"] == "attend":
        lens = _lengths(c, c["longest"])
        shared = c["shared"]
        keys = sum(lens) - sum(min(shared, n) for n in lens) + min(shared, max(lens))
        pairs = sum(max(0, n - c["Nq"] + i + 1) for n in lens for i in range(c["Nq"])) if c["Nq"] < 10 else \
            sum((n - c["Nq"]) * c["Nq"] + c["Nq"] * (c["Nq"] + 1) // 2 if n >= c["Nq"] else n * (n + 1) // 2 for n in lens)
        Hq = c["Hkv"] * c["G"]
        rows = c["B"] * c["Nq"] * Hq
        return {"bytes": keys * c["Hkv"] * 2 * (c["D"] + 4 / BLOCK) + rows * (2 * c["D"] * 2 + 4) + sum(_pages_of(n, c["page"]) for n in lens) * 4,
                "flops": 4.0 * c["D"] * Hq * pairs}
    if c["kind"] == "append":
        before, new = _append_lens(c)
        rows = sum(new)
        blocks = sum(_pages_of(a + n, BLOCK) - a // BLOCK for a, n in zip(before, new) if n)
        return {"bytes": 2 * c["Hkv"] * (rows * c["D"] * 3 + blocks * 4), "flops": 2.0 * 2 * c["Hkv"] * rows * c["D"]}
    if c["kind"] == "turnover":
        parents, of, admitted = _turnover_lens(c)
        moved = sum(1 for p in of if parents[p] % c["page"])
        entries = sum(parents[p] // c["page"] + 1 for p in of) + sum(_pages_of(n, c["page"]) for n in admitted)
        return {"bytes": 2 * moved * _page_bytes(c) + entries * 4 * 6, "flops": 0}
    live, lens = _compact_lens(c)
    moved = live * (1 - c["live"])  # live pages that lie behind the first `live` places, on average
    return {"bytes": 2 * moved * _page_bytes(c) + c["pages"] * 12 + sum(_pages_of(n, c["page"]) for n in lens) * 8, "flops": 0}


# ---------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_attend(c, s):
    B, Nq, Hkv, G, D, page = c["B"], c["Nq"], c["Hkv"], c["G"], c["D"], c["page"]
    o = torch.zeros((B, Nq, Hkv * G, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hkv * G, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["seqlens"][b])
        if n == 0:
            continue
        ids = s["table"][b, : (n + page - 1) // page].long()
        for h in range(Hkv):
            def rows(codes, scales):
                x = codes.view(torch.int8)[ids, h].view(codes.dtype).double().reshape(-1, BLOCK, D) * scales[ids, h].double().reshape(-1, 1, 1)
                return x.reshape(-1, D)[:n]
            K, V = rows(s["k_pages"], s["k_scales"]), rows(s["v_pages"], s["v_scales"])
            for i0 in range(0, Nq, 256):  # queries a part at a time: the scores of all would not fit beside them
                i1 = min(Nq, i0 + 256)
                a = torch.einsum("tgd,kd->gtk", s["q"][b, i0:i1, h * G:(h + 1) * G].double(), K) * D ** -0.5
                last = n - Nq + torch.arange(i0, i1, device="cuda")
                a.masked_fill_(torch.arange(n, device="cuda")[None, :] > last[:, None], -math.inf)
                t = torch.logsumexp(a, -1)
                lse[b, h * G:(h + 1) * G, i0:i1] = t
                w = torch.exp(a - torch.where(torch.isinf(t), 0.0, t)[..., None])
                o[b, i0:i1, h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", w, V)
    return {"o": o, "lse": lse}


def _exact_append(c, s):
    """Block by block: the new rows' largest magnitude, its power of two, the rounding to the nearest code."""
    before, new = _append_lens(c)
    page, qmax = c["page"], QMAX[c["codes"]]
    out = {}
    for x, pn, sn in ((s["k"], "k_pages", "k_scales"), (s["v"], "v_pages", "v_scales")):
        codes, scales, table = s[pn].double(), s[sn].double(), s["table"].cpu()
        for b, (a, n) in enumerate(zip(before, new)):
            for blk in range(a // BLOCK, (a + n + BLOCK - 1) // BLOCK if n else 0):
                lo, hi = max(a, blk * BLOCK), min(a + n, (blk + 1) * BLOCK)
                p, r = int(table[b, blk * BLOCK // page]), blk * BLOCK % page
                rows = x[b, lo - a:hi - a].double().transpose(0, 1)              # [Hkv, rows, D]
                top = rows.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -140) / qmax)).long()
                e = torch.where(top > qmax * _two_to(e), e + 1, torch.where(top <= qmax * _two_to(e - 1), e - 1, e)).clamp_min(-126)
                scale = _two_to(e)
                old = lo - blk * BLOCK
                if old:
                    scale = torch.maximum(scale, scales[p, :, r // BLOCK])
                    codes[p, :, r:r + old] = _nearest(codes[p, :, r:r + old] * (scales[p, :, r // BLOCK] / scale)[:, None, None], c["codes"])
                codes[p, :, r + old:r + old + hi - lo] = _nearest(rows / scale[:, None, None], c["codes"])
                scales[p, :, r // BLOCK] = scale
        out[pn], out[sn] = (codes if c["codes"] == "e4m3" else None), scales
    return out


def _two_to(e):
    """2^e in 64 bits, without a rounding."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(y, codes):
    if codes == "int8":
        return torch.round(y).clamp(-127, 127)
    step = _two_to((torch.frexp(y)[1] - 1).clamp_min(-6) - 3)  # three bits behind the leading one, from 2^-6 on
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(case, seed):
    if case["kind"] == "attend":
        return _exact_attend(case, prepare(case, seed))
    if case["kind"] == "append":
        before, new = _append_lens(case)
        if sum(_pages_of(a + n, BLOCK) - a // BLOCK for a, n in zip(before, new) if n) > 4000:
            return None
        return _exact_append(case, prepare(case, seed))
    return None  # whole numbers and copies: nothing is rounded
