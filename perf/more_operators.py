"""Measured cases of a sparse decode step over the paged cache.

Four operators, one case each time:
  tables  update_block_tables: pages taken and given back, slots, positions and
          offsets of a step's tokens from the requests' lengths
  bounds  update_page_bounds: the least and the largest key of every page that
          was written, per channel, in 8 bits with a power-of-two scale
  select  select_pages: for every query the pages whose bounds allow the largest
          scores
  sparse  paged_sparse_attention: attention of every query over its list of pages

``own`` chooses between the plain torch forms and the library's calls.
"""
import math
import random

import torch

own = False

BF16, F32, F64, I32, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64
U8, I8 = torch.uint8, torch.int8
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
NEG = float("-inf")


def listed():
    return [
        # a decode step of 64 requests: one token each, some done, some new
        dict(name="tables-64", op="tables", batch=64, hi=8192, grow=1, bs=16),
        # chunks of prompts beside many decoding requests
        dict(name="tables-1000", op="tables", batch=1000, hi=32768, grow=500, bs=16),
        # the pages of one decode step's tokens
        dict(name="bounds-64", op="bounds", batch=64, hi=4096, grow=1, hkv=8, d=128, bs=16, layout="NHD", kv="bf16"),
        # the pages of long prompts over an 8-bit cache, head-major
        dict(name="bounds-prompts-fp8", op="bounds", batch=13, hi=100, grow=9001, hkv=8, d=128, bs=32, layout="HND",
             kv="e4m3"),
        # three short sequences, where the call's latency counts
        dict(name="select-3", op="select", batch=3, lo=30, hi=700, qlo=1, qhi=1, hq=4, hkv=2, d=64, bs=32, top=8),
        # an ordinary decode batch of long contexts
        dict(name="select-64x32k", op="select", batch=64, lo=8192, hi=32768, qlo=1, qhi=1, hq=32, hkv=8, d=128, bs=16,
             top=64),
        # one context of a million tokens
        dict(name="select-1x1m", op="select", batch=1, lo=1000003, hi=1000003, qlo=1, qhi=1, hq=64, hkv=8, d=128, bs=16,
             top=256),
        # chunks of prompts, every query with pages of its own
        dict(name="select-chunks", op="select", batch=4, lo=16384, hi=32768, qlo=200, qhi=256, hq=32, hkv=8, d=128,
             bs=16, top=64),
        # three short sequences with sinks
        dict(name="sparse-3", op="sparse", batch=3, lo=30, hi=700, qlo=1, qhi=1, hq=4, hkv=2, d=64, bs=32, top=8,
             layout="NHD", kv="bf16", sink=True, lse=True),
        # an ordinary decode batch of long contexts
        dict(name="sparse-64x32k", op="sparse", batch=64, lo=8192, hi=32768, qlo=1, qhi=1, hq=32, hkv=8, d=128, bs=16,
             top=64, layout="NHD", kv="bf16", sink=False, lse=False),
        # longer contexts in an 8-bit cache
        dict(name="sparse-8x128k-fp8", op="sparse", batch=8, lo=32768, hi=131072, qlo=1, qhi=1, hq=64, hkv=8, d=64,
             bs=16, top=256, layout="HND", kv="e4m3", sink=True, lse=True),
        # chunks of prompts, every query with pages of its own
        dict(name="sparse-chunks", op="sparse", batch=4, lo=16384, hi=32768, qlo=200, qhi=256, hq=32, hkv=8, d=128,
             bs=16, top=64, layout="NHD", kv="bf16", sink=False, lse=False),
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) if hi > lo else lo


def draw(rng):
    op = rng.choice(["tables", "bounds", "select", "select", "sparse", "sparse"])
    if op == "tables":
        return dict(op=op, batch=_log(rng, 1, 1000), hi=_log(rng, 16, 32768), grow=_log(rng, 1, 400),
                    bs=rng.choice([16, 32]))
    c = dict(op=op, hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 80, 96, 112, 128]), bs=rng.choice([16, 32]))
    if op == "bounds":
        b = _log(rng, 1, 64)
        c.update(batch=b, hi=_log(rng, 16, 4096), grow=_log(rng, 1, 40000 // b), layout=rng.choice(["NHD", "HND"]),
                 kv=rng.choice(["bf16", "e4m3"]))
        return c
    # a selection has more pages to choose from than it takes
    hi = _log(rng, 64 * c["bs"] if op == "select" else 40, 24000)
    b = _log(rng, 1, 48)
    # one query each, a few drafted ones, or a chunk
    qhi = min(rng.choice([1, 1, _log(rng, 2, 9), _log(rng, 10, 1 + 800 // b)]), hi)
    c.update(batch=b, hi=hi, lo=max(1, hi // rng.choice([1, 3, 10])), qlo=max(1, qhi // 2), qhi=qhi,
             hq=c["hkv"] * rng.choice([n for n in (1, 2, 3, 4, 5, 8, 16) if n * c["hkv"] <= 32]),
             top=_log(rng, 2, 1024 // c["bs"]))
    c["lo"] = max(c["lo"], qhi)
    if op == "select":
        c["lo"] = max(c["lo"], hi // 2)
        c["top"] = _log(rng, 4, min(1024, hi // 2) // c["bs"])
    if op == "sparse":
        c.update(layout=rng.choice(["NHD", "HND"]), kv=rng.choice(["bf16", "e4m3"]), sink=rng.choice([True, False]),
                 lse=rng.choice([True, False]))
    return c


# ---------------------------------------------------------------------------
# what a case's lengths are (from the case alone: work() needs them)
# ---------------------------------------------------------------------------
def _ceil(a, b):
    return (a + b - 1) // b


def _lengths(case):
    """Per request: (length before, length after), or (queries, length)."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    got = []
    for _ in range(case["batch"]):
        if case["op"] in ("tables", "bounds"):
            n, m = rng.randint(1, case["hi"]), rng.randint(_ceil(case["grow"], 2), case["grow"])
            kind = rng.random() if case["op"] == "tables" else 1.0
            if kind < 0.06:
                got.append((min(n, 8 * m), 0))         # a request that is done
            elif kind < 0.12:
                got.append((0, m))                     # a new one
            elif kind < 0.2:
                got.append((n, max(0, n - m)))         # drafted tokens given back
            else:
                got.append((n, n + m))
        else:
            nq = rng.randint(case["qlo"], case["qhi"])
            got.append((nq, max(nq, rng.randint(case["lo"], case["hi"]))))
    return got


def _grown(pairs):
    return sum(max(0, b - a) for a, b in pairs)


def work(case):
    op, bs, pairs = case["op"], case["bs"], _lengths(case)
    if op == "tables":
        moved = sum(abs(_ceil(a, bs) - _ceil(b, bs)) for a, b in pairs)
        back = [(b, a) for a, b in pairs]
        # there and back: lengths in, offsets, slots and positions out, pages read and written
        return {"bytes": 2 * (16 * len(pairs) + 12 * moved) + 16 * (_grown(pairs) + _grown(back)),
                "flops": 8 * (_grown(pairs) + _grown(back))}
    hkv, d = case["hkv"], case["d"]
    if op == "bounds":
        row = 2 * d if case["kv"] == "bf16" else d + 1
        pages = rows = 0
        for a, b in pairs:
            pages += _ceil(b, bs) - a // bs
            rows += b - a // bs * bs
        return {"bytes": hkv * (rows * row + pages * (2 * d + 1)) + 8 * _grown(pairs), "flops": 2 * rows * hkv * d}
    hq, top = case["hq"], case["top"]
    queries = sum(nq for nq, _ in pairs)
    qpages = [[_ceil(n - nq + i + 1, bs) for i in range(nq)] for nq, n in pairs]
    if op == "select":
        pages = sum(_ceil(n, bs) for _, n in pairs)
        return {"bytes": pages * hkv * (2 * d + 1) + queries * (hq * d * 2 + hkv * top * 4),
                "flops": 4 * d * hq * sum(map(sum, qpages))}
    row = 2 * d if case["kv"] == "bf16" else d + 1
    # one query reads its pages; the queries of a chunk at least as many together
    keys = sum(min(n, max(min(p, top) for p in ps) * bs) for (nq, n), ps in zip(pairs, qpages))
    attended = sum(min(p, top) * bs for ps in qpages for p in ps)
    return {"bytes": 2 * keys * hkv * row + queries * (2 * hq * d * 2 + hkv * top * 4),
            "flops": 4 * d * hq * attended}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pow2(e):
    """2^e as float32, from its bits (-126 <= e <= 127)."""
    return ((e.to(I32) + 127) << 23).view(F32)


def _pow2d(e):
    """2^e as float64, from its bits."""
    return ((e.to(I64) + 1023) << 52).view(F64)


def _quantise(x):
    """[..., D] -> (e4m3 codes, E8M0 bytes [...]) with e = ceil(log2(max|x| / 448))."""
    x = x.float()
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)  # a = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(a > 0, e, torch.full_like(e, -126)).clamp(-126, 119)
    return (x * _pow2(-e).unsqueeze(-1)).clamp(-448, 448).to(E4M3), (e + 127).to(U8)


def _table(g, pages, nb, dev):
    """A block table of shuffled pages, and the pages it does not name."""
    perm = torch.randperm(nb, generator=g, device=dev).to(I32)
    npg = torch.tensor(pages, device=dev)
    col = torch.arange(max(pages + [1]), device=dev)
    first = torch.cumsum(npg, 0) - npg
    idx = (first[:, None] + col).clamp(max=nb - 1)
    table = torch.where(col < npg[:, None], perm[idx], torch.full_like(perm[idx], -1)).contiguous()
    return table, perm[sum(pages):]


def _pool(g, nb, case, dev):
    """One pool and its scales, rows whose sizes differ by head and by token."""
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    x = torch.randn(nb, hkv, bs, d, generator=g, device=dev, dtype=BF16)
    x *= torch.exp2(torch.randn(nb, hkv, bs, 1, generator=g, device=dev)).to(BF16) * 0.5
    nhd = case["layout"] == "NHD"
    if case["kv"] == "bf16":
        return (x.permute(0, 2, 1, 3).contiguous() if nhd else x), None
    code, scale = _quantise(x)
    return (code.view(U8).permute(0, 2, 1, 3).contiguous().view(E4M3) if nhd else code), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, bs, pairs = case["op"], case["bs"], _lengths(case)
    s = dict(case=dict(case), op=op, bs=bs, layout=case.get("layout"))

    def i32(x):
        return torch.tensor(x, dtype=I32, device=dev)

    if op in ("tables", "bounds"):
        s["old"], s["new"] = i32([a for a, _ in pairs]), i32([b for _, b in pairs])
        # rows for the new tokens, a multiple of 8 as in a captured step
        s["rows"] = _ceil(_grown(pairs), 8) * 8
    if op == "tables":
        need = [_ceil(a, bs) for a, _ in pairs]
        most = max(max(need), max(_ceil(b, bs) for _, b in pairs))
        nb = sum(_ceil(max(a, b), bs) for a, b in pairs) + 50
        table, spare = _table(g, need, nb, dev)
        s["table"] = torch.full((len(pairs), most + 3), -1, dtype=I32, device=dev)
        s["table"][:, :table.shape[1]] = table
        s["free"] = torch.zeros(nb, dtype=I32, device=dev)
        s["free"][:spare.numel()] = spare
        s["num_free"] = i32([spare.numel()])
        s["rows_back"] = _ceil(_grown([(b, a) for a, b in pairs]), 8) * 8
        return s
    if op == "bounds":
        need = [_ceil(b, bs) for _, b in pairs]
        nb = sum(need) + 5
        table, _ = _table(g, need, nb, dev)
        at = torch.arange(_grown(pairs), device=dev)
        n = (s["new"] - s["old"]).long()
        req = torch.repeat_interleave(torch.arange(len(pairs), device=dev), n)
        pos = s["old"].long()[req] + at - (torch.cumsum(n, 0) - n)[req]
        slots = torch.full((s["rows"],), -1, dtype=I64, device=dev)
        slots[:at.numel()] = table[req, pos // bs].long() * bs + pos % bs
        s["slots"] = slots
        s["kc"], s["ks"] = _pool(g, nb, case, dev)
        s["bounds"] = torch.zeros(nb, case["hkv"], 2, case["d"], dtype=I8, device=dev)
        s["bscale"] = torch.full((nb, case["hkv"]), 120, dtype=U8, device=dev)
        return s
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    need = [_ceil(n, bs) for _, n in pairs]
    nb = sum(need) + 5
    s["table"], _ = _table(g, need, nb, dev)
    s["lens"] = i32([n for _, n in pairs])
    s["max"], s["maxq"] = max(n for _, n in pairs), max(nq for nq, _ in pairs)
    queries = [nq for nq, _ in pairs]
    s["cu"] = None if case["qhi"] == 1 else i32([sum(queries[:i]) for i in range(len(queries) + 1)])
    total = sum(queries)
    size = torch.exp2(torch.randn(total, hq, 1, generator=g, device=dev))
    s["q"] = (torch.randn(total, hq, d, generator=g, device=dev) * size).to(BF16)
    if op == "select":
        mid = torch.randn(nb, hkv, d, generator=g, device=dev) * 24
        half = 20 + 8 * torch.randn(nb, hkv, d, generator=g, device=dev).abs()
        s["bounds"] = torch.stack([(mid - half).floor(), (mid + half).ceil()], 2).clamp(-127, 127).to(I8)
        s["bscale"] = torch.randint(121, 124, (nb, hkv), generator=g, device=dev).to(U8)
        return s
    s["kc"], s["ks"] = _pool(g, nb, case, dev)
    s["vc"], s["vs"] = _pool(g, nb, case, dev)
    s["sink"] = torch.randn(hq, generator=g, device=dev) if case["sink"] else None
    s["scale"] = d ** -0.5
    # lists of pages: a request's queries agree on most of them; the first and the last always
    req, length = _rows(s)
    n = (length + bs - 1) // bs
    col = torch.arange(max(need), device=dev)
    field = torch.randn(len(pairs), hkv, col.numel(), generator=g, device=dev)
    lists = []
    for at in torch.arange(total, device=dev).split(256):
        x = field[req[at]] + 0.5 * torch.randn(at.numel(), hkv, col.numel(), generator=g, device=dev)
        last = n[at][:, None, None]
        x = torch.where((col == 0) | (col == last - 1), torch.full_like(x, 1e9), x)
        x = x.masked_fill(col >= last, NEG)
        val, idx = torch.topk(x, min(case["top"], col.numel()), -1)
        idx = torch.where(val == NEG, torch.full_like(idx, 1 << 30), idx).sort(-1).values
        lists.append(torch.where(idx == 1 << 30, torch.full_like(idx, -1), idx))
    pages = torch.cat(lists)
    s["pages"] = torch.full((total, hkv, case["top"]), -1, dtype=I32, device=dev)
    s["pages"][..., :pages.shape[-1]] = pages.to(I32)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rows(s):
    """Per query: its request, and how many keys there are up to and with its own."""
    lens = s["lens"].long()
    if s["cu"] is None:
        return torch.arange(lens.numel(), device=lens.device), lens
    cu = s["cu"].long()
    at = torch.arange(s["q"].shape[0], device=cu.device)
    req = torch.searchsorted(cu[1:], at, right=True)
    return req, lens[req] - (cu[1:] - cu[:-1])[req] + (at - cu[req]) + 1


def _plain_tables(s, old, new, rows):
    bs, table, free = s["bs"], s["table"].long(), s["free"]
    old, new = old.long(), new.long()
    have, want = ((old + bs - 1) // bs)[:, None], ((new + bs - 1) // bs)[:, None]
    col = torch.arange(table.shape[1], device=table.device)
    gone, fresh = (col >= want) & (col < have), (col >= have) & (col < want)
    nth = (torch.cumsum(gone.flatten(), 0) - 1).view_as(table)     # the released pages, in order
    jth = (torch.cumsum(fresh.flatten(), 0) - 1).view_as(table)    # the places that take pages
    released, taken, held = gone.sum(), fresh.sum(), s["num_free"].long()
    spare = table.numel()
    back = torch.zeros(spare + 1, dtype=I64, device=table.device)
    back.scatter_(0, torch.where(gone, nth, spare).flatten(), table.flatten())
    top = free.long()[(held - 1 - (jth - released)).clamp(0, free.numel() - 1)]
    page = torch.where(jth < released, back[jth.clamp(0, spare)], top)
    # what is left of the released pages goes on the stack, the first of them topmost
    stack = torch.cat([free, free[:1]])
    at = torch.where(gone & (nth >= taken), held + released - 1 - nth, free.numel())
    stack.scatter_(0, at.flatten(), table.flatten().to(I32))
    free.copy_(stack[:-1])
    s["num_free"].copy_(held + released - taken)
    table = torch.where(fresh, page, torch.where(gone, -1, table))
    s["table"].copy_(table)
    cu = torch.zeros(2, old.numel() + 1, dtype=I64, device=old.device)
    cu[0, 1:] = torch.cumsum((new - old).clamp(min=0), 0)
    cu[1, 1:] = torch.cumsum(new, 0)
    at = torch.arange(rows, device=old.device)
    req = torch.searchsorted(cu[0, 1:], at, right=True)
    live = req < old.numel()
    req = req.clamp(max=old.numel() - 1)
    pos = torch.where(live, old[req] + at - cu[0, req], 0)
    slot = table[req, (pos // bs).clamp(max=table.shape[1] - 1)] * bs + pos % bs
    return [torch.where(live, slot, -1), pos, cu[0].to(I32), cu[1].to(I32)]


def _pages_of(s, pool, scale, blk, head):
    """[..., bs, D] float32 of pages `blk` and kv heads `head` (broadcast together)."""
    x = pool.view(U8) if scale is not None else pool
    if s["layout"] == "NHD":
        x = x.permute(0, 2, 1, 3)
    x = x[blk, head]
    if scale is None:
        return x.float()
    e = scale[blk, head].to(I32)
    m = torch.where(e == 255, torch.full((), float("nan"), device=x.device), _pow2(e.clamp(max=254) - 127))
    return x.view(E4M3).float() * m.unsqueeze(-1)


def _plain_bounds(s):
    bs, hkv = s["bs"], s["case"]["hkv"]
    slots = s["slots"][s["slots"] >= 0]
    blk, inv = torch.unique(slots // bs, return_inverse=True)
    rows = torch.zeros(blk.numel(), dtype=I64, device=blk.device).scatter_reduce_(0, inv, slots % bs + 1, "amax")
    head = torch.arange(hkv, device=blk.device)
    for b, n in zip(blk.split(4096), rows.split(4096)):
        x = _pages_of(s, s["kc"], s["ks"], b[:, None], head)
        held = (torch.arange(bs, device=b.device) < n[:, None])[:, None, :, None]
        lo = torch.where(held, x, float("inf")).amin(2)
        hi = torch.where(held, x, NEG).amax(2)
        a = torch.maximum(lo.abs(), hi.abs()).amax(-1)
        ok = torch.isfinite(a)
        m, e = torch.frexp(a)  # 127 = 0.9921875 * 2^7
        e = torch.where(m > 0.9921875, e - 6, e - 7)
        e = torch.where(ok & (a > 0), e, torch.full_like(e, -126)).clamp(min=-126)
        code = torch.stack([lo, hi], 2).double() * _pow2d(-e)[..., None, None]
        code = torch.stack([code[:, :, 0].floor(), code[:, :, 1].ceil()], 2)
        s["bounds"][b] = torch.where(ok[..., None, None], code, torch.zeros_like(code)).to(I8)
        s["bscale"][b] = torch.where(ok, e + 127, torch.full_like(e, 255)).to(U8)
    return [s["bounds"], s["bscale"].view(E8M0)]


def _spread(s, x):
    """Rows [total, ...] as [B, maxq, ...]."""
    if s["cu"] is None:
        return x[:, None]
    at = s["cu"][:-1, None].long() + torch.arange(s["maxq"], device=x.device)
    return x[at.clamp(max=x.shape[0] - 1)]


def _plain_select(s):
    c, bs = s["case"], s["bs"]
    hq, hkv, d, top = c["hq"], c["hkv"], c["d"], c["top"]
    req, length = _rows(s)
    q = s["q"].float()
    e = (torch.frexp(q.abs().amax(-1)).exponent - 1).clamp(min=-112) - 7
    code = torch.round(q * _pow2(-e)[..., None])
    code = torch.cat([code.clamp(max=0), code.clamp(min=0)], -1)            # for the lower, the upper bounds
    n = (s["max"] + bs - 1) // bs
    blk = s["table"][:, :n].long().clamp(min=0)
    bound = s["bounds"][blk].float().permute(0, 2, 1, 3, 4).flatten(3)     # [B, Hkv, n, 2D]
    code, ex = _spread(s, code), _spread(s, e)
    b, t = code.shape[:2]
    code = code.view(b, t, hkv, hq // hkv, 2 * d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, 2 * d)
    prod = (code @ bound.transpose(2, 3)).view(b, hkv, t, hq // hkv, n)    # whole numbers below 2^24
    ex = ex.view(b, t, hkv, hq // hkv).permute(0, 2, 1, 3)
    size = _pow2d(s["bscale"][blk].to(I32) - 127).transpose(1, 2)          # [B, Hkv, n]
    score = (prod * _pow2d(ex)[..., None]).amax(3) * size[:, :, None]
    score = score.float().permute(0, 2, 1, 3)                              # [B, maxq, Hkv, n]
    if s["cu"] is None:
        score = score[:, 0]
    else:
        score = score[req, torch.arange(req.numel(), device=req.device) - s["cu"].long()[req]]
    own_pages = ((length + bs - 1) // bs)[:, None, None]
    col = torch.arange(n, device=score.device)
    score = torch.where((col == 0) | (col == own_pages - 1), float("inf"), score)
    score = score.masked_fill(col >= own_pages, NEG)
    at = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    at = torch.where(at < own_pages, at, n).sort(-1).values
    pages = torch.full((req.numel(), hkv, top), -1, dtype=I32, device=at.device)
    pages[..., :at.shape[-1]] = torch.where(at < n, at, -1).to(I32)
    return [pages]


def _plain_sparse(s):
    c, bs = s["case"], s["bs"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    req, length = _rows(s)
    head = torch.arange(hkv, device=req.device)[:, None]
    outs, lses = [], []
    for at in torch.arange(req.numel(), device=req.device).split(64):
        pages = s["pages"][at].long()                                       # [t, Hkv, top]
        r = req[at][:, None, None]
        blk = s["table"][r, pages.clamp(min=0)].long().clamp(min=0)
        pos = pages[..., None] * bs + torch.arange(bs, device=req.device)
        keep = (pages >= 0)[..., None] & (pos < length[at][:, None, None, None])
        zero = torch.zeros((), device=req.device)
        k, v = [torch.where(keep[..., None], _pages_of(s, p, sc, blk, head), zero).flatten(2, 3)
                for p, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]      # [t, Hkv, top * bs, D]
        q = s["q"][at].float().view(-1, hkv, hq // hkv, d)
        x = (q @ k.transpose(2, 3) * s["scale"]).masked_fill(~keep.flatten(2)[:, :, None], NEG)
        m = x.amax(-1, keepdim=True)
        if s["sink"] is not None:
            sink = s["sink"].view(1, hkv, hq // hkv, 1)
            m = torch.maximum(m, sink)
        m = torch.where(m == NEG, torch.zeros_like(m), m)
        p = torch.exp(x - m)
        z = p.sum(-1, keepdim=True)
        if s["sink"] is not None:
            z = z + torch.exp(sink - m)
        o = p @ v
        outs.append(torch.where(z > 0, o / z, torch.zeros_like(o)).reshape(-1, hq, d).to(BF16))
        lses.append((torch.log(z) + m).reshape(-1, hq))
    return [torch.cat(outs), torch.cat(lses)] if c["lse"] else [torch.cat(outs)]


def run(s):
    op, c = s["op"], s["case"]
    if own:
        import paged_kv_cache_attention_gb300 as pkv
        if op == "tables":
            there = pkv.update_block_tables(s["table"], s["old"], s["new"], s["free"], s["num_free"], s["bs"],
                                            s["rows"])
            back = pkv.update_block_tables(s["table"], s["new"], s["old"], s["free"], s["num_free"], s["bs"],
                                           s["rows_back"])
            return [*there, *back, s["table"], s["free"], s["num_free"]]
        if op == "bounds":
            pkv.update_page_bounds(s["kc"], s["bounds"], s["bscale"], s["slots"], k_scale=s["ks"],
                                   layout=s["layout"])
            return [s["bounds"], s["bscale"].view(E8M0)]
        if op == "select":
            return [pkv.select_pages(s["q"], s["bounds"], s["bscale"], s["table"], s["lens"], s["max"], c["top"],
                                     s["bs"], cu_seq_lens_q=s["cu"])]
        lse = torch.empty(s["q"].shape[:2], device=s["q"].device) if c["lse"] else None
        o = pkv.paged_sparse_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["pages"],
                                       cu_seq_lens_q=s["cu"], k_scale=s["ks"], v_scale=s["vs"], sink=s["sink"],
                                       sm_scale=s["scale"], lse=lse, layout=s["layout"])
        return [o, lse] if c["lse"] else [o]
    if op == "tables":
        # lengths before -> after, and back again: every pass starts from the same tables
        there = _plain_tables(s, s["old"], s["new"], s["rows"])
        back = _plain_tables(s, s["new"], s["old"], s["rows_back"])
        return [*there, *back, s["table"], s["free"], s["num_free"]]
    if op == "bounds":
        return _plain_bounds(s)
    return _plain_select(s) if op == "select" else _plain_sparse(s)


# ---------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_step(table, free, pairs, bs, rows):
    """One step on Python lists, token by token."""
    gone = []
    for r, (a, b) in enumerate(pairs):
        for p in range(_ceil(b, bs), _ceil(a, bs)):
            gone.append(table[r][p])
            table[r][p] = -1
    free.extend(reversed(gone))
    slots, pos, cuq, cuk = [], [], [0], [0]
    for r, (a, b) in enumerate(pairs):
        for p in range(_ceil(a, bs), _ceil(b, bs)):
            table[r][p] = free.pop()
        for x in range(a, b):
            slots.append(table[r][x // bs] * bs + x % bs)
            pos.append(x)
        cuq.append(len(slots))
        cuk.append(cuk[-1] + b)
    return [slots + [-1] * (rows - len(slots)), pos + [0] * (rows - len(pos)), cuq, cuk]


def _exact_pool(s, pool, scale):
    """A pool in float64 as [num_blocks, Hkv, bs, D] (8-bit ones by a table of the codes' values)."""
    if scale is None:
        x = pool.double()
    else:
        code = torch.arange(256, device=pool.device)
        ex, man = (code >> 3) & 15, code & 7
        val = torch.where(ex == 0, man / 8.0 * 2.0 ** -6, (1 + man / 8.0) * _pow2d(ex - 7))
        val = torch.where(code >= 128, -val, val).double()
        x = val[pool.view(U8).long()]
    if s["layout"] == "NHD":
        x = x.transpose(1, 2)
    return x if scale is None else x * _pow2d(scale.to(I64) - 127)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    op, bs, pairs = case["op"], case["bs"], _lengths(case)
    if op == "tables":
        table = s["table"].tolist()
        free = s["free"][:int(s["num_free"])].tolist()
        there = _exact_step(table, free, pairs, bs, s["rows"])
        back = _exact_step(table, free, [(b, a) for a, b in pairs], bs, s["rows_back"])
        # entries of the stack's array that hold no page any more keep what they held: not defined
        return [torch.tensor(x, device=s["free"].device) for x in there + back] + \
            [torch.tensor(table, device=s["free"].device), None, torch.tensor([len(free)], device=s["free"].device)]
    if op == "bounds":
        x = _exact_pool(s, s["kc"], s["ks"])
        code, size = s["bounds"].double(), _pow2d(s["bscale"].to(I64) - 127)
        rows = {}
        for slot in s["slots"].tolist():
            if slot >= 0:
                rows[slot // bs] = max(rows.get(slot // bs, 0), slot % bs + 1)
        for n in set(rows.values()):
            b = torch.tensor([p for p, m in rows.items() if m == n], device=x.device)
            lo, hi = x[b][:, :, :n].min(2).values, x[b][:, :, :n].max(2).values
            a = torch.maximum(-lo, hi).max(-1).values
            part = torch.frexp(a / 127.0)  # a power of two has mantissa 0.5
            ex = part.exponent - (part.mantissa == 0.5).to(I32)
            ex = torch.where(a == 0, torch.full_like(ex, -126), ex).clamp(min=-126)
            unit = _pow2d(ex)
            code[b] = torch.stack([torch.floor(lo / unit[..., None]), torch.ceil(hi / unit[..., None])], 2)
            size[b] = unit
        return [code, size]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    grp = hq // hkv
    table, outs, lses, start = s["table"].long(), [], [], 0
    dev = table.device
    if op == "select":
        for r, (nq, n) in enumerate(pairs):
            blk = table[r, :_ceil(n, bs)]
            bound = s["bounds"][blk].double() * _pow2d(s["bscale"][blk].to(I64) - 127)[..., None, None]
            q = s["q"][start:start + nq].double()
            unit = _pow2d((torch.frexp(q.abs().max(-1).values).exponent - 1).clamp(min=-112) - 7)[..., None]
            q = torch.round(q / unit) * unit
            best = None
            for h in range(grp):  # head h of every group: what a key inside the bounds can score at most
                w = q[:, h::grp].transpose(0, 1)                              # [Hkv, nq, D]
                x = w.clamp(min=0) @ bound[:, :, 1].permute(1, 2, 0) + w.clamp(max=0) @ bound[:, :, 0].permute(1, 2, 0)
                best = x if best is None else torch.maximum(best, x)
            for i in range(nq):
                m = _ceil(n - nq + i + 1, bs)
                x = best[:, i, :m].clone()
                x[:, 0] = x[:, m - 1] = float("inf")
                at = torch.sort(-x, dim=-1, stable=True).indices[:, :case["top"]].sort(-1).values
                row = torch.full((hkv, case["top"]), -1, dtype=I64, device=dev)
                row[:, :at.shape[1]] = at
                outs.append(row)
            start += nq
        return [torch.stack(outs)]
    # [page, head] rows of the pools, gathered page by page below
    kc, vc = s["kc"], s["vc"]
    for r, (nq, n) in enumerate(pairs):
        blk = table[r, :_ceil(n, bs)]
        k, v = [_exact_pool(s, (p.view(U8)[blk].view(E4M3) if sc is not None else p[blk]), None if sc is None else sc[blk])
                for p, sc in ((kc, s["ks"]), (vc, s["vs"]))]                  # [pages, Hkv, bs, D]
        for i in range(nq):
            length, q = n - nq + i + 1, s["q"][start + i].double().view(hkv, grp, d)
            at = s["pages"][start + i].long()
            held = at >= 0
            at = at.clamp(min=0)
            h = torch.arange(hkv, device=dev)[:, None]
            kk, vv = k[at, h].flatten(1, 2), v[at, h].flatten(1, 2)           # [Hkv, top * bs, D]
            keep = held[..., None] & (at[..., None] * bs + torch.arange(bs, device=dev) < length)
            x = torch.bmm(q, kk.transpose(1, 2)) * s["scale"]
            x = torch.where(keep.flatten(1)[:, None], x, torch.full((), NEG, dtype=F64, device=dev))
            if s["sink"] is not None:
                x = torch.cat([x, s["sink"].double().view(hkv, grp, 1)], -1)
            lse = torch.logsumexp(x, -1)
            w = torch.exp(x - lse[..., None])[..., :kk.shape[1]]
            outs.append(torch.bmm(w, vv).reshape(hq, d))
            lses.append(lse.reshape(hq))
        start += nq
    return [torch.stack(outs), torch.stack(lses)] if case["lse"] else [torch.stack(outs)]
