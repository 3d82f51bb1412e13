"""Measured cases of the 8-bit paged cache, the tree attention and the fused
q/k norm + rotary embedding + cache write.

Five operators, one case each time:
  write   reshape_and_cache_fp8: quantise new K/V rows into e4m3 pages with
          one power-of-two scale (an E8M0 byte) per token and kv head
  gather  gather_cache_fp8: read the pages back as contiguous bf16 rows
  decode  paged_decode_fp8: one query per sequence over e4m3 pages
  tree    paged_tree_attention: a tree of drafted tokens per sequence over
          bf16 or e4m3 pages
  norm    qk_norm_rope_reshape_and_cache: per-head RMS norm of q and k, the
          rotary embedding and the cache write in one pass

``own`` chooses between the plain torch forms and the library's calls.
"""
import math
import random

import torch

own = False

BF16, F32, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6
NEG = float("-inf")


def listed():
    return [
        # one decode step's new tokens of a batch of 64 sequences
        dict(name="write-64", op="write", tokens=64, hkv=8, d=128, bs=16, layout="NHD", dtype="bf16"),
        # the prompt tokens of a long prefill, a ragged count, head-major pages
        dict(name="write-66001-hnd", op="write", tokens=66001, hkv=8, d=128, bs=16, layout="HND", dtype="bf16"),
        # a few short prefixes read back before a chunk's prefill
        dict(name="gather-short", op="gather", batch=5, lo=17, hi=700, hkv=4, d=64, bs=16, layout="NHD"),
        # the cached prefixes of a 16-request chunk prefill
        dict(name="gather-16x8k", op="gather", batch=16, lo=1, hi=8192, hkv=8, d=128, bs=16, layout="NHD"),
        # three short sequences, where the call's latency counts
        dict(name="decode-3", op="decode", batch=3, lo=30, hi=70, hq=4, hkv=2, d=64, bs=32, layout="NHD",
             window=-1, sink=True, lse=True),
        # an ordinary decode batch
        dict(name="decode-64x4k", op="decode", batch=64, lo=512, hi=4096, hq=32, hkv=8, d=128, bs=16,
             layout="NHD", window=-1, sink=False, lse=False),
        # long contexts with attention sinks
        dict(name="decode-8x128k", op="decode", batch=8, lo=32768, hi=131072, hq=64, hkv=8, d=64, bs=16,
             layout="NHD", window=-1, sink=True, lse=False),
        # small trees on short contexts
        dict(name="tree-4x8", op="tree", batch=4, lo=60, hi=900, qlo=3, qhi=8, hq=32, hkv=8, d=128, bs=16,
             layout="NHD", window=-1, sink=False, lse=True, kv="bf16"),
        # an ordinary speculative step over an 8-bit cache
        dict(name="tree-16x24-fp8", op="tree", batch=16, lo=512, hi=8192, qlo=12, qhi=24, hq=32, hkv=8, d=128,
             bs=32, layout="HND", window=-1, sink=True, lse=False, kv="e4m3"),
        # wide trees over long contexts
        dict(name="tree-8x64-32k", op="tree", batch=8, lo=16384, hi=32768, qlo=64, qhi=64, hq=32, hkv=8, d=128,
             bs=16, layout="NHD", window=-1, sink=False, lse=False, kv="bf16"),
        # a decode step's tokens into 8-bit pages
        dict(name="norm-256-fp8", op="norm", tokens=256, hq=32, hkv=8, d=128, rd=128, neox=True, bs=16,
             layout="NHD", kv="e4m3"),
        # a mixed step's new tokens, sliced from one fused projection
        dict(name="norm-8448", op="norm", tokens=8448, hq=32, hkv=8, d=128, rd=128, neox=True, bs=16,
             layout="NHD", kv="bf16"),
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))) if hi > lo else lo


def draw(rng):
    op = rng.choice(["write", "gather", "decode", "decode", "tree", "tree", "norm"])
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 112, 128])
    c = dict(op=op, hkv=hkv, d=d, bs=rng.choice([16, 32]), layout=rng.choice(["NHD", "HND"]))
    if op == "write":
        c.update(tokens=_log(rng, 1, 40000), dtype=rng.choice(["bf16", "bf16", "f32"]))
    elif op == "norm":
        c.update(tokens=_log(rng, 1, 8000), hq=hkv * rng.choice([1, 2, 4]), rd=rng.choice([d // 32 * 32, 32]),
                 neox=rng.choice([True, False]), kv=rng.choice(["bf16", "e4m3"]))
    else:
        hi = _log(rng, 40, 16000)
        c.update(batch=_log(rng, 1, 40), lo=max(1, hi // rng.choice([1, 3, 10])), hi=hi)
        if op != "gather":
            c.update(hq=hkv * rng.choice([1, 2, 3, 4, 5, 8]), window=rng.choice([-1, -1, _log(rng, 1, 5000)]),
                     sink=rng.choice([True, False]), lse=rng.choice([True, False]))
        if op == "tree":
            qhi = _log(rng, 1, min(100, hi))
            c.update(batch=min(c["batch"], 16), qlo=max(1, qhi // 2), qhi=qhi, kv=rng.choice(["bf16", "e4m3"]))
            c["lo"] = max(c["lo"], qhi)
    return c


# ---------------------------------------------------------------------------
# what a case's lengths and trees are (from the case alone: work() needs them)
# ---------------------------------------------------------------------------
def _lengths(case):
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    if case["op"] != "tree":
        return lens, None, None
    qlens = [rng.randint(case["qlo"], case["qhi"]) for _ in lens]
    # node 0 is the root; node i hangs on one of the nodes before it
    parents = [[-1] + [rng.randint(max(0, i - 6), i - 1) for i in range(1, n)] for n in qlens]
    return lens, qlens, parents


def _ancestors(parents):
    """Per node: the set of visible draft nodes (itself and its ancestors) as bits."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
    return bits


def work(case):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    if op == "write":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * hkv
        return {"bytes": 2 * n * (d * e + d + 1) + 8 * case["tokens"], "flops": 4 * n * d}
    if op == "norm":
        t, hq = case["tokens"], case["hq"]
        pool = d * 2 if case["kv"] == "bf16" else d + 1
        return {"bytes": t * ((hq + 2 * hkv) * d * 2 + (hq + hkv) * d * 2 + 2 * hkv * pool + 16),
                "flops": t * (hq + hkv) * d * 8}
    lens, qlens, parents = _lengths(case)
    total = sum(lens)
    if op == "gather":
        return {"bytes": 2 * total * hkv * (d + 1 + 2 * d), "flops": 2 * total * hkv * d}
    w, hq = case["window"], case["hq"]
    if op == "decode":
        keys = sum(min(n, w + 1) if w >= 0 else n for n in lens)
        return {"bytes": 2 * keys * hkv * (d + 1) + 2 * case["batch"] * hq * d * 2, "flops": 4 * d * hq * keys}
    row = d * 2 if case["kv"] == "bf16" else d + 1
    keys = pairs = 0
    for n, q, par in zip(lens, qlens, parents):
        depth = [bin(b).count("1") - 1 for b in _ancestors(par)]
        keys += q + (min(n - q, w) if w >= 0 else n - q)
        pairs += sum(min(t + 1, w + 1) if w >= 0 else t + 1 for t in depth)
        pairs += sum(max(0, min(n - q, w - t)) if w >= 0 else n - q for t in depth)
    return {"bytes": 2 * keys * hkv * row + 2 * sum(qlens) * hq * d * 2, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pow2(e):
    """2^e as float32, from its bits (-126 <= e <= 127)."""
    return ((e.to(I32) + 127) << 23).view(F32)


def _quantise(x):
    """[..., D] -> (e4m3 codes, E8M0 bytes [...]) with e = ceil(log2(max|x| / 448))."""
    x = x.float()
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)  # a = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(a > 0, e, torch.full_like(e, -126)).clamp(-126, 119)
    bad = ~torch.isfinite(a)
    e = torch.where(bad, torch.zeros_like(e), e)
    y = (x * _pow2(-e).unsqueeze(-1)).clamp(-448, 448)
    y = torch.where(bad.unsqueeze(-1), torch.zeros_like(y), y)
    return y.to(E4M3), torch.where(bad, torch.full_like(e, 255), e + 127).to(U8)


def _pools(g, nb, case, fp8, dev):
    """Two pools filled with K/V rows whose sizes differ by head and by token."""
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    out = []
    for _ in range(2):
        x = torch.randn(nb, hkv, bs, d, generator=g, device=dev, dtype=BF16)
        x *= torch.exp2(torch.randn(nb, hkv, bs, 1, generator=g, device=dev)).to(BF16) * 0.5
        code, scale = _quantise(x) if fp8 else (x, None)
        if case["layout"] == "NHD":
            code = code.view(U8).permute(0, 2, 1, 3).contiguous().view(E4M3) if fp8 else \
                code.permute(0, 2, 1, 3).contiguous()
        out.append((code, scale))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, hkv, d, bs = case["op"], case["hkv"], case["d"], case["bs"]
    s = dict(case=dict(case), op=op, bs=bs, layout=case["layout"])

    def randn(*shape, dtype=BF16):
        return torch.randn(*shape, generator=g, device=dev, dtype=F32).to(dtype)

    if op in ("write", "norm"):
        t = case["tokens"]
        nb = (t + bs - 1) // bs + 7
        fp8 = op == "write" or case["kv"] == "e4m3"
        s["kc"], s["vc"], s["ks"], s["vs"] = _pools(g, nb, case, fp8, dev)
        # whole pages in a shuffled order, every 50th token not cached
        perm = torch.randperm(nb, generator=g, device=dev)
        at = torch.arange(t, device=dev)
        slots = perm[at // bs] * bs + at % bs
        s["slots"] = torch.where(at % 50 == 49, torch.full_like(slots, -1), slots)
    if op == "write":
        dt = BF16 if case["dtype"] == "bf16" else F32
        size = torch.exp2(2 * torch.randn(t, hkv, 1, generator=g, device=dev))
        s["key"] = (randn(t, hkv, d, dtype=F32) * size).to(dt)
        s["value"] = randn(t, hkv, d, dtype=dt)
        return s
    if op == "norm":
        hq, rd = case["hq"], case["rd"]
        # q, k and v are slices of one fused projection
        qkv = randn(t, hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["qo"], s["ko"] = torch.zeros(t, hq, d, dtype=BF16, device=dev), torch.zeros(t, hkv, d, dtype=BF16, device=dev)
        s["qw"], s["kw"] = 1 + 0.1 * randn(d, dtype=F32), 1 + 0.1 * randn(d, dtype=F32)
        maxpos = 16384
        s["pos"] = torch.randint(0, maxpos, (t,), generator=g, device=dev)
        f = torch.arange(rd // 2, device=dev, dtype=torch.float64)
        ang = torch.arange(maxpos, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-2 * f / rd)
        s["table"] = torch.stack([ang.cos(), ang.sin()], -1).float()
        return s
    lens, qlens, parents = _lengths(case)
    pages = [(n + bs - 1) // bs for n in lens]
    nb = sum(pages) + 5
    fp8 = op != "tree" or case["kv"] == "e4m3"
    s["kc"], s["vc"], s["ks"], s["vs"] = _pools(g, nb, case, fp8, dev)
    perm = torch.randperm(nb, generator=g, device=dev).to(I32)
    npg = torch.tensor(pages, device=dev)
    col = torch.arange(max(pages), device=dev)
    first = torch.cumsum(npg, 0) - npg
    idx = (first[:, None] + col).clamp(max=nb - 1)
    s["table"] = torch.where(col < npg[:, None], perm[idx], torch.full_like(perm[idx], -1)).contiguous()
    s["lens"] = torch.tensor(lens, dtype=I32, device=dev)
    s["max"] = max(lens)
    if op == "gather":
        s["total"] = sum(lens)
        s["cu"] = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=I32, device=dev)
        return s
    hq = case["hq"]
    s["sink"] = randn(hq, dtype=F32) if case["sink"] else None
    s["scale"] = d ** -0.5
    s["window"], s["want_lse"] = case["window"], case["lse"]
    if op == "decode":
        s["q"] = randn(case["batch"], hq, d)
        return s
    total = sum(qlens)
    s["q"] = randn(total, hq, d)
    s["maxq"] = max(qlens)
    s["cuq"] = torch.tensor([0] + [sum(qlens[:i + 1]) for i in range(len(qlens))], dtype=I32, device=dev)
    words = (s["maxq"] + 63) // 64
    rows, depth = [], []
    for par in parents:
        for b in _ancestors(par):
            w = [(b >> (64 * k)) & (2 ** 64 - 1) for k in range(words)]
            rows.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in w])
            depth.append(bin(b).count("1") - 1)
    s["mask"] = torch.tensor(rows, dtype=I64, device=dev)
    s["depth"] = torch.tensor(depth, dtype=I32, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _scatter(pool, blk, off, rows, layout):
    if layout == "NHD":
        pool[blk, off] = rows
    else:
        pool[blk, :, off] = rows


def _plain_store(s, key, value):
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    blk, off = slots // s["bs"], slots % s["bs"]
    if s["ks"] is None:
        _scatter(s["kc"], blk, off, key[keep], s["layout"])
        _scatter(s["vc"], blk, off, value[keep], s["layout"])
        return
    kq, ke = _quantise(key[keep])
    vq, ve = _quantise(value[keep])
    _scatter(s["kc"].view(U8), blk, off, kq.view(U8), s["layout"])
    _scatter(s["vc"].view(U8), blk, off, vq.view(U8), s["layout"])
    s["ks"][blk, :, off] = ke
    s["vs"][blk, :, off] = ve


def _stored(s):
    """The pools as what they stand for: codes and scales as numbers."""
    if s["ks"] is None:
        return [s["kc"], s["vc"]]
    return [s["kc"], s["vc"], s["ks"].view(E8M0), s["vs"].view(E8M0)]


def _rows(s, pool, scale, blk, off):
    """Rows of a pool as float32 [..., Hkv, D]."""
    if s["layout"] == "NHD":
        x = (pool.view(U8)[blk, off].view(E4M3) if scale is not None else pool[blk, off]).float()
    else:
        x = (pool.view(U8)[blk, :, off].view(E4M3) if scale is not None else pool[blk, :, off]).float()
    if scale is None:
        return x
    e = scale[blk, :, off].to(I32)
    m = torch.where(e == 255, torch.full((), float("nan"), device=x.device), _pow2(e.clamp(max=254) - 127))
    return x * m.unsqueeze(-1)


def _plain_gather(s):
    at = torch.arange(s["total"], device=s["cu"].device)
    req = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    pos = at - s["cu"].long()[req]
    blk = s["table"][req, pos // s["bs"]].long()
    return [_rows(s, s["kc"], s["ks"], blk, pos % s["bs"]).to(BF16),
            _rows(s, s["vc"], s["vs"], blk, pos % s["bs"]).to(BF16)]


def _padded_keys(s):
    """K and V of every sequence, padded to the longest: [B, Hkv, L, D] float32."""
    pos = torch.arange(s["max"], device=s["lens"].device)
    blk = s["table"][:, pos // s["bs"]].long()
    held = (pos < s["lens"][:, None]) & (blk >= 0)
    blk = torch.where(held, blk, torch.zeros_like(blk))
    off = (pos % s["bs"]).expand_as(blk)
    zero = torch.zeros((), device=blk.device)
    return [torch.where(held[..., None, None], _rows(s, p, sc, blk, off), zero).transpose(1, 2)
            for p, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))] + [pos]


def _plain_attend(q, k, v, keep, sink, scale):
    """q [B, T, Hq, D], k/v [B, Hkv, L, D], keep [B, T, L] -> o [B, T, Hq, D], lse [B, T, Hq]."""
    b, t, hq, d = q.shape
    hkv = k.shape[1]
    grp = hq // hkv
    qf = q.float().view(b, t, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * grp, d)
    sc = (qf @ k.transpose(2, 3) * scale).view(b, hkv, t, grp, -1)
    sc = sc.masked_fill(~keep[:, None, :, None, :], NEG)
    m = sc.amax(-1, keepdim=True)
    if sink is not None:
        snk = sink.view(1, hkv, 1, grp, 1)
        m = torch.maximum(m, snk)
    ms = torch.where(m == NEG, torch.zeros_like(m), m)
    p = torch.exp(sc - ms)
    l = p.sum(-1, keepdim=True)
    if sink is not None:
        l = l + torch.exp(snk - ms)
    o = (p.view(b, hkv, t * grp, -1) @ v).view(b, hkv, t, grp, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (torch.log(l) + ms).squeeze(-1)
    return o.permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(q.dtype), lse.permute(0, 2, 1, 3).reshape(b, t, hq)


def _plain_decode(s):
    k, v, pos = _padded_keys(s)
    n = s["lens"][:, None]
    keep = pos < n
    if s["window"] >= 0:
        keep = keep & (pos >= n - 1 - s["window"])
    o, lse = _plain_attend(s["q"][:, None], k, v, keep[:, None], s["sink"], s["scale"])
    return [o[:, 0], lse[:, 0]] if s["want_lse"] else [o[:, 0]]


def _plain_tree(s):
    k, v, pos = _padded_keys(s)
    cu = s["cuq"].long()
    nq, n = (cu[1:] - cu[:-1])[:, None, None], s["lens"].long()[:, None, None]
    row = torch.arange(s["maxq"], device=cu.device)
    at = (cu[:-1, None] + row).clamp(max=s["q"].shape[0] - 1)
    ctx = n - nq
    j = (pos - ctx).expand(-1, s["maxq"], -1)  # the key's draft node (negative: context)
    jc = j.clamp(0, 64 * s["mask"].shape[1] - 1)
    seen = (torch.gather(s["mask"][at], 2, jc // 64) >> (jc % 64)) & 1
    keep = (pos < n) & ((j < 0) | (seen == 1)) & (row[:, None] < nq)
    if s["window"] >= 0:
        depth = s["depth"].long()
        kd = depth[(cu[:-1, None, None] + jc).clamp(max=depth.shape[0] - 1)]
        kpos = torch.where(j < 0, pos.expand_as(j), ctx + kd)
        keep = keep & (kpos >= ctx + depth[at][..., None] - s["window"])
    o, lse = _plain_attend(s["q"][at], k, v, keep, s["sink"], s["scale"])
    total = torch.arange(s["q"].shape[0], device=cu.device)
    r = torch.searchsorted(cu[1:], total, right=True)
    t = total - cu[r]
    return [o[r, t], lse[r, t]] if s["want_lse"] else [o[r, t]]


def _plain_rotate(s, x, w):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    rd = s["case"]["rd"]
    half = rd // 2
    c, sn = s["table"][s["pos"]].unbind(-1)
    c, sn = c[:, None], sn[:, None]
    if s["case"]["neox"]:
        a, b = x[..., :half], x[..., half:rd]
        y = torch.cat([a * c - b * sn, b * c + a * sn, x[..., rd:]], -1)
    else:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), x[..., rd:]], -1)
    return y.to(BF16)


def _plain_norm(s):
    s["qo"].copy_(_plain_rotate(s, s["q"], s["qw"]))
    s["ko"].copy_(_plain_rotate(s, s["k"], s["kw"]))
    _plain_store(s, s["ko"], s["v"])


def run(state):
    s = state
    op = s["op"]
    if own:
        return _own(s, op)
    if op == "write":
        _plain_store(s, s["key"], s["value"])
        return _stored(s)
    if op == "norm":
        _plain_norm(s)
        return [s["qo"], s["ko"]] + _stored(s)
    return {"gather": _plain_gather, "decode": _plain_decode, "tree": _plain_tree}[op](s)


def _own(s, op):
    import paged_kv_cache_attention_gb300 as pkv
    if op == "write":
        pkv.reshape_and_cache_fp8(s["key"], s["value"], s["kc"], s["vc"], s["ks"], s["vs"], s["slots"],
                                  layout=s["layout"])
        return _stored(s)
    if op == "norm":
        pkv.qk_norm_rope_reshape_and_cache(
            s["q"], s["k"], s["v"], s["kc"], s["vc"], s["pos"], s["slots"], s["table"], s["qw"], s["kw"],
            eps=EPS, rotary_dim=s["case"]["rd"], is_neox_style=s["case"]["neox"], query_out=s["qo"],
            key_out=s["ko"], k_scale=s["ks"], v_scale=s["vs"], layout=s["layout"])
        return [s["qo"], s["ko"]] + _stored(s)
    if op == "gather":
        return list(pkv.gather_cache_fp8(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["total"],
                                         layout=s["layout"]))
    lse = torch.empty(s["q"].shape[:2], dtype=F32, device=s["q"].device) if s["want_lse"] else None
    if op == "decode":
        o = pkv.paged_decode_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["max"],
                                 sink=s["sink"], window_left=s["window"], sm_scale=s["scale"], lse=lse,
                                 layout=s["layout"])
    else:
        o = pkv.paged_tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["cuq"], s["lens"], s["maxq"],
                                     s["max"], s["mask"], tree_depth=s["depth"], k_scale=s["ks"],
                                     v_scale=s["vs"], sink=s["sink"], window_left=s["window"],
                                     sm_scale=s["scale"], lse=lse, layout=s["layout"])
    return [o, lse] if s["want_lse"] else [o]


# ---------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_pow2(e):
    """2^e in float64, from its bits."""
    return ((e.to(I64) + 1023) << 52).view(torch.float64)


def _exact_e4m3(y):
    """Nearest e4m3 value (ties to even), saturating at 448."""
    a = y.abs().clamp(max=448.0)
    ex = torch.frexp(a.clamp(min=2.0 ** -6)).exponent - 1
    step = _exact_pow2(ex - 3)
    return torch.copysign((a / step).round() * step, y)  # round(): ties to even


def _exact_store(s, key, value, out):
    """out: the stored tensors as float64 copies, updated token by token."""
    slots = s["slots"].tolist()
    keep = torch.tensor([i for i, x in enumerate(slots) if x >= 0], device=key.device, dtype=I64)
    at = s["slots"][keep]
    b, o = at // s["bs"], at % s["bs"]
    for n, x in enumerate((key, value)):
        x = x.double()[keep]
        if s["ks"] is not None:
            part = torch.frexp(x.abs().max(-1).values / 448.0)  # a power of two has mantissa 0.5
            e = (part.exponent - (part.mantissa == 0.5).to(I32)).clamp(-126, 119)
            e = torch.where(part.mantissa == 0, -126, e)
            size = _exact_pow2(e)
            out[2 + n][b, :, o] = size
            x = _exact_e4m3(x / size[..., None])
        if s["layout"] == "NHD":
            out[n][b, o] = x
        else:
            out[n][b, :, o] = x
    return out


def _exact_pool(s):
    """Both pools in float64 as [slots, Hkv, D]."""
    got = []
    for p, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        x = p.double()
        if s["layout"] == "HND":
            x = x.transpose(1, 2)
        if sc is not None:
            x = x * _exact_pow2(sc.to(I64) - 127).transpose(1, 2)[..., None]
        got.append(x.reshape(-1, x.shape[2], x.shape[3]))
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op, bs = s["op"], s["bs"]
    if op == "write":
        return _exact_store(s, s["key"], s["value"], [x.double() for x in _stored(s)])
    if op == "norm":
        rd = case["rd"]
        inv = 10000.0 ** (-2 * torch.arange(rd // 2, dtype=torch.float64, device=s["pos"].device) / rd)
        ang = (s["pos"].double()[:, None] * inv)[:, None]
        res = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.double()
            x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
            y = x.clone()
            ia = slice(0, rd // 2) if case["neox"] else slice(0, rd, 2)
            ib = slice(rd // 2, rd) if case["neox"] else slice(1, rd, 2)
            y[..., ia] = x[..., ia] * ang.cos() - x[..., ib] * ang.sin()
            y[..., ib] = x[..., ib] * ang.cos() + x[..., ia] * ang.sin()
            res.append(y)
        # what the pages hold is the key as it was rounded to its type
        if s["ks"] is not None:
            return res + [None, None, None, None]
        return res + _exact_store(s, res[1], s["v"], [x.double() for x in _stored(s)])
    kp, vp = _exact_pool(s)
    lens, qlens, parents = _lengths(case)
    outs, lses = [], []
    table = s["table"].long()
    start = 0
    for r, n in enumerate(lens):
        pos = torch.arange(n, device=table.device)
        slot = table[r, pos // bs] * bs + pos % bs
        k, v = kp[slot].transpose(0, 1), vp[slot].transpose(0, 1)  # [Hkv, n, D]
        if op == "gather":
            outs.append(k.transpose(0, 1))
            lses.append(v.transpose(0, 1))
            continue
        nq = qlens[r] if op == "tree" else 1
        q = s["q"][start:start + nq].double()
        start += nq
        bits = _ancestors(parents[r]) if op == "tree" else [1]
        depth = torch.tensor([bin(b).count("1") - 1 for b in bits], device=table.device)
        ctx = n - nq
        keep = torch.ones(nq, n, dtype=torch.bool, device=table.device)
        keep[:, ctx:] = torch.tensor([[bool(b >> j & 1) for j in range(nq)] for b in bits], device=table.device)
        if s["window"] >= 0:
            kpos = torch.cat([pos[:ctx], ctx + depth])
            keep &= kpos[None] >= (ctx + depth)[:, None] - s["window"]
        hq, d = q.shape[1:]
        hkv = k.shape[0]
        qs = q.transpose(0, 1).reshape(hkv, hq // hkv * nq, d)  # rows: (head of the group, token)
        logit = torch.bmm(qs, k.transpose(1, 2)).reshape(hq, nq, n) * s["scale"]
        logit = torch.where(keep[None], logit, torch.full((), NEG, device=logit.device, dtype=logit.dtype))
        if s["sink"] is not None:
            logit = torch.cat([logit, s["sink"].double()[:, None, None].expand(hq, nq, 1)], -1)
        lse = torch.logsumexp(logit, -1)
        wgt = torch.exp(logit - torch.where(lse == NEG, torch.zeros_like(lse), lse)[..., None])[..., :n]
        o = torch.bmm(wgt.reshape(hkv, hq // hkv * nq, n), v).reshape(hq, nq, d)
        outs.append(o.transpose(0, 1))
        lses.append(lse.transpose(0, 1))
    if op == "gather":
        return [torch.cat(outs), torch.cat(lses)]
    return [torch.cat(outs), torch.cat(lses)] if s["want_lse"] else [torch.cat(outs)]
