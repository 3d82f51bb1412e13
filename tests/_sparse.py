"""A sparse step's operators from their definitions: block tables on Python lists,
page bounds and selection scores in 64 bits.  CPU only."""
from __future__ import annotations

import torch

from tests import _fp8 as R


def pages_of(n, bs):
    return (n + bs - 1) // bs


def step(table, free, old, new, bs, rows):
    """One step on lists (table rows and the stack, in place): slots, positions, cu_q, cu_k."""
    gone = []
    for r, (a, b) in enumerate(zip(old, new)):
        for p in range(pages_of(b, bs), pages_of(a, bs)):
            gone.append(table[r][p])
            table[r][p] = -1
    free.extend(reversed(gone))
    slots, pos, cuq, cuk = [], [], [0], [0]
    for r, (a, b) in enumerate(zip(old, new)):
        for p in range(pages_of(a, bs), pages_of(b, bs)):
            table[r][p] = free.pop()
        slots += [table[r][x // bs] * bs + x % bs for x in range(a, b)]
        pos += range(a, b)
        cuq.append(len(slots))
        cuk.append(cuk[-1] + b)
    return slots + [-1] * (rows - len(slots)), pos + [0] * (rows - len(pos)), cuq, cuk


def pow2(e):
    """2^e in float64, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def bounds(keys):
    """keys [..., n, D] (float64) -> codes int8 [..., 2, D], bytes uint8 [...]."""
    lo, hi = keys.amin(-2), keys.amax(-2)      # a NaN stays
    a = torch.maximum(lo.abs(), hi.abs()).amax(-1)
    bad = ~torch.isfinite(a)
    part = torch.frexp(torch.where(bad | (a == 0), torch.ones_like(a), a) / 127.0)
    e = torch.where(part.mantissa == 0.5, part.exponent - 1, part.exponent)
    e = torch.where(bad | (a == 0), torch.full_like(e, -126), e).clamp(min=-126)
    unit = pow2(e)[..., None]
    codes = torch.stack([torch.floor(lo / unit), torch.ceil(hi / unit)], -2)
    codes = torch.where(bad[..., None, None], torch.zeros_like(codes), codes)
    return codes.to(torch.int8), torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def scores(q, codes, byte):
    """q [Hq, D], codes [n, Hkv, 2, D], byte [n, Hkv] -> [Hkv, n] float64 holding fp32 values."""
    hq, d = q.shape
    hkv = codes.shape[1]
    q = q.to(torch.float64)
    amax = q.abs().amax(-1)
    ok = torch.isfinite(amax)
    e = (torch.frexp(torch.where(ok, amax, torch.ones_like(amax))).exponent - 1)
    e = torch.where(amax == 0, torch.full_like(e, -112), e).clamp(min=-112) - 7
    c = torch.where(ok[:, None], torch.round(q / pow2(e)[:, None]), torch.zeros_like(q))
    b = codes.to(torch.float64).permute(1, 2, 3, 0)          # [Hkv, 2, D, n]
    c = c.view(hkv, hq // hkv, d)
    prod = c.clamp(max=0) @ b[:, 0] + c.clamp(min=0) @ b[:, 1]
    x = prod * pow2(e.view(hkv, -1)[:, :, None] + (byte.to(torch.int32) - 127).t()[:, None])
    x = x.to(torch.float32).to(torch.float64)                # one rounding
    x = torch.where(ok.view(hkv, -1)[:, :, None], x, torch.full_like(x, float("-inf")))
    x = x.amax(1)
    return torch.where(byte.t() == 255, torch.full_like(x, float("inf")), x)


def choose(score, top_k, first, recent):
    """score [Hkv, n] -> pages [Hkv, top_k] (list): forced ones, then by score, then by number."""
    hkv, n = score.shape
    out = torch.full((hkv, top_k), -1, dtype=torch.int32)
    for g in range(hkv):
        s = score[g].tolist()
        order = sorted(range(n), key=lambda p: (0 if p < first or p >= n - recent else 1, -s[p], p))
        chosen = sorted(order[:top_k])
        out[g, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return out


def rows_of(queries, lens):
    """(request, keys up to and with its own) of every row."""
    return [(r, max(0, n - m + i + 1)) for r, (m, n) in enumerate(zip(queries, lens))
            for i in range(m)]


def attend_lists(q, pools, slots, rows, pages, bs, scale, sink):
    """Every row over its lists: out [T, Hq, D], lse [T, Hq] and the bound's ingredients
    (tests._fp8.attend), each row's largest |v| that it keeps."""
    hkv = pages.shape[1]
    grp = q.shape[1] // hkv
    outs = []
    vmax = []
    for t, (r, n) in enumerate(rows):
        k, v = pools.at(slots[r][:n])
        parts = []
        for g in range(hkv):
            keep = torch.zeros(1, n, dtype=torch.bool)
            for p in pages[t, g].tolist():
                if p < 0:
                    break
                keep[0, p * bs:min(n, (p + 1) * bs)] = True
            hs = slice(g * grp, (g + 1) * grp)
            parts.append(R.attend(q[t:t + 1, hs], k[:, g:g + 1], v[:, g:g + 1], keep, scale,
                                  None if sink is None else sink[hs]))
        outs.append([torch.cat([p[i] for p in parts], 1) for i in range(4)])
        vmax.append(R.f16_floor(v))
    got = [torch.cat([o[i] for o in outs]) for i in range(4)]
    return (*got, torch.tensor(vmax)[:, None, None])
