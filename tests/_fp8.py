"""The 8-bit cache, the masked attention and the q/k norm in 64 bits, written
from their definitions; inputs for the parity tests.  CPU only."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn

# every e4m3 code's value (0x7f and 0xff are NaN)
CODE_VALUES = torch.arange(256, dtype=torch.uint8).view(E4M3).to(torch.float64)


def quantise(x):
    """[..., D] rows -> (codes uint8 [..., D], E8M0 bytes uint8 [...])."""
    x = x.to(torch.float64)
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    safe = torch.where(bad | (amax == 0), torch.ones_like(amax), amax)
    m, e = torch.frexp(safe / 448.0)
    e = torch.where(m == 0.5, e - 1, e)          # ceil(log2(amax / 448))
    e = torch.where(amax == 0, torch.full_like(e, -126), e).clamp(-126, 119)
    y = x / torch.pow(torch.tensor(2.0, dtype=torch.float64), e.to(torch.float64))[..., None]
    y = torch.where(bad[..., None], torch.zeros_like(y), y).clamp(-448.0, 448.0)
    a = y.abs()
    _, ex = torch.frexp(a.clamp(min=2.0 ** -6))
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), (ex - 4).to(torch.float64))
    v = torch.round(a / step) * step             # ties to even
    mag = torch.searchsorted(CODE_VALUES[:127].contiguous(), v.contiguous())
    assert torch.equal(CODE_VALUES[mag], v)
    codes = (mag + 128 * torch.signbit(y)).to(torch.uint8)
    return codes, torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def scales(byte):
    """2^(byte - 127) in float64; 255 is NaN."""
    e = byte.to(torch.float64) - 127
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64), e)
    return torch.where(byte == 255, torch.full_like(s, float("nan")), s)


class Pools:
    """Two pools with every slot written (values that differ in size by head
    and token) unless `poison`: then unowned slots hold NaN rows (bf16) or
    scale bytes 255 over arbitrary codes (8-bit)."""

    def __init__(self, num_blocks, bs, hkv, d, layout, fp8, gen, spread=1.0, dtype=torch.bfloat16):
        self.nb, self.bs, self.hkv, self.d, self.layout, self.fp8 = num_blocks, bs, hkv, d, layout, fp8
        x = torch.randn(2, num_blocks, hkv, bs, d, generator=gen)
        size = torch.exp2(spread * torch.randn(2, num_blocks, hkv, bs, 1, generator=gen)) * 0.7
        self.rows = (x * size).to(dtype)          # [2, nb, Hkv, bs, D]
        if fp8:
            codes, byte = quantise(self.rows)
            self.codes, self.byte = codes, byte

    def poison(self, slots):
        """NaN rows at flat slots."""
        s = torch.as_tensor(slots, dtype=torch.int64)
        for i in range(2):
            if self.fp8:
                self.byte[i][s // self.bs, :, s % self.bs] = 255
                self.codes[i][s // self.bs, :, s % self.bs] = 0x7f
            else:
                self.rows[i][s // self.bs, :, s % self.bs] = float("nan")

    def device(self, dev):
        """(k_cache, v_cache, k_scale, v_scale) on the device, in the layout."""
        x = self.codes if self.fp8 else self.rows
        if self.layout == "NHD":
            x = x.permute(0, 1, 3, 2, 4)
        x = x.contiguous()
        if not self.fp8:
            x = x.to(dev)
            return x[0], x[1], None, None
        x = x.to(dev)
        b = self.byte.to(dev)
        return x[0].view(E4M3), x[1].view(E4M3), b[0], b[1]

    def at(self, slots):
        """K and V rows [n, Hkv, D] in float64 of flat slots."""
        s = torch.as_tensor(slots, dtype=torch.int64)
        got = []
        for i in range(2):
            if self.fp8:
                v = CODE_VALUES[self.codes[i][s // self.bs, :, s % self.bs].long()]
                v = v * scales(self.byte[i][s // self.bs, :, s % self.bs])[..., None]
            else:
                v = self.rows[i][s // self.bs, :, s % self.bs].to(torch.float64)
            got.append(v)
        return got


def paged(lens, bs, num_blocks, gen):
    """A block table of shuffled pages and the flat slots of every position."""
    pages = [(n + bs - 1) // bs for n in lens]
    assert sum(pages) <= num_blocks
    perm = torch.randperm(num_blocks, generator=gen)
    table = torch.full((len(lens), max(pages + [1])), -1, dtype=torch.int32)
    slots, at = [], 0
    for i, (n, p) in enumerate(zip(lens, pages)):
        ids = perm[at:at + p]
        at += p
        table[i, :p] = ids.to(torch.int32)
        pos = torch.arange(n)
        slots.append(ids[pos // bs] * bs + pos % bs if n else torch.zeros(0, dtype=torch.int64))
    return table, slots


def attend(q, k, v, keep, scale, sink=None, bias=None):
    """q [T, Hq, D], k/v [n, Hkv, D] (float64), keep [T, n] -> out, lse and the
    bound's ingredients: sum_j p_j |v_j| and |scale| * max_j sum |q k_j|."""
    t, hq, d = q.shape
    n, hkv = k.shape[0], k.shape[1]
    grp = hq // hkv
    q = q.to(torch.float64)
    out = torch.zeros(t, hq, d, dtype=torch.float64)
    absv = torch.zeros_like(out)
    lse = torch.full((t, hq), float("-inf"), dtype=torch.float64)
    smax = torch.zeros(t, hq, dtype=torch.float64)
    for h in range(hq):
        kk, vv = k[:, h // grp], v[:, h // grp]
        for i in range(t):
            sel = keep[i]
            lg = (kk[sel] @ q[i, h]) * scale
            if bias is not None:
                lg = lg + bias[h, i][sel]
            if lg.numel():
                smax[i, h] = abs(scale) * (kk[sel].abs() @ q[i, h].abs()).max()
            if sink is not None:
                lg = torch.cat([lg, sink[h:h + 1].to(torch.float64)])
            if not lg.numel():
                continue
            lse[i, h] = torch.logsumexp(lg, 0)
            p = torch.exp(lg - lse[i, h])[:int(sel.sum())]
            out[i, h] = p @ vv[sel]
            absv[i, h] = p @ vv[sel].abs()
    return out, lse, absv, smax


def out_bound(ref, absv, smax, d, p_eps, f16_floor=0.0):
    """Half a bf16 step of the output, plus the weights' error: each p rounds to
    p_eps relative; its score is an fp32 sum of d products (d + 8 roundings of
    2^-24 of sum |q k|), which moves p and the normaliser.  f16_floor: see there."""
    p_err = p_eps + 2 * (d + 8) * 2.0 ** -24 * smax[..., None] + 2.0 ** -19
    return 2.0 ** -8 * ref.abs() + p_err * absv * (1 + 2.0 ** -8) + f16_floor + 2.0 ** -100


def f16_floor(v):
    """What f16 weights may add over 8-bit pools: weights are held times 2^6 at the
    softmax's reference (p <= 1) and the largest V scale 2^E, and f16's smallest
    step is 2^-24, so a small weight is off by at most 2^-25 * 2^-6 of p * 2^E = 1 *
    2^E; a code is at most 448 and the row with the scale 2^E has a value of at
    least 224 * 2^E, so n keys add at most n * 2^-31 * 2 max|v|."""
    n = v.shape[0]
    v = v[torch.isfinite(v)].abs()
    return float(v.max()) * 2.0 ** -30 * n if v.numel() else 0.0


def lse_bound(lse, smax, d):
    return (d + 8) * 2.0 ** -24 * smax + 2.0 ** -20 * (1 + lse.abs())


def assert_within(got, ref, bound, what):
    got = got.to(torch.float64).cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    off = torch.where(same, torch.zeros_like(ref), (got - ref).abs() - bound)
    off = torch.where(torch.isnan(off), torch.full_like(off, math.inf), off)
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 0.0, f"{what}: off by {worst} more than the bound"


def norm_rope(x, w, eps, table, pos, rd, neox):
    """[T, H, D] -> the normed and rotated rows in float64, and the sum of the
    magnitudes that each output adds (for the bound)."""
    x = x.to(torch.float64)
    y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w.to(torch.float64)
    cs = table[pos].to(torch.float64)             # [T, rd/2, 2]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    ia = slice(0, rd // 2) if neox else slice(0, rd, 2)
    ib = slice(rd // 2, rd) if neox else slice(1, rd, 2)
    out, mag = y.clone(), y.abs()
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag = mag.clone()
    mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out, mag


def to_numpy_bits(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def same_bits(a, b):
    return np.array_equal(to_numpy_bits(a), to_numpy_bits(b))
