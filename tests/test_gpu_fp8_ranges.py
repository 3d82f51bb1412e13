"""Rows of very different sizes in one 8-bit cache: what a key adds to a row is
off by a share of that row's largest weighted value, whatever other keys hold
that the row does not attend or hardly weighs."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
I32 = torch.int32


def floor_of(q, k, v, keep, scale, per_key):
    """per_key * n * max_j p_j max_d |v_jd| of every row: [T, Hq, 1]."""
    t, hq, _ = q.shape
    grp = hq // k.shape[1]
    out = torch.zeros(t, hq, 1, dtype=torch.float64)
    for h in range(hq):
        big = v[:, h // grp].abs().amax(-1)
        for i in range(t):
            sel = keep[i]
            p = torch.softmax((k[:, h // grp][sel] @ q[i, h].to(torch.float64)) * scale, 0)
            if p.numel():
                out[i, h] = per_key * p.numel() * (p * big[sel]).max()
    return out


def check(out, lse, q, k, v, keep, scale, per_key, what):
    ref, rl, absv, smax = R.attend(q, k, v, keep, scale)
    d = q.shape[-1]
    # f16 weights: 2^-11; a weight's exponent holds the score and V's exponent, below
    # 2^9 in all, in fp32: off by 4 roundings of 2^-24 * 2^9, so by 2^-13 of the weight
    bound = R.out_bound(ref, absv, smax, d, 2.0 ** -11 + 2.0 ** -13) + \
        floor_of(q, k, v, keep, scale, per_key)
    R.assert_within(out, ref, bound, what)
    if lse is not None:
        R.assert_within(lse, rl, R.lse_bound(rl, smax, d), what + " lse")


# decode: a key's weight is held to 2^-25, the row's largest weighted scale stands at
# 2^6 or more, and a row's largest code is above 224 of 448: 2^-31 * 2 per key
DECODE_FLOOR = 2.0 ** -30


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 1), (128, 8, 2), (256, 12, 1), (96, 3, 3)])
@pytest.mark.parametrize("size", [20, 24, 28, 30, 60, 100, 118])
def test_decode_a_large_value_of_little_weight(size, d, hq, hkv):
    """One key's V is 2^size times the others' and its weight 2^-(size + 40)."""
    g = torch.Generator().manual_seed(size + d)
    n, bs = 150, 16
    nb = n // bs + 2
    pools = R.Pools(nb, bs, hkv, d, "NHD", True, g)
    table, slots = R.paged([n], bs, nb, g)
    scale = d ** -0.5
    # queries near one direction, and a key against it
    way = torch.randn(d, generator=g)
    q = (way + 0.05 * torch.randn(1, hq, d, generator=g)).to(BF16)
    odd = slots[0][77]
    pools.rows[0] = 0.3 * torch.randn(pools.rows[0].shape, generator=g).to(BF16)
    pools.rows[0][odd // bs, :, odd % bs] = \
        (-way * ((size + 40) * 0.693 / (scale * float(way @ way)))).to(BF16)
    pools.rows[1] = torch.randn(pools.rows[1].shape, generator=g).to(BF16)
    pools.rows[1][odd // bs, :, odd % bs] *= 2.0 ** size
    pools.codes, pools.byte = R.quantise(pools.rows)
    k, v = pools.at(slots[0])
    keep = torch.ones(1, n, dtype=torch.bool)
    for part in (512, 64):
        lse = torch.zeros(1, hq, device=DEV)
        out = pkv.paged_decode_fp8(q.to(DEV), *pools.device(DEV), table.to(DEV),
                                   torch.tensor([n], dtype=I32, device=DEV), n, lse=lse,
                                   partition_size=part)
        check(out, lse, q, k, v, keep, scale, DECODE_FLOOR, f"partition {part}")


@pytest.mark.parametrize("size", [-118, -60, 60, 118])
def test_decode_values_of_one_far_size(size):
    """All of V near either end of the format's range."""
    g = torch.Generator().manual_seed(7)
    n, bs, d, hq = 100, 32, 128, 4
    pools = R.Pools(5, bs, 1, d, "HND", True, g)
    table, slots = R.paged([n], bs, 5, g)
    pools.rows[1] = (torch.randn(pools.rows[1].shape, generator=g) * 2.0 ** size).to(BF16)
    pools.codes, pools.byte = R.quantise(pools.rows)
    q = torch.randn(1, hq, d, generator=g).to(BF16)
    k, v = pools.at(slots[0])
    for part in (512, 32):
        out = pkv.paged_decode_fp8(q.to(DEV), *pools.device(DEV), table.to(DEV),
                                   torch.tensor([n], dtype=I32, device=DEV), n, layout="HND",
                                   partition_size=part)
        got = out.to(torch.float64).cpu() * 2.0 ** -size
        check(got, None, q, k, v * 2.0 ** -size, torch.ones(1, n, dtype=torch.bool), d ** -0.5,
              DECODE_FLOOR, f"partition {part}")
