"""What the values of some keys may do to drafts that keep them, that hardly weigh
them, or that do not see them."""
import random

import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R
from tests.test_gpu_fp8_ranges import check
from tests.test_gpu_tree import pack, run, tree

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
I32 = torch.int32


def step(n, m, hq, hkv, d, fp8, kind, seed, bs=16):
    """One request of n tokens, m of them drafts: pools, q, table, mask, keep."""
    g = torch.Generator().manual_seed(seed)
    nb = (n + bs - 1) // bs + 2
    pools = R.Pools(nb, bs, hkv, d, "NHD", fp8, g)
    table, slots = R.paged([n], bs, nb, g)
    q = torch.randn(m, hq, d, generator=g).to(BF16)
    bits, _ = tree(m, random.Random(seed), kind)
    keep = torch.ones(m, n, dtype=torch.bool)
    keep[:, n - m:] = torch.tensor([[bool(b >> j & 1) for j in range(m)] for b in bits])
    return pools, q, table, slots[0], pack(bits, (m + 63) // 64 + 1), keep


def attend(pools, q, table, n, mask, partition, scale=None):
    m, hq, _ = q.shape
    kc, vc, ks, vs = pools.device(DEV)
    out = torch.full(q.shape, 7.0, dtype=BF16, device=DEV)
    lse = torch.full((m, hq), 7.0, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    pkv.paged_tree_attention(
        q.to(DEV), kc, vc, table.to(DEV), torch.tensor([0, m], dtype=I32, device=DEV),
        torch.tensor([n], dtype=I32, device=DEV), m, n, mask.to(DEV), k_scale=ks, v_scale=vs,
        sm_scale=scale, partition_size=partition, out=out, lse=lse, dev_error=err)
    assert pkv.get_device_error(err) == 0
    return out, lse


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("partition", [0, 1024])
@pytest.mark.parametrize("kind,m,d", [("tree", 12, 128), ("random", 40, 64), ("chain", 3, 256)])
def test_lse_is_of_the_scores_alone(kind, m, d, partition, fp8, value):
    """A value that is not finite makes the outputs of those who keep its key NaN
    (an infinity may stay one where the whole tile is seen), not their lse, in a
    tile of drafts and in one of context."""
    n, hq, hkv = 600, 8, 2
    pools, q, table, slots, mask, keep = step(n, m, hq, hkv, d, fp8, kind, 11 + m)
    for at in (n - m + 1, n - m // 2 - 1, 30):
        s = slots[at]
        rows = pools.rows.clone()
        pools.rows[1][s // 16, :, s % 16, d // 2] = value
        if fp8:
            pools.codes, pools.byte = R.quantise(pools.rows)
        out, lse = attend(pools, q, table, n, mask, partition)
        k, v = pools.at(slots)
        ref, rl, absv, smax = R.attend(q, k, v, keep, d ** -0.5)
        R.assert_within(lse, rl, R.lse_bound(rl, smax, d), f"lse, value at {at}")
        sees = keep[:, at]
        if at == 30 and not fp8:    # a whole tile: the column alone, as the sum makes it
            bad = torch.zeros(out.shape, dtype=torch.bool)
            bad[..., d // 2] = True
        else:
            bad = sees[:, None, None].expand(out.shape)
        got = out.cpu()
        assert not bool(torch.isfinite(got[bad]).any())
        ok = ~bad
        bound = R.out_bound(ref, absv, smax, d, 2.0 ** -11, R.f16_floor(v)) if fp8 else \
            R.out_bound(ref, absv, smax, d, 2.0 ** -8)
        R.assert_within(got[ok], ref[ok], bound[ok], f"out, value at {at}")
        pools.rows = rows


# a key's weight is held to 2^-25 where the largest score beside its tile's largest V
# scale stands at 2^6 or more; the row's weightiest key may have 2^-8 of that scale,
# and a code is at most twice as large as another row's largest: 2^-31 * 2^8 * 2
TREE_FLOOR = 2.0 ** -22


@pytest.mark.parametrize("size", [9, 14, 16, 20, 24, 40, 100])
@pytest.mark.parametrize("m,hq,hkv,d,partition", [(12, 8, 2, 128, 0), (40, 8, 2, 64, 1024),
                                                  (5, 4, 1, 256, 1024), (80, 4, 1, 128, 0)])
def test_a_hidden_draft_costs_nothing(m, hq, hkv, d, partition, size):
    """K and V of one draft are 2^size times the others'; only it sees itself."""
    n = 430
    pools, q, table, slots, mask, keep = step(n, m, hq, hkv, d, True, "tree", size + m)
    at = m // 2
    keep[:, n - m + at] = False
    keep[at, n - m + at] = True
    mask = pack([sum(1 << j for j in range(m) if keep[i, n - m + j]) for i in range(m)], 2)
    s = slots[n - m + at]
    pools.rows = 0.7 * torch.randn(pools.rows.shape, generator=torch.Generator().manual_seed(3)).to(BF16)
    pools.rows[:, s // 16, :, s % 16] *= 2.0 ** size
    pools.codes, pools.byte = R.quantise(pools.rows)
    out, lse = attend(pools, q, table, n, mask, partition)
    others = [i for i in range(m) if i != at]
    check(out[others], lse[others], q[others], *pools.at(slots), keep[others], d ** -0.5,
          TREE_FLOOR, "others")


@pytest.mark.parametrize("size", [7, 8, 12, 24, 30, 60, 118])
@pytest.mark.parametrize("m,hq,hkv,d,partition", [(12, 8, 2, 128, 0), (40, 8, 2, 64, 1024),
                                                  (5, 4, 1, 256, 1024), (80, 4, 1, 128, 0)])
@pytest.mark.parametrize("where", ["context", "draft"])
def test_a_large_value_of_little_weight(where, m, hq, hkv, d, partition, size):
    """One key's V is 2^size times the others' and its weight 2^-(size + 40)."""
    n = 430
    pools, q, table, slots, mask, keep = step(n, m, hq, hkv, d, True, "chain", size + m)
    g = torch.Generator().manual_seed(4)
    scale = d ** -0.5
    way = torch.randn(d, generator=g)
    q = (way + 0.05 * torch.randn(m, hq, d, generator=g)).to(BF16)
    s = slots[77 if where == "context" else n - m]
    pools.rows[0] = 0.3 * torch.randn(pools.rows[0].shape, generator=g).to(BF16)
    pools.rows[0][s // 16, :, s % 16] = \
        (-way * ((size + 40) * 0.693 / (scale * float(way @ way)))).to(BF16)
    pools.rows[1] = torch.randn(pools.rows[1].shape, generator=g).to(BF16)
    pools.rows[1][s // 16, :, s % 16] *= 2.0 ** size
    pools.codes, pools.byte = R.quantise(pools.rows)
    out, lse = attend(pools, q, table, n, mask, partition)
    check(out, lse, q, *pools.at(slots), keep, scale, TREE_FLOOR, where)


@pytest.mark.parametrize("size", [15, 16, 20, 24, 60, 118])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_large_key_across_the_queries(d, size):
    """A kept key 2^size times the others', in dims where every query is 0."""
    m, n, hq, hkv = 9, 300, 6, 2
    pools, q, table, slots, mask, keep = step(n, m, hq, hkv, d, True, "tree", size)
    g = torch.Generator().manual_seed(5)
    q[..., :16] = 0
    pools.rows = torch.randn(pools.rows.shape, generator=g).to(BF16)
    s = slots[40]
    pools.rows[0][s // 16, :, s % 16, :16] *= 2.0 ** size
    pools.rows[0][s // 16, :, s % 16, 16:] = 0
    pools.codes, pools.byte = R.quantise(pools.rows)
    for partition in (0, 1024):
        out, lse = attend(pools, q, table, n, mask, partition)
        check(out, lse, q, *pools.at(slots), keep, d ** -0.5, TREE_FLOOR, f"partition {partition}")


@pytest.mark.parametrize("sizes", [(60, 0, -60, 30), (-60, -20, 30, 60), (118, -110, 0, 118),
                                   (-118, 118, -118, 118), (-118, -118, -118, -118),
                                   (118, 118, 118, 118)])
@pytest.mark.parametrize("d,m", [(128, 10), (64, 70), (256, 3)])
def test_tiles_of_very_different_values(d, m, sizes):
    """V of every 128 keys at a size of its own: the weights' sum does not follow V."""
    n, hq, hkv = 470, 4, 1
    pools, q, table, slots, mask, keep = step(n, m, hq, hkv, d, True, "chain", m)
    g = torch.Generator().manual_seed(6)
    pools.rows = torch.randn(pools.rows.shape, generator=g).to(BF16)
    for t, e in enumerate(sizes):
        s = slots[128 * t:128 * t + 128]
        pools.rows[1][s // 16, :, s % 16] *= 2.0 ** e
    pools.codes, pools.byte = R.quantise(pools.rows)
    k, v = pools.at(slots)
    top = 2.0 ** -max(sizes)  # near the ends of the range the definition is computed beside 1
    for partition in (0, 1024):
        out, lse = attend(pools, q, table, n, mask, partition)
        check(out.to(torch.float64).cpu() * top, lse, q, k, v * top, keep, d ** -0.5, TREE_FLOOR,
              f"partition {partition}")


@pytest.mark.parametrize("partition", [0, 1024])
@pytest.mark.parametrize("d", [128, 64])
def test_rows_of_every_size_and_shape(d, partition):
    """Scales that vary by 2^N(0, 4) from row to row, zero rows and a NaN row that no draft
    sees among them."""
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        m, n, hq, hkv = 20 + 30 * (seed % 2), 390 + 17 * seed, 8, 2
        pools, q, table, slots, mask, keep = step(n, m, hq, hkv, d, True, "tree", seed)
        size = torch.exp2(4 * torch.randn(pools.rows.shape[:-1] + (1,), generator=g))
        size[0] = torch.exp2(torch.log2(size[0]).clamp(max=2))
        pools.rows = (torch.randn(pools.rows.shape, generator=g) * size).to(BF16)
        for at in (3, 200, n - m + 2):
            pools.rows[:, slots[at] // 16, :, slots[at] % 16] = 0
        blind = n - m + 5
        keep[:, blind] = False
        mask = pack([sum(1 << j for j in range(m) if keep[i, n - m + j]) for i in range(m)], 2)
        pools.rows[:, slots[blind] // 16, :, slots[blind] % 16] = float("nan")
        pools.codes, pools.byte = R.quantise(pools.rows)
        out, lse = attend(pools, q, table, n, mask, partition)
        check(out, lse, q, *pools.at(slots), keep, d ** -0.5, TREE_FLOOR, f"seed {seed}")


@pytest.mark.parametrize("scale", [1.0, 8.0, -8.0])
@pytest.mark.parametrize("d,hkv", [(128, 2), (64, 1)])
def test_scores_that_grow_by_hundreds(d, hkv, scale):
    """Maxima far above the first tile's: the sum's reference has to follow."""
    run([900, 700], [9, 40], 4, hkv, d, fp8=True, scale=scale, partition=1024)
    run([900, 700], [9, 40], 4, hkv, d, fp8=True, scale=scale, sink=True, spread=2.0)


@pytest.mark.parametrize("partition", [0, 1024])
@pytest.mark.parametrize("window,slopes,sink", [(70, False, False), (-1, True, True),
                                                (260, True, True), (-1, False, True)])
@pytest.mark.parametrize("d,m", [(128, 12), (64, 70), (256, 4)])
def test_wide_tiles_under_every_mask(d, m, window, slopes, sink, partition):
    """Scales by 2^N(0, 4) from key to key, with a window, ALiBi slopes, a sink, and a draft
    of NaN values that some drafts see."""
    n, hq, hkv = 420, 8, 2
    pools, q, table, slots, mask, keep = step(n, m, hq, hkv, d, True, "tree", m)
    g = torch.Generator().manual_seed(d)
    ctx = n - m
    depth = torch.tensor([bin(sum(int(keep[i, ctx + j]) << j for j in range(m))).count("1") - 1
                          for i in range(m)], dtype=I32)
    size = torch.exp2(4 * torch.randn(pools.rows.shape[:-1] + (1,), generator=g))
    size[0] = torch.exp2(torch.log2(size[0]).clamp(max=2))
    pools.rows = (torch.randn(pools.rows.shape, generator=g) * size).to(BF16)
    bad = m // 3
    pools.rows[1][slots[ctx + bad] // 16, :, slots[ctx + bad] % 16, 3] = float("nan")
    pools.codes, pools.byte = R.quantise(pools.rows)
    kpos = torch.cat([torch.arange(ctx), ctx + depth.long()])
    qpos = ctx + depth.long()
    if window >= 0:
        keep = keep & (kpos[None] >= qpos[:, None] - window)
    snk = 2 * torch.randn(hq, generator=g) if sink else None
    alibi = torch.exp2(-8.0 * (torch.arange(hq) + 1) / hq) if slopes else None
    bias = None
    if slopes:
        bias = alibi.to(torch.float64)[:, None, None] * \
            (kpos[None] - qpos[:, None]).to(torch.float64)[None]
    kc, vc, ks, vs = pools.device(DEV)
    lse = torch.zeros(m, hq, device=DEV)
    out = pkv.paged_tree_attention(
        q.to(DEV), kc, vc, table.to(DEV), torch.tensor([0, m], dtype=I32, device=DEV),
        torch.tensor([n], dtype=I32, device=DEV), m, n, mask.to(DEV), tree_depth=depth.to(DEV),
        k_scale=ks, v_scale=vs, sink=None if snk is None else snk.to(DEV), window_left=window,
        partition_size=partition, lse=lse, alibi_slopes=None if alibi is None else alibi.to(DEV))
    k, v = pools.at(slots)
    ref, rl, absv, smax = R.attend(q, k, v, keep, d ** -0.5, snk, bias)
    if slopes:
        smax = smax + bias.abs().max()
    R.assert_within(lse, rl, R.lse_bound(rl, smax, d), "lse")
    sees = keep[:, ctx + bad]
    assert not bool(torch.isfinite(out.cpu()[sees]).any())
    # the row's largest weighted value, in the weights' own terms
    floor = torch.zeros(m, hq, 1, dtype=torch.float64)
    for h in range(hq):
        big = v[:, h // 4].abs().amax(-1)
        for i in range(m):
            sc = (k[:, h // 4][keep[i]] @ q[i, h].to(torch.float64)) * d ** -0.5
            if bias is not None:
                sc = sc + bias[h, i][keep[i]]
            floor[i, h] = TREE_FLOOR * sc.numel() * (torch.exp(sc - rl[i, h]) * big[keep[i]]).max()
    bound = R.out_bound(ref, absv, smax, d, 2.0 ** -11 + 2.0 ** -13) + floor
    R.assert_within(out[(~sees).to(DEV)], ref[~sees], bound[~sees], "out")
