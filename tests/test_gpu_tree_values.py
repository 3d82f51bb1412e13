"""What the values of some keys may do to drafts that keep them, that hardly weigh
them, or that do not see them."""
import random

import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R
from tests.test_gpu_tree import pack, tree

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
