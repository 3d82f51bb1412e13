"""update_page_bounds on the GPU, bit for bit."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R
from tests import _sparse as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, I32, U8, I8 = torch.bfloat16, torch.int32, torch.uint8, torch.int8


def fresh(nb, hkv, d):
    return (torch.full((nb, hkv, 2, d), 99, dtype=I8, device=DEV),
            torch.full((nb, hkv), 33, dtype=U8, device=DEV))


def values(pools):
    """The keys as float64 [nb, Hkv, bs, D]."""
    nb, bs = pools.nb, pools.bs
    k, _ = pools.at(torch.arange(nb * bs))
    return k.view(nb, bs, pools.hkv, pools.d).permute(0, 2, 1, 3)


def expect(pools, slots, b, s):
    keys = values(pools)
    rows = {}
    for x in slots:
        if 0 <= x < pools.nb * pools.bs:
            rows[x // pools.bs] = x % pools.bs + 1
    want, wantb = b.cpu().clone(), s.cpu().clone()
    for page, n in rows.items():
        want[page], wantb[page] = S.bounds(keys[page, :, :n])
    return want, wantb


def check(pools, slots, layout, err_bits=0):
    kc, _, ks, _ = pools.device(DEV)
    b, s = fresh(pools.nb, pools.hkv, pools.d)
    want, wantb = expect(pools, slots, b, s)
    err = torch.zeros(1, dtype=I32, device=DEV)
    pkv.update_page_bounds(kc, b, s, torch.tensor(slots, dtype=torch.int64, device=DEV), k_scale=ks,
                           dev_error=err, layout=layout)
    assert torch.equal(s.cpu(), wantb)
    assert torch.equal(b.cpu(), want)
    assert pkv.get_device_error(err) == err_bits


def token_slots(lens, old, bs, nb, g):
    _, slots = R.paged(lens, bs, nb, g)
    return [x for s, a in zip(slots, old) for x in s[a:].tolist()]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 16), (2, 80, 32), (3, 96, 16), (8, 128, 16),
                                      (1, 112, 32), (4, 256, 16), (8, 128, 32), (2, 64, 32)])
def test_tokens(fp8, layout, hkv, d, bs):
    """One token each, chunks that begin and end inside pages, padding between."""
    g = torch.Generator().manual_seed(d + bs + hkv)
    lens, old = [1, 16, 33, 70, 200, 17], [0, 15, 32, 9, 100, 0]
    nb = 40
    pools = R.Pools(nb, bs, hkv, d, layout, fp8, g, spread=3.0)
    slots = token_slots(lens, old, bs, nb, g)
    slots[3:3] = [-1] * 5
    check(pools, slots + [-1, -7], layout)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_tokens(fp8):
    """Prompts over many CTAs, of a ragged count."""
    g = torch.Generator().manual_seed(5)
    lens, old = [4099, 2000, 777], [0, 30, 770]
    pools = R.Pools(450, 16, 2, 64, "NHD", fp8, g)
    check(pools, token_slots(lens, old, 16, 450, g), "NHD")


def test_rows_behind_the_last_token_are_not_read():
    """Rows beyond the last written one may hold anything; rows before count."""
    g = torch.Generator().manual_seed(6)
    pools = R.Pools(4, 16, 2, 128, "HND", False, g)
    pools.poison([1 * 16 + x for x in range(5, 16)])
    check(pools, [1 * 16 + 4], "HND")
    pools.poison([1 * 16 + 2])                 # now a row before it is NaN
    check(pools, [1 * 16 + 4], "HND")


@pytest.mark.parametrize("fp8", [False, True])
def test_not_finite(fp8):
    g = torch.Generator().manual_seed(7)
    pools = R.Pools(6, 16, 2, 64, "NHD", fp8, g)
    if fp8:
        pools.byte[0][2, 1, 7] = 255
        pools.byte[0][3, 0, 0] = 254          # codes times 2^127: beyond a float
    else:
        pools.rows[0][2, 1, 7, 3] = float("nan")
        pools.rows[0][3, 0, 0, 63] = float("inf")
        pools.rows[0][4, 1, 15, 0] = float("-inf")
    kc = values(pools)
    if fp8:  # a float's infinity counts as not finite
        kc[kc.abs() > 3.4028235677973366e38] = float("inf")
    k, _, ks, _ = pools.device(DEV)
    b, s = fresh(6, 2, 64)
    pkv.update_page_bounds(k, b, s, torch.arange(96, device=DEV), k_scale=ks)
    want, wantb = S.bounds(kc)
    assert torch.equal(s.cpu(), wantb) and torch.equal(b.cpu(), want)
    assert int((wantb == 255).sum()) >= 2


def test_special_values():
    """Zeros, subnormals, 127 * 2^e and the values beside it, bf16's ends, tiny beside huge."""
    rows = torch.zeros(12, 1, 16, 64)
    g = torch.Generator().manual_seed(8)
    base = torch.randn(16, 64, generator=g)
    rows[1] = -0.0
    rows[2, 0, 3, 5] = 127.0
    rows[3, 0, 3, 5] = -127.5                 # 1.9921875 * 2^6
    rows[4, 0, 3, 5] = 2.0 ** 40 * 1.984375
    rows[5, 0] = base * 2.0 ** -130
    rows[6, 0] = base * 2.0 ** 120
    rows[7, 0, 0, 0] = torch.finfo(BF16).max
    rows[7, 0, 1, 1] = 2.0 ** -133            # the smallest subnormal: up to 1, down to 0
    rows[7, 0, :, 2] = -2.0 ** -133
    rows[7, 0, :, 3] = 2.0 ** -133
    rows[8, 0] = base.abs() + 1               # all above zero
    rows[9, 0] = -base.abs() - 1
    rows[10, 0, 0, 0] = torch.finfo(BF16).smallest_normal
    rows[11, 0] = torch.round(base * 20)
    pools = R.Pools(12, 16, 1, 64, "NHD", False, g)
    pools.rows[0] = rows.to(BF16)
    check(pools, list(range(12 * 16)), "NHD")


def test_bounds_hold():
    """Every key lies between its page's bounds."""
    g = torch.Generator().manual_seed(9)
    pools = R.Pools(30, 16, 2, 128, "NHD", False, g, spread=4.0)
    kc, _, _, _ = pools.device(DEV)
    b, s = fresh(30, 2, 128)
    pkv.update_page_bounds(kc, b, s, torch.arange(480, device=DEV))
    unit = S.pow2(s.cpu().to(I32) - 127)[..., None, None]
    lim = b.cpu().to(torch.float64) * unit
    keys = values(pools)
    assert bool((keys >= lim[:, :, :1]).all()) and bool((keys <= lim[:, :, 1:]).all())


def test_slots_outside_the_pool():
    g = torch.Generator().manual_seed(10)
    pools = R.Pools(3, 32, 2, 64, "NHD", False, g)
    check(pools, [5, 96, 40, 41, 1 << 40, -1], "NHD", pkv.DEVERR_SLOT)


def test_skipped_tokens_inside_a_page():
    """Tokens of a page that are not side by side: the last one counts."""
    g = torch.Generator().manual_seed(11)
    pools = R.Pools(8, 16, 1, 64, "NHD", False, g)
    check(pools, [0, -1, -1, 1] + [-1] * 31 + [2, 40, 3] + [16, 48] + [17], "NHD")


def test_no_tokens_and_a_graph():
    g = torch.Generator().manual_seed(12)
    pools = R.Pools(8, 16, 2, 64, "NHD", False, g)
    kc, _, _, _ = pools.device(DEV)
    b, s = fresh(8, 2, 64)
    slots = torch.full((40,), -1, dtype=torch.int64, device=DEV)
    pkv.update_page_bounds(kc, b, s, slots[:0])
    pkv.update_page_bounds(kc, b, s, slots)
    assert bool((b == 99).all()) and bool((s == 33).all())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.update_page_bounds(kc, b, s, slots)
    slots[:20] = torch.arange(30, 50, device=DEV)
    want, wantb = expect(pools, list(range(30, 50)), b, s)
    graph.replay()
    assert torch.equal(b.cpu(), want) and torch.equal(s.cpu(), wantb)
