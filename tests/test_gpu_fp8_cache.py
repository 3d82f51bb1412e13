"""The 8-bit cache on the GPU: quantised writes and read-back bit for bit,
decode over e4m3 pages within derived bounds of the 64-bit attention."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def empty_pools(nb, bs, hkv, d, layout):
    shape = (nb, bs, hkv, d) if layout == "NHD" else (nb, hkv, bs, d)
    return [torch.full(shape, 0x11, dtype=U8, device=DEV).view(R.E4M3) for _ in range(2)] + \
        [torch.full((nb, hkv, bs), 77, dtype=U8, device=DEV) for _ in range(2)]


def check_written(key, value, slots, pools, layout, bs):
    """Every slot of the pools: the reference's bits where written, else untouched."""
    for x, pool, scale in ((key, pools[0], pools[2]), (value, pools[1], pools[3])):
        codes, byte = R.quantise(x.cpu())
        want = torch.full(pool.shape, 0x11, dtype=U8)
        wantb = torch.full(scale.shape, 77, dtype=U8)
        keep = slots >= 0
        s = slots[keep]
        b, o = s // bs, s % bs
        if layout == "NHD":
            want[b, o] = codes[keep]
        else:
            want[b, :, o] = codes[keep]
        wantb[b, :, o] = byte[keep]
        assert torch.equal(pool.view(U8).cpu(), want)
        assert torch.equal(scale.cpu(), wantb)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,hkv,d,bs", [(1, 1, 64, 16), (3, 2, 80, 32), (37, 8, 128, 16),
                                             (65, 3, 96, 16), (130, 1, 112, 32), (19, 4, 256, 16),
                                             (4099, 8, 128, 32)])
def test_write(layout, dtype, tokens, hkv, d, bs):
    g = gen(tokens + d)
    nb = (tokens + bs - 1) // bs + 3
    x = torch.randn(2, tokens, hkv, d, generator=g) * \
        torch.exp2(6 * torch.randn(2, tokens, hkv, 1, generator=g))
    x = x.to(dtype)
    slots = torch.randperm(nb * bs, generator=g)[:tokens]
    slots[::7] = -1
    pools = empty_pools(nb, bs, hkv, d, layout)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.reshape_and_cache_fp8(x[0].to(DEV), x[1].to(DEV), *pools, slots.to(DEV), layout=layout,
                              dev_error=err)
    check_written(x[0], x[1], slots, pools, layout, bs)
    assert pkv.get_device_error(err) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_write_special_rows(dtype):
    """Zeros, signed zeros, subnormals, the scale's borders, the largest finite
    values, NaN and infinities."""
    fi = torch.finfo(dtype)
    rows = torch.zeros(16, 1, 64)
    g = gen(3)
    base = torch.randn(64, generator=g)
    base[0] = 0.0
    base[1] = -0.0
    rows[1] = base
    rows[2, 0, 5] = 448.0                    # exactly 2^0 * 448
    rows[3, 0, 5] = 450.0 if dtype is BF16 else 448.00003
    rows[4] = base * 2.0 ** -130             # subnormal values
    rows[5] = base.sign() * fi.max           # saturates at 448 * 2^119
    rows[6] = base
    rows[6, 0, 9] = float("nan")
    rows[7] = base
    rows[7, 0, 63] = float("inf")
    rows[8] = base
    rows[8, 0, 0] = float("-inf")
    rows[9, 0, 3] = fi.smallest_normal
    rows[10] = -0.0
    rows[11] = torch.linspace(-448, 448, 64)
    rows[12] = torch.arange(64) * 2.0 ** -9  # the subnormal codes, and ties between codes
    rows[12, 0, 63] = 448.0
    rows[13] = (torch.arange(64) + 0.5) * 2.0 ** -9
    rows[13, 0, 63] = 448.0
    rows[14] = torch.arange(64).float() + 0.5
    rows[14, 0, 0] = 300.0
    rows[15, 0, 7] = 1e30
    x = rows.to(dtype)
    pools = empty_pools(2, 16, 1, 64, "NHD")
    slots = torch.arange(16)
    pkv.reshape_and_cache_fp8(x.to(DEV), x.flip(0).to(DEV), *pools, slots.to(DEV))
    check_written(x, x.flip(0), slots, pools, "NHD", 16)


def test_write_strided_and_skipped():
    """Slices of one fused projection; slots outside the pool are flagged and
    change nothing; an empty call is a no-op."""
    g = gen(8)
    t, hq, hkv, d, bs = 33, 6, 2, 128, 16
    qkv = torch.randn(t, hq + 2 * hkv, d, generator=g).to(BF16).to(DEV)
    key, value = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pools = empty_pools(4, bs, hkv, d, "HND")
    slots = torch.randperm(64, generator=g)[:t]
    bad = slots.clone()
    bad[4], bad[9] = 64, 1 << 40
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.reshape_and_cache_fp8(key, value, *pools, bad.to(DEV), layout="HND", dev_error=err)
    want = bad.clone()
    want[4] = want[9] = -1
    check_written(key, value, want, pools, "HND", bs)
    assert pkv.get_device_error(err) == pkv.DEVERR_SLOT
    pkv.reshape_and_cache_fp8(key[:0], value[:0], *pools, bad[:0].to(DEV), layout="HND")
    check_written(key, value, want, pools, "HND", bs)


def test_read_back_of_every_code_and_scale():
    """code * 2^(byte - 127) rounded once to bf16, for all codes under scales
    over the whole range."""
    codes = torch.arange(256, dtype=U8)
    codes[127] = codes[255] = 0              # e4m3's NaN codes are not valid in a pool
    bytes_ = torch.tensor([0, 1, 2, 6, 7, 8, 64, 119, 120, 121, 126, 127, 128, 133, 134, 135,
                           136, 180, 240, 245, 246, 255], dtype=U8)
    n = bytes_.numel()
    kc = codes.view(1, 1, 1, 256).repeat(2, 16, 1, 1).to(DEV).view(R.E4M3)
    sc = torch.zeros(2, 1, 16, dtype=U8)
    sc.view(-1)[:n] = bytes_
    table = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    k, v = pkv.gather_cache_fp8(kc, kc, sc.to(DEV), sc.to(DEV), table, cu, n)
    want = (R.CODE_VALUES[codes.long()][None] * R.scales(bytes_)[:, None])
    # one rounding: float64 -> bf16 through a float32 that holds these exactly
    want = want.to(torch.float32).to(BF16)
    got = k.cpu()[:, 0]
    ok = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert bool(ok.all()), (got[~ok][:8], want[~ok][:8])
    assert R.same_bits(k, v)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("lens,hkv,d,bs", [([1], 1, 64, 16), ([5, 0, 33, 16], 2, 80, 16),
                                           ([700, 1, 0, 64, 31], 8, 128, 32), ([0, 0], 4, 96, 16),
                                           ([17, 300], 3, 256, 16), ([2500] * 3, 4, 112, 16)])
def test_gather(layout, lens, hkv, d, bs):
    g = gen(sum(lens) + d)
    nb = sum((n + bs - 1) // bs for n in lens) + 3
    pools = R.Pools(nb, bs, hkv, d, layout, True, g, spread=3.0)
    table, slots = R.paged(lens, bs, nb, g)
    pools.poison([s for s in range(nb * bs) if s not in set(torch.cat(slots).tolist())])
    total = sum(lens) + 3                    # three rows behind the last request
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    key = torch.full((total, hkv, d), 9.0, dtype=BF16, device=DEV)
    value = key.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pkv.gather_cache_fp8(*pools.device(DEV), table.to(DEV), cu, total, key=key, value=value,
                               dev_error=err, layout=layout)
    assert got[0] is key and got[1] is value
    wk, wv = pools.at(torch.cat(slots))
    for x, w in ((key, wk), (value, wv)):
        assert torch.equal(x[:total - 3].cpu().to(torch.float64), w)
        assert bool((x[total - 3:] == 9.0).all())
    assert pkv.get_device_error(err) == 0


def test_gather_flags_bad_pages_and_offsets():
    g = gen(2)
    pools = R.Pools(6, 16, 2, 64, "NHD", True, g)
    dev = pools.device(DEV)
    table = torch.tensor([[0, 1, -1], [2, 99, 3]], dtype=torch.int32)
    cu = torch.tensor([0, 20, 68], dtype=torch.int32)
    key = torch.full((68, 2, 64), 5.0, dtype=BF16, device=DEV)
    value = key.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.gather_cache_fp8(*dev, table.to(DEV), cu.to(DEV), 68, key=key, value=value, dev_error=err)
    assert pkv.get_device_error(err, clear=True) == pkv.DEVERR_BLOCK_ID
    assert bool((key[36:52] == 5.0).all())               # page 99
    slots = torch.cat([torch.arange(20), 32 + torch.arange(16), 48 + torch.arange(16)])
    rows = torch.cat([torch.arange(36), torch.arange(52, 68)])
    assert torch.equal(key[rows.to(DEV)].cpu().to(torch.float64), pools.at(slots)[0])
    # offsets that decrease or leave the output; a request longer than its table
    for bad, bits in (([0, 30, 20], pkv.DEVERR_SEQLEN), ([0, 20, 90], pkv.DEVERR_SEQLEN),
                      ([-4, 20, 40], pkv.DEVERR_SEQLEN)):
        pkv.gather_cache_fp8(*dev, table[:, :2].abs().clamp(max=3).to(DEV).contiguous(),
                             torch.tensor(bad, dtype=torch.int32, device=DEV), 68,
                             dev_error=err)
        assert pkv.get_device_error(err, clear=True) & bits, bad


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
def run_decode(lens, hq, hkv, d, bs, layout="NHD", window=-1, sink=False, alibi=False,
               partition=512, seed=0, spread=1.0, q_scale=1.0, poison=True, max_seqlen=None):
    g = gen(seed + d + sum(lens))
    nb = sum((n + bs - 1) // bs for n in lens) + 2
    pools = R.Pools(nb, bs, hkv, d, layout, True, g, spread=spread)
    table, slots = R.paged(lens, bs, nb, g)
    if poison:  # unowned slots, the rest of the last pages among them
        pools.poison([s for s in range(nb * bs) if s not in set(torch.cat(slots).tolist())])
    q = (torch.randn(len(lens), hq, d, generator=g) * q_scale).to(BF16)
    snk = torch.randn(hq, generator=g) if sink else None
    slopes = torch.exp2(-8.0 * (torch.arange(hq) + 1) / hq) if alibi else None
    lse = torch.full((len(lens), hq), 7.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev = pools.device(DEV)
    out = pkv.paged_decode_fp8(
        q.to(DEV), *dev, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
        max(lens) if max_seqlen is None else max_seqlen, sink=None if snk is None else snk.to(DEV),
        window_left=window, partition_size=partition, lse=lse, dev_error=err,
        alibi_slopes=None if slopes is None else slopes.to(DEV), layout=layout)
    assert pkv.get_device_error(err) == 0
    for i, n in enumerate(lens):
        k, v = pools.at(slots[i])
        pos = torch.arange(n)
        keep = torch.ones(1, n, dtype=torch.bool)
        if window >= 0:
            keep &= pos >= n - 1 - window
        bias = None if slopes is None else \
            slopes.to(torch.float64)[:, None, None] * (pos - (n - 1)).to(torch.float64)[None, None]
        ref, rl, absv, smax = R.attend(q[i:i + 1], k, v, keep, d ** -0.5, snk, bias)
        if bias is not None:  # the bias is one more fp32 term of the score
            smax = smax + bias.abs().max()
        bound = R.out_bound(ref, absv, smax, d, 2.0 ** -11, R.f16_floor(v))
        R.assert_within(out[i:i + 1], ref, bound, f"out {i}")
        R.assert_within(lse[i:i + 1], rl, R.lse_bound(rl, smax, d), f"lse {i}")


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("d", [64, 80, 96, 112, 128, 256])
def test_decode_head_sizes(d, bs, layout):
    run_decode([1, 31, 0, 33, 700, 513], 8, 2, d, bs, layout)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (7, 1), (8, 1), (9, 1), (16, 1), (32, 2),
                                    (10, 5), (24, 8)])
def test_decode_groups(hq, hkv):
    run_decode([64, 5, 1030], hq, hkv, 128, 16, sink=True)
    run_decode([64, 5, 300], hq, hkv, 64, 32, "HND")


@pytest.mark.parametrize("window", [0, 1, 15, 16, 40, 511, 512, 5000])
@pytest.mark.parametrize("partition", [32, 512])
def test_decode_window(window, partition):
    run_decode([1, 17, 0, 600, 1025], 4, 2, 64, 16, window=window, partition=partition, sink=True)


@pytest.mark.parametrize("partition", [16, 48, 64, 512, 4096])
def test_decode_partitions(partition):
    run_decode([1, 15, 16, 17, 2100], 8, 2, 128, 16, partition=partition)


def test_decode_alibi_sink_and_many_partitions():
    run_decode([40, 3000], 8, 2, 128, 16, alibi=True, sink=True, partition=64)
    run_decode([9000], 8, 1, 64, 32, alibi=True, partition=128)


def test_decode_rows_of_very_different_sizes():
    """Scale bytes spread over 2^+-40: the V weights' common gauge moves all the
    time; large and tiny queries."""
    run_decode([400, 33], 4, 2, 64, 16, spread=4.0, q_scale=0.05)
    run_decode([400, 33], 4, 2, 128, 16, spread=0.0, q_scale=1e-3)
    run_decode([1, 3], 4, 2, 128, 16, spread=6.0, q_scale=1e-8)


def test_decode_a_nan_row_reaches_only_those_who_attend_it():
    g = gen(4)
    lens = [40, 200]
    pools = R.Pools(20, 16, 1, 64, "NHD", True, g)
    table, slots = R.paged(lens, 16, 20, g)
    pools.poison(slots[1][:1])               # the second sequence's first key
    q = torch.randn(2, 4, 64, generator=g).to(BF16).to(DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = pkv.paged_decode_fp8(q, *pools.device(DEV), table.to(DEV), sl, 200)
    assert bool(torch.isfinite(out[0]).all()) and bool(torch.isnan(out[1]).all())
    out = pkv.paged_decode_fp8(q, *pools.device(DEV), table.to(DEV), sl, 200, window_left=150)
    assert bool(torch.isfinite(out).all())


def test_decode_flags_bad_pages_and_lengths():
    g = gen(5)
    pools = R.Pools(8, 16, 1, 64, "NHD", True, g)
    dev = pools.device(DEV)
    q = torch.randn(1, 2, 64, generator=g).to(BF16).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.tensor([[3, -1, 5]], dtype=torch.int32, device=DEV)
    out = pkv.paged_decode_fp8(q, *dev, table, torch.tensor([48], dtype=torch.int32, device=DEV),
                               48, dev_error=err)
    assert pkv.get_device_error(err, clear=True) == pkv.DEVERR_BLOCK_ID
    k, v = pools.at(torch.cat([48 + torch.arange(16), 80 + torch.arange(16)]))
    ref, _, absv, smax = R.attend(q.cpu(), k, v, torch.ones(1, 32, dtype=torch.bool), 0.125)
    R.assert_within(out, ref, R.out_bound(ref, absv, smax, 64, 2.0 ** -11), "out")
    for n in (-3, 49, 1 << 30):
        pkv.paged_decode_fp8(q, *dev, table.clamp(min=0),
                             torch.tensor([n], dtype=torch.int32, device=DEV), 48, dev_error=err)
        assert pkv.get_device_error(err, clear=True) == pkv.DEVERR_SEQLEN


def test_decode_agrees_with_the_bf16_cache():
    """The read-back rows in bf16 pages give the same attention."""
    g = gen(6)
    lens, bs, nb = [300, 1000, 64], 16, 90
    pools = R.Pools(nb, bs, 2, 128, "NHD", True, g)
    table, slots = R.paged(lens, bs, nb, g)
    dev = pools.device(DEV)
    kc, vc = (torch.zeros(nb, bs, 2, 128, dtype=BF16, device=DEV) for _ in range(2))
    cu = torch.tensor([0, 300, 1300, 1364], dtype=torch.int32, device=DEV)
    k, v = pkv.gather_cache_fp8(*dev, table.to(DEV), cu, 1364)
    pkv.reshape_and_cache(k, v, kc, vc, torch.cat(slots).to(DEV))
    q = torch.randn(3, 8, 128, generator=g).to(BF16).to(DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    a = pkv.paged_decode_fp8(q, *dev, table.to(DEV), sl, 1000)
    b = pkv.paged_decode(q, kc, vc, table.to(DEV), sl, 1000)
    # two bf16 roundings of the output, and of the bf16 cache's weights
    bound = 2.0 ** -7 * b.abs().float() + 2.0 ** -7 * float(v.abs().max()) / 8
    assert bool(((a.float() - b.float()).abs() <= bound).all())


def test_a_step_captured_replayed_and_on_another_stream():
    """Write, decode and read-back in a CUDA graph, replayed twice, and on a
    stream of their own: the eager bits each time."""
    g = gen(7)
    lens, bs, nb = [33, 700, 512], 16, 100
    pools = R.Pools(nb, bs, 2, 128, "NHD", True, g)
    table, slots = R.paged(lens, bs, nb, g)
    table = table.to(DEV)
    new = torch.randn(2, 3, 2, 128, generator=g).to(BF16).to(DEV)
    at = torch.stack([s[-1] for s in slots]).to(DEV)
    q = torch.randn(3, 8, 128, generator=g).to(BF16).to(DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 33, 733, 1245], dtype=torch.int32, device=DEV)

    def step(dev, out, k, v, stream=None):
        pkv.reshape_and_cache_fp8(new[0], new[1], *dev, at, stream=stream)
        pkv.paged_decode_fp8(q, *dev, table, sl, 700, out=out, stream=stream)
        pkv.gather_cache_fp8(*dev, table, cu, 1245, key=k, value=v, stream=stream)

    def fresh():
        return (pools.device(DEV), torch.zeros_like(q),
                torch.zeros(1245, 2, 128, dtype=BF16, device=DEV),
                torch.zeros(1245, 2, 128, dtype=BF16, device=DEV))

    want = fresh()
    step(*want)
    side = torch.cuda.Stream()
    other = fresh()
    torch.cuda.synchronize()
    step(*other, stream=side)
    side.synchronize()
    cap = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*cap)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got in (other, cap):
        for a, b in zip(got[0] + got[1:], want[0] + want[1:]):
            assert R.same_bits(a, b)
