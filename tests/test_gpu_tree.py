"""paged_tree_attention on the GPU within derived bounds of the 64-bit
attention, over bf16 and 8-bit pools."""
import random

import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
I32 = torch.int32


def tree(n, rng, kind="tree"):
    """(bits per node, depth per node)."""
    if kind == "chain":
        return [(1 << (i + 1)) - 1 for i in range(n)], list(range(n))
    if kind == "random":  # any bits, empty rows among them, bits past the end
        return [0 if rng.random() < 0.3 else rng.getrandbits(n + 9) for _ in range(n)], \
            [rng.randint(0, 5) for _ in range(n)]
    bits, depth = [], []
    for i in range(n):
        par = rng.randint(max(0, i - 5), i - 1) if i else -1
        bits.append((1 << i) | (bits[par] if i else 0))
        depth.append(depth[par] + 1 if i else 0)
    return bits, depth


def pack(bits, words):
    rows = []
    for b in bits:
        w = [(b >> (64 * k)) & (2 ** 64 - 1) for k in range(words)]
        rows.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in w])
    return torch.tensor(rows, dtype=torch.int64).reshape(len(bits), words)


def run(lens, qlens, hq, hkv, d, bs=16, layout="NHD", fp8=False, kind="tree", window=-1,
        sink=False, alibi=False, partition=0, seed=0, nan_draft=False, extra_rows=0,
        check=None, scale=None, spread=1.0):
    g = torch.Generator().manual_seed(seed + d + sum(lens))
    rng = random.Random(seed + sum(qlens))
    nb = sum((n + bs - 1) // bs for n in lens) + 2
    pools = R.Pools(nb, bs, hkv, d, layout, fp8, g, spread=spread)
    table, slots = R.paged(lens, bs, nb, g)
    owned = set(torch.cat(slots).tolist())
    pools.poison([s for s in range(nb * bs) if s not in owned])
    if nan_draft:  # the second draft of every request is NaN
        pools.poison([s[n - m + 1] for s, n, m in zip(slots, lens, qlens) if m > 1])
    total = sum(qlens) + extra_rows
    q = torch.randn(total, hq, d, generator=g).to(BF16)
    words = max(1, (max(qlens) + 63) // 64)
    trees = [tree(m, rng, kind) for m in qlens]
    mask = torch.cat([pack(b, words + 1)[:, :words] for b, _ in trees] +
                     [torch.full((extra_rows, words), -1, dtype=torch.int64)]).contiguous()
    depth = torch.tensor([x for _, ds in trees for x in ds] + [0] * extra_rows, dtype=I32)
    cu = torch.tensor([0] + torch.tensor(qlens).cumsum(0).tolist(), dtype=I32)
    snk = torch.randn(hq, generator=g) if sink else None
    slopes = torch.exp2(-8.0 * (torch.arange(hq) + 1) / hq) if alibi else None
    kc, vc, ks, vs = pools.device(DEV)
    out = torch.full((total, hq, d), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((total, hq), 7.0, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    sc = d ** -0.5 if scale is None else scale
    needs = window >= 0 or alibi
    got = pkv.paged_tree_attention(
        q.to(DEV), kc, vc, table.to(DEV), cu.to(DEV), torch.tensor(lens, dtype=I32, device=DEV),
        max(qlens), max(lens), mask.to(DEV), tree_depth=depth.to(DEV) if needs else None,
        k_scale=ks, v_scale=vs, sink=None if snk is None else snk.to(DEV), window_left=window,
        sm_scale=sc, partition_size=partition, out=out, lse=lse, dev_error=err,
        alibi_slopes=None if slopes is None else slopes.to(DEV), layout=layout)
    assert got is out
    assert pkv.get_device_error(err) == 0
    at = 0
    for i, (n, m) in enumerate(zip(lens, qlens)):
        k, v = pools.at(slots[i])
        ctx = n - m
        bits, dep = trees[i]
        dep = torch.tensor(dep, dtype=torch.int64)
        kpos = torch.cat([torch.arange(ctx), ctx + dep])
        keep = torch.ones(m, n, dtype=torch.bool)
        keep[:, ctx:] = torch.tensor([[bool(b >> j & 1) for j in range(m)] for b in bits])
        if window >= 0:
            keep &= kpos[None] >= (ctx + dep)[:, None] - window
        bias = None
        if slopes is not None:
            bias = slopes.to(torch.float64)[:, None, None] * \
                (kpos[None] - (ctx + dep)[:, None]).to(torch.float64)[None]
        rows = slice(at, at + m)
        ref, rl, absv, smax = R.attend(q[rows], k, v, keep, sc, snk, bias)
        if bias is not None:
            smax = smax + bias.abs().max()
        if nan_draft and m > 1:  # a NaN value makes the whole row NaN where it is kept
            sees = keep[:, ctx + 1]
            assert bool(torch.isnan(out[rows][sees.to(DEV)]).all())
            ref, rl, absv, smax = (x[~sees] for x in (ref, rl, absv, smax))
            o, s = out[rows][(~sees).to(DEV)], lse[rows][(~sees).to(DEV)]
        else:
            o, s = out[rows], lse[rows]
        # bf16 weights: half a step is 2^-8 (f16 ones over 8-bit pools: 2^-11)
        bound = R.out_bound(ref, absv, smax, d, 2.0 ** -11, R.f16_floor(v)) if fp8 else \
            R.out_bound(ref, absv, smax, d, 2.0 ** -8)
        R.assert_within(o, ref, bound, f"out {i}")
        R.assert_within(s, rl, R.lse_bound(rl, smax, d), f"lse {i}")
        at += m
    assert bool((out[at:] == 7.0).all()) and bool((lse[at:] == 7.0).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_small(fp8):
    run([40], [3], 4, 2, 128, fp8=fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout,bs", [("NHD", 16), ("HND", 32), ("NHD", 32), ("HND", 16)])
@pytest.mark.parametrize("d", [64, 80, 96, 112, 128, 256])
def test_head_sizes(d, layout, bs, fp8):
    run([300, 5, 129, 1, 700], [7, 5, 2, 1, 9], 4, 2, d, bs, layout, fp8, sink=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("partition", [0, 128, 256, 1024])
@pytest.mark.parametrize("lens,qlens", [([1], [1]), ([128, 127, 129, 256], [1, 2, 3, 128]),
                                        ([255, 257, 513], [1, 64, 65]),
                                        ([8, 2000, 40], [8, 33, 17])])
def test_lengths_and_partitions(lens, qlens, partition, fp8):
    run(lens, qlens, 8, 2, 128, partition=partition, fp8=fp8, extra_rows=3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 1), (16, 1), (12, 4), (32, 8)])
def test_groups(hq, hkv, fp8):
    run([200, 333], [11, 30], hq, hkv, 64, fp8=fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["chain", "random", "tree"])
@pytest.mark.parametrize("qlen", [1, 31, 64, 100, 256])
def test_masks(kind, qlen, fp8):
    run([qlen, qlen + 70, qlen + 300], [qlen, max(1, qlen // 2), qlen], 4, 2, 64, kind=kind,
        fp8=fp8, sink=kind == "chain")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 1, 3, 17, 128, 300, 4000])
@pytest.mark.parametrize("partition", [0, 128])
def test_window(window, partition, fp8):
    run([600, 20, 1030, 9], [20, 9, 40, 9], 4, 2, 64, window=window, partition=partition,
        fp8=fp8, kind="tree", sink=True)
    run([400, 30], [12, 30], 4, 2, 128, window=window, partition=partition, fp8=fp8,
        kind="random")


@pytest.mark.parametrize("fp8", [False, True])
def test_alibi_and_scales(fp8):
    run([500, 60], [10, 25], 8, 2, 128, alibi=True, fp8=fp8, sink=True)
    run([500, 60], [10, 25], 8, 2, 64, alibi=True, window=40, partition=128, fp8=fp8)
    run([300], [9], 4, 2, 64, scale=-0.05, fp8=fp8)
    run([300], [9], 4, 2, 64, scale=0.0, fp8=fp8)
    run([900], [9], 4, 1, 128, scale=1.0, fp8=fp8)  # peaked rows: maxima that grow late


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_of_very_different_sizes(fp8):
    run([700, 130], [9, 20], 4, 2, 128, spread=5.0, fp8=fp8, scale=1e-3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("partition", [0, 128])
def test_a_nan_draft_reaches_only_the_drafts_that_see_it(partition, fp8):
    run([140, 30, 600], [12, 5, 40], 4, 2, 128, nan_draft=True, partition=partition, fp8=fp8)
    run([140, 30, 600], [12, 5, 40], 4, 2, 64, nan_draft=True, partition=partition, fp8=fp8)


def test_a_chain_is_causal_prefill():
    """A chain of drafts is the causal chunk of varlen_prefill."""
    g = torch.Generator().manual_seed(3)
    lens, qlens, bs = [513, 90], [30, 90], 16
    pools = R.Pools(50, bs, 2, 128, "NHD", False, g)
    table, _ = R.paged(lens, bs, 50, g)
    kc, vc, _, _ = pools.device(DEV)
    q = torch.randn(120, 8, 128, generator=g).to(BF16).to(DEV)
    cu = torch.tensor([0, 30, 120], dtype=I32, device=DEV)
    cuk = torch.tensor([0, 513, 603], dtype=I32, device=DEV)
    mask = torch.cat([pack(tree(m, None, "chain")[0], 2) for m in qlens]).to(DEV)
    a = pkv.paged_tree_attention(q, kc, vc, table.to(DEV), cu,
                                 torch.tensor(lens, dtype=I32, device=DEV), 90, 513, mask)
    b = pkv.varlen_prefill(q, kc, vc, table.to(DEV), cu, cuk, 90, 513)
    # two outputs with bf16 weights and a bf16 rounding each
    v = pools.rows[1].abs().max()
    assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -6 * float(v)


def test_single_drafts_are_decode():
    g = torch.Generator().manual_seed(4)
    lens, bs = [700, 1, 64], 32
    pools = R.Pools(40, bs, 2, 64, "HND", True, g)
    table, _ = R.paged(lens, bs, 40, g)
    dev = pools.device(DEV)
    q = torch.randn(3, 4, 64, generator=g).to(BF16).to(DEV)
    sl = torch.tensor(lens, dtype=I32, device=DEV)
    a = pkv.paged_tree_attention(q, dev[0], dev[1], table.to(DEV),
                                 torch.arange(4, dtype=I32, device=DEV), sl, 1, 700,
                                 torch.ones(3, 1, dtype=torch.int64, device=DEV),
                                 k_scale=dev[2], v_scale=dev[3], layout="HND")
    b = pkv.paged_decode_fp8(q, *dev, table.to(DEV), sl, 700, layout="HND")
    v = pools.at(torch.arange(40 * bs))[1]
    v = v[torch.isfinite(v)].abs().max()
    assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(v)


def test_bad_metadata_is_flagged_and_stays_inside():
    g = torch.Generator().manual_seed(5)
    for fp8 in (False, True):
        pools = R.Pools(12, 16, 1, 64, "NHD", fp8, g)
        kc, vc, ks, vs = pools.device(DEV)
        q = torch.randn(6, 2, 64, generator=g).to(BF16).to(DEV)
        mask = pack([(1 << (i + 1)) - 1 for i in range(6)], 1).to(DEV)
        err = torch.zeros(1, dtype=I32, device=DEV)
        table = torch.tensor([[0, 1, 99, 3], [4, 5, 6, 7]], dtype=I32, device=DEV)

        def call(cu, sl, tab=table, maxq=4, maxl=64, part=0):
            out = torch.full_like(q, 7.0)
            pkv.paged_tree_attention(
                q, kc, vc, tab, torch.tensor(cu, dtype=I32, device=DEV),
                torch.tensor(sl, dtype=I32, device=DEV), maxq, maxl, mask, k_scale=ks, v_scale=vs,
                out=out, dev_error=err, partition_size=part)
            return out, pkv.get_device_error(err, clear=True)

        out, bits = call([0, 3, 6], [64, 64])          # page 99: skipped
        assert bits == pkv.DEVERR_BLOCK_ID
        keep = torch.ones(3, 48, dtype=torch.bool)
        keep[:, 45:] = torch.tensor([[1, 0, 0], [1, 1, 0], [1, 1, 1]], dtype=torch.bool)
        k, v = pools.at(torch.cat([torch.arange(32), 48 + torch.arange(16)]))
        ref, _, absv, smax = R.attend(q[:3].cpu(), k, v, keep, 0.125)
        R.assert_within(out[:3], ref, R.out_bound(ref, absv, smax, 64, 2.0 ** -8), "out")
        ok = table.clamp(max=11)
        for part in (0, 128):
            out, bits = call([0, 3, 6], [2, 64], ok, part=part)   # drafts longer than the length
            assert bits == pkv.DEVERR_SEQLEN and bool((out[:3] == 0).all())
            assert call([0, 3, 6], [64, 65], ok, part=part)[1] == pkv.DEVERR_SEQLEN
            assert call([0, 3, 6], [-1, 64], ok, part=part)[1] == pkv.DEVERR_SEQLEN
            assert call([0, 5, 6], [64, 64], ok, part=part)[1] == pkv.DEVERR_SEQLEN  # q_len > max
            assert call([0, 3, 9], [64, 64], ok, part=part)[1] == pkv.DEVERR_SEQLEN  # past q
            assert call([-2, 1, 4], [64, 64], ok, part=part)[1] == pkv.DEVERR_SEQLEN
            out, bits = call([2, 4, 4], [64, 64], ok, part=part)  # rows of no request
            assert bits == 0
            assert bool((out[:2] == 7.0).all()) and bool((out[4:] == 7.0).all())


def test_captured_replayed_and_on_another_stream():
    g = torch.Generator().manual_seed(6)
    lens, qlens, bs = [700, 65, 300], [20, 5, 64], 16
    for fp8 in (False, True):
        pools = R.Pools(80, bs, 2, 128, "NHD", fp8, g)
        table, _ = R.paged(lens, bs, 80, g)
        kc, vc, ks, vs = pools.device(DEV)
        total = sum(qlens)
        q = torch.randn(total, 8, 128, generator=g).to(BF16).to(DEV)
        rng = random.Random(1)
        mask = torch.cat([pack(tree(m, rng)[0], 1) for m in qlens]).to(DEV)
        args = (q, kc, vc, table.to(DEV), torch.tensor([0, 20, 25, 89], dtype=I32, device=DEV),
                torch.tensor(lens, dtype=I32, device=DEV), 64, 700, mask)
        kw = dict(k_scale=ks, v_scale=vs, partition_size=256)
        want = pkv.paged_tree_attention(*args, **kw)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        other = pkv.paged_tree_attention(*args, stream=side, **kw)
        side.synchronize()
        assert R.same_bits(want, other)
        cap = torch.zeros_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_tree_attention(*args, out=cap, **kw)
        for _ in range(2):
            cap.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert R.same_bits(cap, want)


def test_a_speculative_step_over_the_8_bit_cache():
    """Norm, rotation and quantised write of the drafts, then their attention:
    as a server runs them, against the definition step by step."""
    g = torch.Generator().manual_seed(7)
    lens, qlens, bs, hq, hkv, d = [200, 33], [6, 9], 16, 8, 2, 128
    pools = R.Pools(20, bs, hkv, d, "NHD", True, g)
    table, slots = R.paged(lens, bs, 20, g)
    dev = pools.device(DEV)
    total = sum(qlens)
    qkv = torch.randn(total, hq + 2 * hkv, d, generator=g).to(BF16).to(DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    qo = torch.empty(total, hq, d, dtype=BF16, device=DEV)
    ko = torch.empty(total, hkv, d, dtype=BF16, device=DEV)
    rng = random.Random(2)
    trees = [tree(m, rng) for m in qlens]
    depth = torch.tensor([x for _, ds in trees for x in ds], dtype=I32)
    ctx = torch.tensor([n - m for n, m in zip(lens, qlens)]).repeat_interleave(torch.tensor(qlens))
    at = torch.cat([s[-m:] for s, m in zip(slots, qlens)])
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).to(DEV)
    tab = pkv.rope_cos_sin_table(512, d)
    pkv.qk_norm_rope_reshape_and_cache(q, k, v, dev[0], dev[1], (ctx + depth).to(DEV), at.to(DEV),
                                       tab, w[0], w[1], query_out=qo, key_out=ko, k_scale=dev[2],
                                       v_scale=dev[3])
    out = pkv.paged_tree_attention(
        qo, dev[0], dev[1], table.to(DEV), torch.tensor([0, 6, 15], dtype=I32, device=DEV),
        torch.tensor(lens, dtype=I32, device=DEV), 9, 200,
        torch.cat([pack(b, 1) for b, _ in trees]).to(DEV), tree_depth=depth.to(DEV),
        k_scale=dev[2], v_scale=dev[3])
    # the pools as they are now
    pools.codes = torch.stack([dev[0], dev[1]]).view(torch.uint8).cpu().permute(0, 1, 3, 2, 4)
    pools.byte = torch.stack([dev[2], dev[3]]).cpu()
    codes, byte = R.quantise(torch.stack([ko.cpu(), v.cpu()]))
    for i in range(2):
        assert torch.equal(pools.codes[i][at // bs, :, at % bs], codes[i])
        assert torch.equal(pools.byte[i][at // bs, :, at % bs], byte[i])
    row = 0
    for i, (n, m) in enumerate(zip(lens, qlens)):
        kk, vv = pools.at(slots[i])
        keep = torch.ones(m, n, dtype=torch.bool)
        keep[:, n - m:] = torch.tensor([[bool(b >> j & 1) for j in range(m)] for b in trees[i][0]])
        ref, _, absv, smax = R.attend(qo[row:row + m].cpu(), kk, vv, keep, d ** -0.5)
        R.assert_within(out[row:row + m], ref, R.out_bound(ref, absv, smax, d, 2.0 ** -8), "out")
        row += m
