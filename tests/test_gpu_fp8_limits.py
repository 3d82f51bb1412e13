"""The 8-bit cache and the tree attention where a long-running server takes
them: pages beyond 32-bit offsets, workspaces shared between captured graphs,
two streams at once, many requests, more kv heads than SMs."""
import random

import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R
from tests.test_gpu_tree import pack, run, tree

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, I32 = torch.bfloat16, torch.int32


def _tree_args(qlens, hq, d, g, rng):
    total = sum(qlens)
    q = torch.randn(total, hq, d, generator=g).to(BF16).to(DEV)
    mask = torch.cat([pack(tree(m, rng)[0], 1) for m in qlens]).to(DEV)
    cu = torch.tensor([0] + torch.tensor(qlens).cumsum(0).tolist(), dtype=I32, device=DEV)
    return q, mask, cu


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("fp8", [True, False])
def test_pages_beyond_32_bit_offsets(fp8, layout):
    """The same rows in a small pool and at the end of one of more than 2^32
    bytes: every call gives the same bits."""
    g = torch.Generator().manual_seed(11)
    bs, hkv, hq, d, n = 16, 8, 16, 128, 200
    far = 2 ** 32 // (bs * hkv * d) + 2 ** 15    # pages; the pools hold a few more
    lens = [n, 77]
    small = 24
    table, slots = R.paged(lens, bs, small, g)
    key, value = torch.randn(2, sum(lens), hkv, d, generator=g).to(BF16).to(DEV)
    query = torch.randn(sum(lens), hq, d, generator=g).to(BF16).to(DEV)
    at = torch.cat(slots).to(DEV)
    pos = torch.cat([torch.arange(m) for m in lens]).to(DEV)
    tab = pkv.rope_cos_sin_table(256, d)
    w = torch.ones(d, device=DEV)
    sl = torch.tensor(lens, dtype=I32, device=DEV)
    q, mask, cu = _tree_args([9, 5], hq, d, g, random.Random(3))
    results = []
    for base, nb in ((0, small), (far, far + small)):
        shape = (nb, bs, hkv, d) if layout == "NHD" else (nb, hkv, bs, d)
        kc, vc = (torch.empty(shape, dtype=torch.uint8 if fp8 else BF16, device=DEV)
                  for _ in range(2))
        if base:
            assert kc.numel() > 2 ** 32
        bt = (table.clamp(min=0) + base).to(DEV)
        got = []
        if fp8:
            kc, vc = kc.view(R.E4M3), vc.view(R.E4M3)
            ks, vs = (torch.empty(nb, hkv, bs, dtype=torch.uint8, device=DEV) for _ in range(2))
            dev = (kc, vc, ks, vs)
            ck = torch.tensor([0, n, n + 77], dtype=I32, device=DEV)
            pkv.reshape_and_cache_fp8(key, value, *dev, at + base * bs, layout=layout)
            got += pkv.gather_cache_fp8(*dev, bt, ck, n + 77, layout=layout)
        else:
            ks = vs = None
        qo, ko = torch.empty_like(query), torch.empty_like(key)
        pkv.qk_norm_rope_reshape_and_cache(query, key, value, kc, vc, pos, at + base * bs, tab, w,
                                           w, query_out=qo, key_out=ko, k_scale=ks, v_scale=vs,
                                           layout=layout)
        if fp8:
            got += pkv.gather_cache_fp8(*dev, bt, ck, n + 77, layout=layout)
            got.append(pkv.paged_decode_fp8(q[:2], *dev, bt, sl, n, layout=layout))
        got.append(pkv.paged_tree_attention(q, kc, vc, bt, cu, sl, 9, n, mask, k_scale=ks,
                                            v_scale=vs, layout=layout))
        results.append([qo, ko] + got)
        del kc, vc, ks, vs
    for i, (a, b) in enumerate(zip(*results)):
        assert bool(torch.isfinite(a.float()).all())
        assert R.same_bits(a, b), i


def _problem(lens, qlens, fp8, seed):
    g = torch.Generator().manual_seed(seed)
    bs, hkv, hq, d = 16, 2, 8, 128
    nb = sum((n + bs - 1) // bs for n in lens)
    pools = R.Pools(nb, bs, hkv, d, "NHD", fp8, g)
    table, _ = R.paged(lens, bs, nb, g)
    kc, vc, ks, vs = pools.device(DEV)
    q, mask, cu = _tree_args(qlens, hq, d, g, random.Random(seed))
    sl = torch.tensor(lens, dtype=I32, device=DEV)
    args = (q, kc, vc, table.clamp(min=0).to(DEV), cu, sl, max(qlens), max(lens), mask)
    calls = [lambda **kw: pkv.paged_tree_attention(*args, k_scale=ks, v_scale=vs, **kw)]
    if fp8:
        q1 = q[:len(lens)].contiguous()
        calls.append(lambda **kw: pkv.paged_decode_fp8(q1, kc, vc, ks, vs, args[3], sl, max(lens),
                                                       partition_size=128, **kw))
    return calls


def test_graphs_share_a_workspace():
    """Two captured steps of different shapes with one workspace, full of NaN at
    first, replayed in turn: the bits of calls with workspaces of their own."""
    calls = _problem([700, 65, 300], [20, 5, 60], True, 1) + \
        _problem([40, 2000], [3, 9], True, 2) + _problem([900], [64], False, 3)
    want = [c() for c in calls]
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(w) for w in want]
    graphs = []
    for part in (slice(0, 2), slice(2, 5)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for c, o in zip(calls[part], outs[part]):
                c(workspace=ws, out=o)
        graphs.append(graph)
    for first in (0, 1, 0):
        for o in outs:
            o.fill_(7.0)
        graphs[first].replay()
        graphs[1 - first].replay()
        torch.cuda.synchronize()
        for i, (o, w) in enumerate(zip(outs, want)):
            assert R.same_bits(o, w), i


def test_two_streams_at_once():
    calls = _problem([700, 65, 300], [20, 5, 60], True, 4)[:1] + \
        _problem([1500, 65], [33, 5], False, 5)
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[c(stream=s) for c, s in zip(calls, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for outs in got:
        assert all(R.same_bits(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("fp8", [False, True])
def test_many_requests(fp8):
    """More requests than a warp, some without drafts, some longer than others."""
    rng = random.Random(9)
    lens = [rng.choice([1, 3, 40, 130]) for _ in range(150)] + [2500] + [17] * 20
    qlens = [min(n, rng.choice([0, 1, 2, 5])) for n in lens]
    run(lens, qlens, 2, 1, 64, fp8=fp8, extra_rows=2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(alibi=True, sink=True), dict(window=3, nan_draft=True),
                                dict(kind="random")], ids=["alibi", "window", "random"])
def test_many_short_requests_per_cta(d, kw, fp8):
    """A CTA that takes request after request, every key tile of them a general
    one, its V rows repaired ahead of the softmax."""
    rng = random.Random(10)
    lens = [rng.randint(1, 140) for _ in range(60)]
    run(lens, [min(n, rng.randint(1, 6)) for n in lens], 6, 2, d, fp8=fp8, partition=2048, **kw)


@pytest.mark.parametrize("fp8", [False, True])
def test_more_kv_heads_than_sms(fp8):
    run([40, 300], [3, 5], 160, 160, 64, fp8=fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_as_many_rows_as_a_call_takes(fp8):
    run([600], [256], 16, 1, 128, fp8=fp8)


def test_requests_that_share_their_pages():
    g = torch.Generator().manual_seed(12)
    pools = R.Pools(40, 16, 2, 128, "NHD", True, g)
    table, _ = R.paged([600], 16, 40, g)
    q = torch.randn(1, 8, 128, generator=g).to(BF16).to(DEV).expand(3, 8, 128).contiguous()
    out = pkv.paged_decode_fp8(q, *pools.device(DEV), table.expand(3, -1).contiguous().to(DEV),
                               torch.full((3,), 600, dtype=I32, device=DEV), 600)
    assert R.same_bits(out[0], out[1]) and R.same_bits(out[0], out[2])
    assert bool(torch.isfinite(out).all())
