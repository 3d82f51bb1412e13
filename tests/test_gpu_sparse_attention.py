"""paged_sparse_attention on the GPU within derived bounds of the 64-bit attention
over the keys of each row's pages."""
import random

import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R
from tests import _sparse as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, I32 = torch.bfloat16, torch.int32


# Rows of no request: enough of them that the queries before them are taken in tiles
# (few rows are taken one at a time).
MANY = 2000


def lists(rows, hkv, top_k, bs, rng, kind):
    """Pages of every row and kv head: strictly ascending, then -1."""
    out = torch.full((len(rows), hkv, top_k), -1, dtype=I32)
    for t, (_, n) in enumerate(rows):
        pages = S.pages_of(n, bs)
        for g in range(hkv):
            m = min(pages, top_k)
            if kind == "random":                 # any number of them, none among those
                m = rng.randint(0, m)
            chosen = set(rng.sample(range(pages), m))
            if kind == "last" and m:             # the page that may end inside
                chosen = set(sorted(chosen)[:m - 1]) | {pages - 1}
            chosen = sorted(chosen)
            out[t, g, :len(chosen)] = torch.tensor(chosen, dtype=I32)
    return out


def run(lens, queries, hq, hkv, d, bs=16, layout="NHD", fp8=False, top_k=6, kind="last",
        sink=False, seed=0, spread=1.0, scale=None, extra=0, chunk=None, edit=None, qsize=1.0):
    g = torch.Generator().manual_seed(seed + d + sum(lens))
    rng = random.Random(seed + sum(queries))
    nb = sum(S.pages_of(n, bs) for n in lens) + 2
    pools = R.Pools(nb, bs, hkv, d, layout, fp8, g, spread=spread)
    table, slots = R.paged(lens, bs, nb, g)
    owned = set(torch.cat(slots).tolist())
    pools.poison([s for s in range(nb * bs) if s not in owned])
    if edit:
        edit(pools, slots)
    rows = S.rows_of(queries, lens)
    pages = lists(rows, hkv, top_k, bs, rng, kind)
    total = len(rows) + extra
    q = (qsize * torch.randn(total, hq, d, generator=g)).to(BF16)
    snk = torch.randn(hq, generator=g) if sink else None
    cu = torch.tensor([0] + torch.tensor(queries).cumsum(0).tolist(), dtype=I32, device=DEV)
    chunk = any(m != 1 for m in queries) if chunk is None else chunk
    kc, vc, ks, vs = pools.device(DEV)
    out = torch.full((total, hq, d), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((total, hq), 7.0, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    sc = d ** -0.5 if scale is None else scale
    dpages = torch.cat([pages, torch.zeros(extra, hkv, top_k, dtype=I32)]).to(DEV)
    got = pkv.paged_sparse_attention(
        q.to(DEV), kc, vc, table.to(DEV), torch.tensor(lens, dtype=I32, device=DEV), dpages,
        cu_seq_lens_q=cu if chunk else None, k_scale=ks, v_scale=vs,
        sink=None if snk is None else snk.to(DEV), sm_scale=sc, out=out, lse=lse, dev_error=err,
        layout=layout)
    assert got is out
    assert pkv.get_device_error(err) == 0
    ref, rl, absv, smax, floor = S.attend_lists(q, pools, slots, rows, pages, bs, sc, snk)
    m = len(rows)
    # bf16 weights: half a step is 2^-8 (f16 ones over 8-bit pools: 2^-11)
    bound = R.out_bound(ref, absv, smax, d, 2.0 ** -11, floor) if fp8 else \
        R.out_bound(ref, absv, smax, d, 2.0 ** -8)
    if not edit:
        R.assert_within(out[:m], ref, bound, "out")
        R.assert_within(lse[:m], rl, R.lse_bound(rl, smax, d), "lse")
    assert bool((out[m:] == 7.0).all()) and bool((lse[m:] == 7.0).all())
    return out[:m].cpu(), lse[:m].cpu(), ref, rl, bound, R.lse_bound(rl, smax, d)


KINDS = [("NHD", False), ("HND", False), ("NHD", True), ("HND", True)]


@pytest.mark.parametrize("layout,fp8", KINDS)
@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 2, 64, 32), (8, 8, 128, 16), (32, 8, 128, 32),
                                         (3, 1, 80, 16), (10, 2, 96, 16), (16, 1, 112, 32),
                                         (12, 1, 256, 16), (64, 4, 64, 16), (6, 2, 256, 32)])
def test_one_query_each(layout, fp8, hq, hkv, d, bs):
    lens = [1, bs - 1, bs, bs + 1, 9 * bs + 5, 40 * bs, 3 * bs + 7]
    run(lens, [1] * len(lens), hq, hkv, d, bs, layout, fp8, top_k=7, sink=True)
    run(lens, [1] * len(lens), hq, hkv, d, bs, layout, fp8, top_k=5, kind="random", seed=1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("top_k", [1, 2, 3, 4, 8, 17, 64, 129, 300])
def test_list_lengths(fp8, top_k):
    """One CTA and clusters of two to eight, lists that fill and leave room."""
    run([16 * 250 + 9, 16 * top_k, 40], [1] * 3, 8, 2, 64, fp8=fp8, top_k=top_k)
    run([16 * 250 + 9, 16 * top_k + 1, 1], [1] * 3, 4, 1, 128, fp8=fp8, top_k=top_k, layout="HND")


@pytest.mark.parametrize("fp8", [False, True])
def test_many_rows(fp8):
    """More rows than run at once: no clusters."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 300, (130,), generator=g).tolist()
    run(lens, [1] * 130, 8, 4, 64, fp8=fp8, top_k=20, sink=True)


@pytest.mark.parametrize("extra", [4, MANY])
@pytest.mark.parametrize("layout,fp8", KINDS)
@pytest.mark.parametrize("queries,lens", [([3, 1, 8, 5], [3, 300, 500, 9]), ([33], [500]),
                                          ([0, 2, 0, 17, 1], [30, 90, 0, 17, 200]),
                                          ([6, 4], [3, 100]), ([30, 1, 8, 13], [30, 300, 500, 50]),
                                          ([0, 20, 0, 47, 1], [30, 90, 0, 47, 200])])
def test_chunks(layout, fp8, queries, lens, extra):
    """Rows of a chunk, each up to its own position; rows of no request stay."""
    run(lens, queries, 8, 2, 64, 16, layout, fp8, top_k=9, sink=True, extra=extra, chunk=True)


@pytest.mark.parametrize("kind", ["last", "random"])
@pytest.mark.parametrize("hq,hkv,d,bs", [(2, 2, 64, 16), (4, 2, 80, 32), (6, 2, 128, 16),
                                         (5, 1, 96, 16), (8, 1, 128, 32), (11, 1, 112, 16),
                                         (32, 2, 64, 32), (6, 2, 256, 16)])
def test_tiles_of_queries(hq, hkv, d, bs, kind):
    """Every width of a group; tiles that hold the ends of requests."""
    run([17 * bs + 5, 3, 60 * bs, 11 * bs + 1], [21, 3, 37, 9], hq, hkv, d, bs, top_k=8, kind=kind,
        sink=True, extra=MANY, layout="HND")


@pytest.mark.parametrize("most,hq", [(5, 4), (12, 8)])
@pytest.mark.parametrize("batch", [256, 257])
def test_chunks_of_many_requests(batch, most, hq):
    """Tiles request by request, and beyond that count every so many rows."""
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 60, (batch,), generator=g).tolist()
    queries = [min(n, most) if i % 9 else 0 for i, n in enumerate(lens)]
    queries[7] = lens[7] = 200
    run(lens, queries, hq, 2, 64, top_k=3, chunk=True, extra=MANY if most > 5 else 3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("decodes,chunks", [(40, 1), (120, 3), (262, 4)])
def test_decodes_beside_chunks(decodes, chunks, fp8):
    """Requests of one query beside chunks, in tiles request by request, in tiles of
    whatever rows come, and row by row."""
    g = torch.Generator().manual_seed(decodes)
    lens = torch.randint(1, 200, (decodes,), generator=g).tolist() + [230 + 40 * i for i in range(chunks)]
    queries = [1] * decodes + [200 + 13 * i for i in range(chunks)]
    run(lens, queries, 8, 2, 64, fp8=fp8, top_k=5, sink=True, extra=MANY if decodes > 250 else 0)


@pytest.mark.parametrize("n,hq", [(8, 2), (MANY, 4)])
def test_offsets_that_are_none(n, hq):
    """Offsets that decrease or leave the rows: nothing outside is read or written."""
    pools, table, slots, _ = small()
    kc, vc, _, _ = pools.device(DEV)
    q = torch.randn(n, hq, 64, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    pages = torch.arange(4, dtype=I32, device=DEV).expand(n, 1, 4).contiguous()
    two = torch.cat([table, table]).to(DEV)
    lens = torch.tensor([100, 100], dtype=I32, device=DEV)
    for cu in ([2, 1, n], [0, n + 11, 3], [3, 3, 3], [-5, 0, 9000], [n, 2, 0], [0, n // 2, n]):
        out = torch.full((n, hq, 64), 7.0, dtype=BF16, device=DEV)
        pkv.paged_sparse_attention(q, kc, vc, two, lens, pages, out=out,
                                   cu_seq_lens_q=torch.tensor(cu, dtype=I32, device=DEV))
        assert bool(torch.isfinite(out.float()).all())
    assert not bool((out == 7.0).any())


def guarded(n, *shape, dtype=BF16):
    """A tensor of 3 + n + 3 rows of sevens, and the n rows in its middle."""
    whole = torch.full((n + 6, *shape), 7.0, dtype=dtype, device=DEV)
    return whole, whole[3:3 + n]


def untouched(whole):
    return bool((whole[:3] == 7.0).all()) and bool((whole[-3:] == 7.0).all())


def by_offsets(cu, lens, n):
    """(request, keys up to and with its own) of the rows that offsets which do not decrease
    leave a request, by row: the rows that exist, the last of them at the last position."""
    rows = {}
    for r, (a, b) in enumerate(zip(cu, cu[1:])):
        b = min(b, n)
        for t in range(max(a, 0), b):
            rows[t] = (r, max(0, lens[r] - (b - t) + 1))
    return rows


@pytest.mark.parametrize("n,hq,fp8", [(4, 2, False), (4, 2, True), (MANY, 4, False)])
@pytest.mark.parametrize("cu", ["0 n+2", "0 n-1 n+7", "0 2 n+9 n+9", "-3 2 n", "-9 -4 n", "2 n+1 n+1",
                                "0 n n+5 n+9", "n n+1 n+2", "0 2 2**31-1 2**31-1"])
def test_offsets_outside_the_rows(cu, n, hq, fp8):
    """They are flagged; a request has the rows that exist, its last one at its last
    position, and nothing else is written."""
    cu = [eval(x, {"n": n}) for x in cu.split()]
    g = torch.Generator().manual_seed(6)
    lens = [100, 77, 130][:len(cu) - 1]
    pools = R.Pools(24, 16, 1, 64, "NHD", fp8, g)
    table, slots = R.paged(lens, 16, 24, g)
    kc, vc, ks, vs = pools.device(DEV)
    q = torch.randn(n, hq, 64, generator=g).to(BF16)
    rows = by_offsets(cu, lens, n)
    at = sorted(rows)
    held = lists([rows[t] for t in at], 1, 4, 16, random.Random(6), "last")
    pages = torch.full((n, 1, 4), -1, dtype=I32)
    pages[at] = held
    (whole, out), (whole_lse, lse) = guarded(n, hq, 64), guarded(n, hq, dtype=torch.float32)
    err = torch.zeros(1, dtype=I32, device=DEV)
    pkv.paged_sparse_attention(q.to(DEV), kc, vc, table.to(DEV),
                               torch.tensor(lens, dtype=I32, device=DEV), pages.to(DEV), k_scale=ks,
                               v_scale=vs, out=out, lse=lse, dev_error=err,
                               cu_seq_lens_q=torch.tensor(cu, dtype=I32, device=DEV))
    assert pkv.get_device_error(err) == pkv.DEVERR_SEQLEN
    assert untouched(whole) and untouched(whole_lse)
    none = [t for t in range(n) if t not in rows]
    assert bool((out[none] == 7.0).all()) and bool((lse[none] == 7.0).all())
    if at:
        ref, rl, absv, smax, floor = S.attend_lists(q[at], pools, slots, [rows[t] for t in at], held,
                                                    16, 0.125, None)
        bound = R.out_bound(ref, absv, smax, 64, 2.0 ** -11, floor) if fp8 else \
            R.out_bound(ref, absv, smax, 64, 2.0 ** -8)
        R.assert_within(out[at], ref, bound, "out")
        R.assert_within(lse[at], rl, R.lse_bound(rl, smax, 64), "lse")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 8, MANY])
def test_offsets_that_decrease(n, fp8):
    """Flagged wherever they stand, also in requests that no row belongs to; nothing outside
    the rows is written."""
    pools, table, slots, _ = small(fp8)
    kc, vc, ks, vs = pools.device(DEV)
    q = torch.randn(n, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    pages = torch.full((n, 1, 4), -1, dtype=I32, device=DEV)
    for batch in (3, 300, 1000):
        for at in {1, batch // 2, batch - 1, batch}:
            cu = [0] + [n] * batch
            cu[at] = n - 1 if at > 1 else n + 1   # (in the second place: above the third)
            err = torch.zeros(1, dtype=I32, device=DEV)
            whole, out = guarded(n, 4, 64)
            pkv.paged_sparse_attention(
                q, kc, vc, table.expand(batch, -1).contiguous().to(DEV),
                torch.full((batch,), 100, dtype=I32, device=DEV), pages, k_scale=ks, v_scale=vs,
                out=out, dev_error=err, cu_seq_lens_q=torch.tensor(cu, dtype=I32, device=DEV))
            assert pkv.get_device_error(err) == pkv.DEVERR_SEQLEN, (batch, at)
            assert untouched(whole)


@pytest.mark.parametrize("extra", [0, MANY])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_chunk_scales(scale, extra):
    run([300, 33], [9, 7], 4, 2, 64, top_k=9, scale=scale, sink=True, extra=extra)


@pytest.mark.parametrize("extra", [0, MANY])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_a_scale_of_zero_times_a_query_that_is_not_finite(value, extra):
    """0 times it is NaN, in tiles as row by row; other heads and rows are not touched."""
    pools, table, slots, _ = small()
    kc, vc, _, _ = pools.device(DEV)
    q = torch.randn(9 + extra, 4, 64, generator=torch.Generator().manual_seed(8)).to(BF16)
    q[2, 1, 40], q[7, 3, 0] = float(value), float(value)
    rows = S.rows_of([9], [100])
    pages = lists(rows, 1, 4, 16, random.Random(8), "last")
    padded = torch.cat([pages, torch.zeros(extra, 1, 4, dtype=I32)]).to(DEV)
    lse = torch.zeros(9 + extra, 4, device=DEV)
    cu, lens = (torch.tensor(x, dtype=I32, device=DEV) for x in ([0, 9], [100]))
    out = pkv.paged_sparse_attention(q.to(DEV), kc, vc, table.to(DEV), lens, padded, cu_seq_lens_q=cu,
                                     sm_scale=0.0, lse=lse)[:9].cpu()
    bad = torch.zeros(9, 4, dtype=torch.bool)
    bad[2, 1] = bad[7, 3] = True
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(out).any(-1), bad)
    assert torch.equal(torch.isnan(lse[:9]).cpu(), bad)
    ref, rl, absv, smax, _ = S.attend_lists(q[:9].nan_to_num(0.0, 0.0, 0.0), pools, slots, rows, pages,
                                            16, 0.0, None)
    fine = ~bad
    R.assert_within(out[fine], ref[fine], R.out_bound(ref, absv, smax, 64, 2.0 ** -8)[fine], "out")
    R.assert_within(lse[:9].cpu()[fine], rl[fine], R.lse_bound(rl, smax, 64)[fine], "lse")


@pytest.mark.parametrize("extra", [0, MANY])
def test_wide_lists_and_tables(extra):
    """Unions of hundreds of pages; tables much wider than their requests."""
    run([16 * 700 + 3], [9], 4, 1, 64, top_k=150, extra=extra)
    g = torch.Generator().manual_seed(9)
    pools = R.Pools(40, 16, 2, 64, "NHD", False, g)
    narrow, slots = R.paged([300, 200], 16, 40, g)
    kc, vc, _, _ = pools.device(DEV)
    q = torch.randn(10 + extra, 4, 64, generator=g).to(BF16).to(DEV)
    lens = torch.tensor([300, 200], dtype=I32, device=DEV)
    cu = torch.tensor([0, 6, 10], dtype=I32, device=DEV)
    rows = S.rows_of([6, 4], [300, 200])
    pages = lists(rows, 2, 5, 16, random.Random(9), "last")
    padded = torch.cat([pages, torch.zeros(extra, 2, 5, dtype=I32)]).to(DEV)
    wide = torch.full((2, 700000), -1, dtype=I32)
    wide[:, :narrow.shape[1]] = narrow
    outs = [pkv.paged_sparse_attention(q, kc, vc, t.to(DEV), lens, padded, cu_seq_lens_q=cu)
            for t in (narrow, wide)]
    ref, _, absv, smax, _ = S.attend_lists(q[:10].cpu(), pools, slots, rows, pages, 16, 0.125, None)
    for o in outs:
        R.assert_within(o[:10], ref, R.out_bound(ref, absv, smax, 64, 2.0 ** -8), "out")


@pytest.mark.parametrize("top_k", [2, 40])
@pytest.mark.parametrize("kind", ["last", "random"])
@pytest.mark.parametrize("hq,hkv,bs,n", [(2, 2, 16, 1700), (1, 1, 32, 1500), (4, 1, 16, 4600)])
def test_chunks_of_long_contexts(hq, hkv, bs, n, kind, top_k):
    """More pages than a tile's bitmaps hold at a time, windows without a page."""
    run([bs * n + 3, 700], [33, 35], hq, hkv, 64, bs, kind=kind, top_k=top_k, sink=True, extra=MANY)


@pytest.mark.parametrize("extra", [0, MANY])
@pytest.mark.parametrize("pool", [0, 1])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_chunk_with_a_key_that_is_not_finite(pool, value, extra):
    """It reaches the queries that keep it, and not those that share its page's loads:
    a page of some, a page of all of which some see only a part, a page of all."""
    def edit(pools, slots):
        for at in (slots[0][37], slots[0][295], slots[1][3]):
            pools.rows[pool][at // 16, 0, at % 16, 5] = float(value)

    out, lse, ref, rl, bound, lb = run([300, 40], [16, 8], 4, 1, 64, top_k=9, edit=edit, seed=7,
                                       extra=extra)
    fin = torch.isfinite(ref)
    assert 0 < int(fin.sum()) < fin.numel()
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    bad = ~fin & ~torch.isnan(ref)
    assert torch.equal(out.double()[bad], ref[bad])
    off = torch.where(fin, (out.double() - ref).abs() - bound, torch.zeros_like(ref))
    assert float(off.max()) <= 0
    # (a row with a score of +inf: its sum is infinite, and taken relative to its largest
    # score it is inf - inf, so that such an lse is either)
    fin = torch.isfinite(rl)
    assert torch.equal(torch.isfinite(lse), fin)
    off = torch.where(fin, (lse.double() - rl).abs() - lb, torch.zeros_like(rl))
    assert float(off.max()) <= 0


@pytest.mark.parametrize("extra", [0, MANY])
def test_chunk_lists_that_end_early(extra):
    """Lists of a chunk with errors and entries behind their end; pages out of the pool."""
    pools, table, slots, _ = small()
    g = torch.Generator().manual_seed(11)
    q = torch.randn(6 + extra, 2, 64, generator=g).to(BF16)
    given = [[1, 3, 5, -1], [1, -1, 3, 5], [1, 3, 3, 5], [3, 1, 4, 5], [1, 3, 7, 8], [0, 2, 4, 6]]
    held = [[1, 3, 5, -1], [1, -1, -1, -1], [1, 3, -1, -1], [3, -1, -1, -1], [1, 3, -1, -1],
            [0, 2, -1, -1]]
    padded = torch.zeros(6 + extra, 1, 4, dtype=I32)
    padded[:6, 0] = torch.tensor(given)
    kc, vc, _, _ = pools.device(DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    cu, lens = (torch.tensor(x, dtype=I32, device=DEV) for x in ([0, 6], [100]))
    for broken, bits in ((False, pkv.DEVERR_BLOCK_ID), (True, pkv.DEVERR_BLOCK_ID)):
        t = table.clone()
        want = [list(x) for x in held]
        if broken:
            t[0, 4] = -1
            want[-1] = [0, 2, 6, -1]
        else:
            want[-1] = [0, 2, 4, 6]
        out = pkv.paged_sparse_attention(q.to(DEV), kc, vc, t.to(DEV), lens,
                                         padded.to(DEV), cu_seq_lens_q=cu, dev_error=err)
        assert pkv.get_device_error(err, clear=True) == bits
        pages = torch.tensor(want, dtype=I32).view(6, 1, 4)
        ref, _, absv, smax, _ = S.attend_lists(q[:6], pools, slots, S.rows_of([6], [100]), pages, 16,
                                               0.125, None)
        R.assert_within(out[:6], ref, R.out_bound(ref, absv, smax, 64, 2.0 ** -8), "out")


@pytest.mark.parametrize("fp8", [False, True])
def test_empty_lists(fp8):
    """Rows without keys: zeros, and the sink (or -inf) as lse."""
    for sink in (False, True):
        out, lse, *_ = run([50, 0, 70], [1] * 3, 4, 2, 64, fp8=fp8, kind="random", top_k=1,
                           sink=sink, seed=4)
        assert bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_growing_scores(fp8):
    """Scores of hundreds, either sign, a scale of zero."""
    run([900, 333], [1, 1], 8, 2, 128, fp8=fp8, top_k=50, qsize=40.0)
    run([900, 333], [1, 1], 8, 2, 128, fp8=fp8, top_k=50, scale=-0.3)
    run([900, 333], [1, 1], 8, 2, 128, fp8=fp8, top_k=50, scale=0.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_values_of_very_different_sizes(fp8):
    run([2000, 500], [1, 1], 8, 2, 64, fp8=fp8, top_k=100, spread=6.0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("pool", [0, 1])
def test_a_key_that_is_not_finite(fp8, pool):
    """A NaN key or value reaches the rows whose lists hold its page, and no other."""
    def edit(pools, slots):
        at = slots[0][37]                     # page 2 of request 0, both kv heads
        if fp8:
            pools.byte[pool][at // 16, :, at % 16] = 255
        else:
            pools.rows[pool][at // 16, :, at % 16] = float("nan")

    out, lse, ref, rl, bound, lb = run([640, 200], [1, 1], 4, 2, 64, fp8=fp8, top_k=40, edit=edit)
    assert bool(torch.isnan(out[0]).all())
    assert bool(torch.isnan(lse[0]).all()) if pool == 0 else bool(torch.isfinite(lse[0]).all())
    R.assert_within(out[1:], ref[1:], bound[1:], "out")
    R.assert_within(lse[1:], rl[1:], lb[1:], "lse")
    out, lse, ref, rl, bound, lb = run([640], [1], 4, 2, 64, fp8=fp8, top_k=2, edit=edit, seed=3)
    assert bool(torch.isfinite(out.float()).all())
    R.assert_within(out, ref, bound, "out")


def small(fp8=False, top_k=4):
    g = torch.Generator().manual_seed(2)
    pools = R.Pools(12, 16, 1, 64, "NHD", fp8, g)
    table, slots = R.paged([100], 16, 12, g)
    q = torch.randn(1, 2, 64, generator=g).to(BF16)
    return pools, table, slots, q


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("given,held,bits", [
    ([1, 3, 6, -1], [1, 3, 6, -1], 0),
    ([1, -1, 3, 6], [1, -1, -1, -1], 0),
    ([-1, 1, 3, 6], [-1] * 4, 0),
    ([-2 ** 31, 5, 5, 5], [-1] * 4, 0),
    ([1, 3, 3, 6], [1, 3, -1, -1], pkv.DEVERR_BLOCK_ID),
    ([3, 1, 4, 6], [3, -1, -1, -1], pkv.DEVERR_BLOCK_ID),
    ([1, 3, 7, 8], [1, 3, -1, -1], pkv.DEVERR_BLOCK_ID),
    ([2 ** 31 - 1, 1, 2, 3], [-1] * 4, pkv.DEVERR_BLOCK_ID),
])
def test_lists_that_end_early(fp8, given, held, bits):
    pools, table, slots, q = small(fp8)
    kc, vc, ks, vs = pools.device(DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    out = pkv.paged_sparse_attention(
        q.to(DEV), kc, vc, table.to(DEV), torch.tensor([100], dtype=I32, device=DEV),
        torch.tensor(given, dtype=I32, device=DEV).view(1, 1, 4), k_scale=ks, v_scale=vs,
        dev_error=err)
    assert pkv.get_device_error(err) == bits
    pages = torch.tensor(held, dtype=I32).view(1, 1, 4)
    ref, _, absv, smax, floor = S.attend_lists(q, pools, slots, [(0, 100)], pages, 16, 0.125, None)
    bound = R.out_bound(ref, absv, smax, 64, 2.0 ** -11, floor) if fp8 else \
        R.out_bound(ref, absv, smax, 64, 2.0 ** -8)
    R.assert_within(out, ref, bound, "out")


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_out_of_the_pool(fp8):
    """They are left out, and flagged."""
    pools, table, slots, q = small(fp8)
    kc, vc, ks, vs = pools.device(DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    broken = table.clone()
    broken[0, 3], broken[0, 5] = -1, 12
    pages = torch.arange(7, dtype=I32).view(1, 1, 7)
    args = (torch.tensor([100], dtype=I32, device=DEV), pages.to(DEV))
    out = pkv.paged_sparse_attention(q.to(DEV), kc, vc, broken.to(DEV), *args, k_scale=ks,
                                     v_scale=vs, dev_error=err)
    assert pkv.get_device_error(err) == pkv.DEVERR_BLOCK_ID
    held = torch.tensor([0, 1, 2, 4, 6, -1, -1], dtype=I32).view(1, 1, 7)
    ref, _, absv, smax, floor = S.attend_lists(q, pools, slots, [(0, 100)], held, 16, 0.125, None)
    bound = R.out_bound(ref, absv, smax, 64, 2.0 ** -11, floor) if fp8 else \
        R.out_bound(ref, absv, smax, 64, 2.0 ** -8)
    R.assert_within(out, ref, bound, "out")


@pytest.mark.parametrize("fp8", [False, True])
def test_the_whole_context_is_the_dense_decode(fp8):
    """Lists of all pages: the dense calls' answer within both bounds."""
    g = torch.Generator().manual_seed(3)
    lens = [700, 33, 1025]
    pools = R.Pools(130, 16, 2, 128, "HND", fp8, g)
    table, slots = R.paged(lens, 16, 130, g)
    kc, vc, ks, vs = pools.device(DEV)
    q = torch.randn(3, 8, 128, generator=g).to(BF16)
    dl = torch.tensor(lens, dtype=I32, device=DEV)
    pages = torch.arange(66, dtype=I32).expand(3, 2, 66).clone()
    for r, n in enumerate(lens):
        pages[r, :, S.pages_of(n, 16):] = -1
    a = pkv.paged_sparse_attention(q.to(DEV), kc, vc, table.to(DEV), dl, pages.to(DEV), k_scale=ks,
                                   v_scale=vs, layout="HND")
    if fp8:
        b = pkv.paged_decode_fp8(q.to(DEV), kc, vc, ks, vs, table.to(DEV), dl, 1025, layout="HND")
    else:
        b = pkv.paged_decode(q.to(DEV), kc, vc, table.to(DEV), dl, 1025, layout="HND")
    ref, _, absv, smax, floor = S.attend_lists(q, pools, slots, [(r, n) for r, n in enumerate(lens)],
                                               pages, 16, 128 ** -0.5, None)
    bound = R.out_bound(ref, absv, smax, 128, 2.0 ** -11, floor) if fp8 else \
        R.out_bound(ref, absv, smax, 128, 2.0 ** -8)
    R.assert_within(a, ref, bound, "sparse")
    R.assert_within(b, ref, bound, "dense")


def test_large_pool_offsets():
    """Pages beyond 2^31 elements of the pool."""
    nb, hkv, d = 140000, 8, 128               # 2.29e9 elements a pool
    kc = torch.zeros(nb, 16, hkv, d, dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    g = torch.Generator().manual_seed(4)
    pools = R.Pools(4, 16, hkv, d, "NHD", False, g)
    sk, sv, _, _ = pools.device(DEV)
    ids = torch.tensor([nb - 1, 131072, 5, nb - 2])
    kc[ids.to(DEV)], vc[ids.to(DEV)] = sk, sv
    q = torch.randn(1, 16, d, generator=g).to(BF16)
    pages = torch.tensor([0, 1, 3], dtype=I32).expand(1, hkv, 3).contiguous()
    out = pkv.paged_sparse_attention(q.to(DEV), kc, vc, ids.to(I32)[None].to(DEV),
                                     torch.tensor([60], dtype=I32, device=DEV), pages.to(DEV))
    ref, _, absv, smax, _ = S.attend_lists(q, pools, [torch.arange(60)], [(0, 60)], pages, 16,
                                           d ** -0.5, None)
    R.assert_within(out, ref, R.out_bound(ref, absv, smax, d, 2.0 ** -8), "out")


def test_in_a_graph_and_on_two_streams():
    g = torch.Generator().manual_seed(5)
    pools = R.Pools(60, 16, 2, 64, "NHD", False, g)
    table, slots = R.paged([500, 300], 16, 60, g)
    kc, vc, _, _ = pools.device(DEV)
    q = torch.randn(2, 8, 64, generator=g).to(BF16).to(DEV)
    lens = torch.tensor([500, 300], dtype=I32, device=DEV)
    pages = lists([(0, 500), (1, 300)], 2, 12, 16, random.Random(5), "last").to(DEV)
    table = table.to(DEV)
    first = pkv.paged_sparse_attention(q, kc, vc, table, lens, pages)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pkv.paged_sparse_attention(q, kc, vc, table, lens, pages)
    graph.replay()
    assert torch.equal(got, first)
    torch.cuda.synchronize()
    outs = [pkv.paged_sparse_attention(q, kc, vc, table, lens, pages, stream=s)
            for s in [torch.cuda.Stream() for _ in range(2)] for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
