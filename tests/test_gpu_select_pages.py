"""select_pages on the GPU: the same lists as the definition's, entry for entry."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _sparse as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, I32, U8, I8 = torch.bfloat16, torch.int32, torch.uint8, torch.int8


def make(lens, queries, hq, hkv, d, bs, seed=0, spread=1):
    g = torch.Generator().manual_seed(seed + d + sum(lens))
    pages = [S.pages_of(n, bs) for n in lens]
    nb = sum(pages) + 3
    perm = torch.randperm(nb, generator=g)
    table = torch.full((len(lens), max(pages + [1]) + 1), -1, dtype=I32)
    at = 0
    for r, p in enumerate(pages):
        table[r, :p] = perm[at:at + p].to(I32)
        at += p
    mid = torch.randn(nb, hkv, d, generator=g) * 24
    half = 20 + 8 * torch.randn(nb, hkv, d, generator=g).abs()
    codes = torch.stack([(mid - half).floor(), (mid + half).ceil()], 2).clamp(-127, 127).to(I8)
    byte = torch.randint(122 - spread, 122 + spread, (nb, hkv), generator=g).to(U8)
    q = torch.randn(sum(queries), hq, d, generator=g) * \
        torch.exp2(torch.randn(sum(queries), hq, 1, generator=g))
    return dict(q=q.to(BF16), codes=codes, byte=byte, table=table, lens=list(lens),
                queries=list(queries), bs=bs)


def want(c, top_k, first, recent):
    out = []
    for t, (r, n) in enumerate(S.rows_of(c["queries"], c["lens"])):
        ids = c["table"][r, :S.pages_of(n, c["bs"])].long()
        sc = S.scores(c["q"][t], c["codes"][ids], c["byte"][ids])
        out.append(S.choose(sc, top_k, first, recent))
    return torch.stack(out)


def check(c, top_k, first=1, recent=1, chunk=None, extra=0, max_seqlen=None):
    queries, lens = c["queries"], c["lens"]
    chunk = any(m != 1 for m in queries) if chunk is None else chunk
    cu = torch.tensor([0] + torch.tensor(queries).cumsum(0).tolist(), dtype=I32, device=DEV)
    q = torch.cat([c["q"], torch.zeros(extra, *c["q"].shape[1:], dtype=BF16)])
    hkv = c["codes"].shape[1]
    err = torch.zeros(1, dtype=I32, device=DEV)
    pages = torch.full((q.shape[0], hkv, top_k), -9, dtype=I32, device=DEV)
    got = pkv.select_pages(q.to(DEV), c["codes"].to(DEV), c["byte"].to(DEV), c["table"].to(DEV),
                           torch.tensor(lens, dtype=I32, device=DEV), max_seqlen or max(lens), top_k,
                           c["bs"], num_first=first, num_recent=recent,
                           cu_seq_lens_q=cu if chunk else None, pages=pages, dev_error=err)
    assert got is pages
    assert pkv.get_device_error(err) == 0
    w = want(c, top_k, first, recent)
    assert torch.equal(got[:w.shape[0]].cpu(), w)
    assert bool((got[w.shape[0]:] == -9).all())


@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 2, 64, 32), (8, 8, 128, 16), (32, 8, 128, 16),
                                         (3, 1, 80, 16), (10, 2, 96, 32), (16, 1, 112, 16),
                                         (12, 1, 256, 16), (64, 4, 64, 16), (6, 2, 256, 32)])
def test_one_query_each(hq, hkv, d, bs):
    lens = [1, bs, bs + 1, 40 * bs + 3, 97 * bs, 300 * bs - 1, 5 * bs]
    c = make(lens, [1] * len(lens), hq, hkv, d, bs)
    check(c, 8)
    check(c, 2)
    check(c, 33, first=3, recent=4)


@pytest.mark.parametrize("top_k", [1, 2, 7, 64, 100, 256, 1000])
def test_sizes_of_lists(top_k):
    lens = [16 * 1000 + 5, 999, 16 * top_k, 16 * top_k + 1, 16 * top_k + 17]
    c = make(lens, [1] * 5, 8, 2, 128, 16)
    check(c, top_k, first=0)


# Rows of no request: enough of them that the queries before them are taken in tiles
# (few rows are taken one at a time).
MANY = 500


@pytest.mark.parametrize("extra", [5, MANY])
@pytest.mark.parametrize("queries,lens", [([3, 1, 8, 5], [3, 700, 1200, 9]), ([40], [2500]),
                                          ([0, 2, 0, 17, 1], [30, 900, 0, 17, 2000])])
def test_chunks(queries, lens, extra):
    """Rows of a chunk, each up to its own position; rows of no request stay."""
    c = make(lens, queries, 8, 2, 64, 16)
    check(c, 12, recent=2, chunk=True, extra=extra)


@pytest.mark.parametrize("hq,hkv,d,bs", [(2, 2, 64, 16), (4, 2, 80, 32), (6, 2, 128, 16),
                                         (8, 2, 256, 16), (5, 1, 96, 32), (8, 1, 128, 16),
                                         (11, 1, 112, 16), (32, 2, 128, 32), (16, 1, 256, 16)])
def test_tiles_of_queries(hq, hkv, d, bs):
    """Every width of a group; tiles that hold the ends of requests, and rows of which
    some take all their pages."""
    c = make([37 * bs + 5, 3, 200 * bs, 21 * bs + 1], [11, 3, 19, 9], hq, hkv, d, bs)
    check(c, 20, recent=2, extra=MANY)
    check(c, 1, first=0, extra=MANY)
    check(c, 20, recent=2, extra=2)


@pytest.mark.parametrize("batch", [256, 257])
def test_chunks_of_many_requests(batch):
    """Tiles request by request, and beyond that count every so many rows."""
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 400, (batch,), generator=g).tolist()
    queries = [min(n, 5) if i % 9 else 0 for i, n in enumerate(lens)]
    queries[7] = lens[7] = 300
    check(make(lens, queries, 4, 2, 64, 16), 6, chunk=True, extra=3)


@pytest.mark.parametrize("decodes,chunks", [(40, 1), (120, 3), (262, 4)])
def test_decodes_beside_chunks(decodes, chunks):
    """Requests of one query beside chunks, in tiles request by request, in tiles of
    whatever rows come, and one at a time."""
    g = torch.Generator().manual_seed(decodes)
    lens = torch.randint(1, 900, (decodes,), generator=g).tolist() + [930 + 40 * i for i in range(chunks)]
    check(make(lens, [1] * decodes + [100 + 13 * i for i in range(chunks)], 8, 2, 64, 16), 9, recent=2,
          extra=MANY if decodes > 250 else 0)


@pytest.mark.parametrize("extra", [0, MANY])
@pytest.mark.parametrize("hq", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("n", [3000, 70000, 300000])
def test_tiles_over_long_contexts(n, hq, extra):
    """Clusters share a tile's pages; one query at a time where the scores do not fit."""
    check(make([n], [5], hq, 1, 64, 16, spread=3), 64, recent=3, extra=extra)
    check(make([n], [4], hq, 1, 64, 16, spread=3), 200, extra=extra)


def test_tiles_over_the_longest_contexts():
    check(make([16 * 65536 + 3, 40], [5, 11], 4, 1, 64, 16, spread=3), 64, recent=3, extra=MANY)


@pytest.mark.parametrize("extra", [0, MANY])
@pytest.mark.parametrize("queries,lens", [([6, 4], [3, 100]), ([5], [0])])
def test_rows_before_the_first_position(queries, lens, extra):
    """More queries than keys: rows without a key have empty lists."""
    check(make(lens, queries, 4, 2, 64, 16), 3, chunk=True, extra=extra)


@pytest.mark.parametrize("n", [65536 * 16 + 9, 300000])
def test_long(n):
    check(make([n, 50], [1, 1], 8, 2, 64, 16, spread=3), 256, first=2, recent=8)


def test_many_requests_and_a_loose_maximum():
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 3000, (70,), generator=g).tolist()
    c = make(lens, [1] * 70, 4, 1, 64, 16)
    check(c, 16, max_seqlen=100000)


def test_ties():
    """Equal scores go to the lower page, over CTAs and warps; all equal; two values."""
    c = make([16 * 5000], [1], 2, 2, 64, 16)
    c["codes"][:] = c["codes"][:1]
    c["byte"][:] = 120
    check(c, 100)
    g = torch.Generator().manual_seed(2)
    c["byte"] = torch.where(torch.rand(c["byte"].shape, generator=g) < 0.01, 121, 120).to(U8)
    check(c, 100)
    c["codes"].zero_()                       # all scores 0, from either side
    c["q"][0, 0] = -c["q"][0, 0]
    check(c, 100, first=0)


def test_extreme_codes():
    """The largest products: |c| = 255 against 127 in every channel, both signs."""
    for d in (64, 256):
        c = make([16 * 400], [1], 16, 1, d, 16)
        g = torch.Generator().manual_seed(d)
        c["codes"] = torch.where(torch.rand(c["codes"].shape, generator=g) < 0.02, 126, 127).to(I8)
        c["codes"][:, :, 0] *= -1
        c["byte"][:] = 120
        sign = torch.where(torch.rand(1, 16, d, generator=g) < 0.5, -1.0, 1.0)
        c["q"] = (sign * 1.9921875).to(BF16)
        check(c, 50)
        c["q"] = torch.where(torch.rand(1, 16, d, generator=g) < 0.1, 1.984375, 1.9921875).to(BF16) * sign.to(BF16)
        check(c, 50)


def test_scales_far_apart():
    """Heads and pages of very different sizes, subnormal and infinite scores."""
    c = make([16 * 300], [1], 8, 1, 64, 16)
    size = torch.tensor([2.0 ** x for x in (120, -120, 0, 100, -130, 60, -60, 127)])
    c["q"] = (torch.randn(1, 8, 64, generator=torch.Generator().manual_seed(3)).clamp(-1, 1)
              * size[None, :, None]).to(BF16)
    g = torch.Generator().manual_seed(4)
    for lo, hi in ((1, 250), (1, 30), (200, 250), (120, 124)):
        c["byte"] = torch.randint(lo, hi, c["byte"].shape, generator=g).to(U8)
        check(c, 40)
        # heads whose say is only in small ones
        keep = c["q"]
        c["q"] = c["q"] * torch.tensor([0, 1, 0, 0, 1, 0, 1, 0])[None, :, None]
        check(c, 40)
        c["q"] = -c["q"].abs()
        c["codes"][:, :, 0] = c["codes"][:, :, 0].abs().clamp(min=1)   # every score is negative
        check(c, 40)
        c["q"] = keep


@pytest.mark.parametrize("hq", [1, 2, 8, 16])
def test_values_in_tiles(hq):
    """Scales far apart, ties, scores of 0 and values that are not finite, for several
    queries at a time."""
    c = make([16 * 300, 16 * 50 + 3], [11, 5], hq, 1, 64, 16)
    kept = c["q"], c["codes"], c["byte"]
    g = torch.Generator().manual_seed(6)
    size = torch.randint(-130, 127, (16, hq, 1), generator=g).float()
    c["q"] = (kept[0].float().clamp(-1, 1) * torch.exp2(size)).to(BF16)
    for lo, hi in ((1, 250), (1, 30), (200, 250), (120, 124)):
        c["byte"] = torch.randint(lo, hi, c["byte"].shape, generator=g).to(U8)
        check(c, 40, extra=MANY)
    c["q"], c["byte"] = kept[0].clone(), kept[2].clone()
    bad = torch.rand(c["byte"].shape, generator=g) < 0.05
    c["byte"][bad] = 255
    check(c, 30, extra=MANY)
    check(c, 3, extra=MANY)
    c["q"][3, 0, 7] = float("nan")
    c["q"][5] = float("inf")
    c["q"][6, :, 1] = float("-inf")
    check(c, 30, extra=MANY)
    c["q"], c["byte"] = kept[0], torch.full_like(c["byte"], 120)
    c["codes"] = kept[1].clone()
    c["codes"][:] = c["codes"][:1]
    check(c, 40, extra=MANY)                  # all alike
    c["byte"] = torch.where(torch.rand(c["byte"].shape, generator=g) < 0.05, 121, 120).to(U8)
    check(c, 40, extra=MANY)                  # two values
    c["codes"].zero_()
    check(c, 40, first=0, extra=MANY)


def test_page_ids_out_of_range_in_tiles():
    c = make([16 * 90], [9], 4, 1, 64, 16)
    w = want(c, 20, 1, 1)
    lost = [p for p in range(1, 85) if p in w[4, 0].tolist()][3]
    table = c["table"].clone()
    table[0, lost] = c["codes"].shape[0]
    err = torch.zeros(1, dtype=I32, device=DEV)
    q = torch.cat([c["q"], torch.zeros(MANY, 4, 64, dtype=BF16)])
    cu, lens = (torch.tensor(x, dtype=I32, device=DEV) for x in ([0, 9], [16 * 90]))
    got = pkv.select_pages(q.to(DEV), c["codes"].to(DEV), c["byte"].to(DEV), table.to(DEV), lens, 16 * 90,
                           20, 16, cu_seq_lens_q=cu, dev_error=err)
    assert pkv.get_device_error(err) == pkv.DEVERR_BLOCK_ID
    for t in range(9):
        pages = got[t, 0].tolist()
        assert lost not in pages and set(w[t, 0].tolist()) - {lost} <= set(pages)


def test_zero_queries():
    c = make([16 * 100], [1], 4, 2, 64, 16)
    c["q"].zero_()
    check(c, 10)
    c["q"][0, 1, 3] = -1.0
    check(c, 10)


def test_not_finite():
    """Pages with byte 255 come first, heads that are not finite have no say."""
    c = make([16 * 200, 16 * 90], [1, 1], 6, 2, 64, 16)
    g = torch.Generator().manual_seed(5)
    bad = torch.rand(c["byte"].shape, generator=g) < 0.05
    c["byte"][bad] = 255
    c["codes"][bad] = 0
    check(c, 30)
    check(c, 4)                               # more of them than there is room for
    c["q"][0, 1, 7] = float("nan")
    c["q"][0, 2, 0] = float("inf")
    c["q"][1, 3:, 5] = float("-inf")          # the whole group of kv head 1
    check(c, 30)


def test_page_ids_and_lengths_out_of_range():
    c = make([16 * 60], [1], 4, 1, 64, 16)
    ok = want(c, 20, 1, 1)[0, 0].tolist()
    out = [p for p in range(60) if p not in ok]
    args = [c["q"].to(DEV), c["codes"].to(DEV), c["byte"].to(DEV)]
    err = torch.zeros(1, dtype=I32, device=DEV)
    table = c["table"].clone()
    table[0, out[3]], table[0, ok[4]] = -1, c["codes"].shape[0]
    lens = torch.tensor([16 * 60], dtype=I32, device=DEV)
    got = pkv.select_pages(*args, table.to(DEV), lens, 16 * 60, 20, 16, dev_error=err)
    assert pkv.get_device_error(err, clear=True) == pkv.DEVERR_BLOCK_ID
    assert set(ok) - {ok[4]} <= set(got[0, 0].tolist()) and out[3] not in got[0, 0].tolist()
    lens.fill_(16 * 61 + 1)                   # beyond the maximum: clipped to it
    got = pkv.select_pages(*args, c["table"].to(DEV), lens, 16 * 60, 20, 16, dev_error=err)
    assert pkv.get_device_error(err, clear=True) == pkv.DEVERR_SEQLEN
    assert got[0, 0].tolist() == ok
    lens.fill_(-4)
    got = pkv.select_pages(*args, c["table"].to(DEV), lens, 16 * 60, 20, 16, dev_error=err)
    assert pkv.get_device_error(err) == pkv.DEVERR_SEQLEN
    assert bool((got == -1).all())


@pytest.mark.parametrize("rows", [4, 4 + MANY])
def test_offsets_that_are_none(rows):
    """Offsets that decrease or leave the rows: no row is written twice or read beyond."""
    c = make([160, 160], [rows // 2, rows // 2], 2, 1, 64, 16)
    args = (c["q"].to(DEV), c["codes"].to(DEV), c["byte"].to(DEV), c["table"].to(DEV),
            torch.tensor(c["lens"], dtype=I32, device=DEV), 160, 4, 16)
    for cu in ([2, 1, rows], [0, rows + 5, 3], [3, 3, 3], [-5, 0, 900], [rows, 2, 0]):
        got = pkv.select_pages(*args, cu_seq_lens_q=torch.tensor(cu, dtype=I32, device=DEV),
                               pages=torch.full((rows, 1, 4), -9, dtype=I32, device=DEV))
        assert bool(((got >= -1) & (got < 10) | (got == -9)).all())


@pytest.mark.parametrize("n", [4, 4 + MANY])
@pytest.mark.parametrize("cu", ["0 n+2", "0 n-1 n+7", "0 2 n+9 n+9", "-3 2 n", "-9 -4 n", "2 n+1 n+1",
                                "0 n n+5 n+9", "n n+1 n+2", "0 2 2**31-1 2**31-1"])
def test_offsets_outside_the_rows(cu, n):
    """They are flagged; a request has the rows that exist, its last one at its last
    position, and nothing else is written."""
    cu = [eval(x, {"n": n}) for x in cu.split()]
    lens = [1000, 777, 1300][:len(cu) - 1]
    c = make(lens, [0] * (len(lens) - 1) + [n], 4, 2, 64, 16)
    whole = torch.full((n + 6, 2, 9), -9, dtype=I32, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    pkv.select_pages(c["q"].to(DEV), c["codes"].to(DEV), c["byte"].to(DEV), c["table"].to(DEV),
                     torch.tensor(lens, dtype=I32, device=DEV), 1300, 9, 16, dev_error=err,
                     cu_seq_lens_q=torch.tensor(cu, dtype=I32, device=DEV), pages=whole[3:3 + n])
    assert pkv.get_device_error(err) == pkv.DEVERR_SEQLEN
    w = torch.full((n + 6, 2, 9), -9, dtype=I32)
    for r, (a, b) in enumerate(zip(cu, cu[1:])):
        b = min(b, n)
        for t in range(max(a, 0), b):
            m = max(0, lens[r] - (b - t) + 1)
            ids = c["table"][r, :S.pages_of(m, 16)].long()
            w[3 + t] = S.choose(S.scores(c["q"][t], c["codes"][ids], c["byte"][ids]), 9, 1, 1)
    assert torch.equal(whole.cpu(), w)


@pytest.mark.parametrize("n", [1, 8, 4 + MANY])
def test_offsets_that_decrease(n):
    """Flagged wherever they stand, also in requests that no row belongs to; nothing outside
    the rows is written."""
    c = make([160], [n], 2, 1, 64, 16)
    args = [c[x].to(DEV) for x in ("q", "codes", "byte")]
    for batch in (3, 300, 1000):
        table = c["table"].expand(batch, -1).contiguous().to(DEV)
        lens = torch.full((batch,), 160, dtype=I32, device=DEV)
        for at in {1, batch // 2, batch - 1, batch}:
            cu = [0] + [n] * batch
            cu[at] = n - 1 if at > 1 else n + 1   # (in the second place: above the third)
            err = torch.zeros(1, dtype=I32, device=DEV)
            whole = torch.full((n + 6, 1, 4), -9, dtype=I32, device=DEV)
            pkv.select_pages(*args, table, lens, 160, 4, 16, dev_error=err, pages=whole[3:3 + n],
                             cu_seq_lens_q=torch.tensor(cu, dtype=I32, device=DEV))
            assert pkv.get_device_error(err) == pkv.DEVERR_SEQLEN, (batch, at)
            assert bool((whole[:3] == -9).all()) and bool((whole[-3:] == -9).all())


def test_in_a_graph_and_on_two_streams():
    c = make([16 * 700, 16 * 30 + 4], [1, 1], 8, 2, 128, 16)
    a = [x.to(DEV) for x in (c["q"], c["codes"], c["byte"], c["table"])]
    lens = torch.tensor(c["lens"], dtype=I32, device=DEV)
    w = want(c, 32, 1, 1)
    graph = torch.cuda.CUDAGraph()
    pkv.select_pages(*a, lens, 16 * 700, 32, 16)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = pkv.select_pages(*a, lens, 16 * 700, 32, 16)
    for _ in range(3):
        got.zero_()
        graph.replay()
        assert torch.equal(got.cpu(), w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [pkv.select_pages(*a, lens, 16 * 700, 32, 16, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), w) for o in outs)
