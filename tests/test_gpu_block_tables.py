"""update_block_tables on the GPU against the same steps on Python lists."""
import random

import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _sparse as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32, I64 = torch.int32, torch.int64


class Book:
    """The same tables on the device and as lists."""

    def __init__(self, batch, max_blocks, num_blocks, bs, seed=0):
        self.bs, self.nb, self.mb = bs, num_blocks, max_blocks
        ids = list(range(num_blocks))
        random.Random(seed).shuffle(ids)
        self.free, self.table = ids, [[-1] * max_blocks for _ in range(batch)]
        self.dtable = torch.full((batch, max_blocks), -1, dtype=I32, device=DEV)
        self.dfree = torch.tensor(ids, dtype=I32, device=DEV)
        self.dnum = torch.tensor([num_blocks], dtype=I32, device=DEV)
        self.lens = [0] * batch
        self.err = torch.zeros(1, dtype=I32, device=DEV)

    def call(self, new, rows, old=None, **kw):
        return pkv.update_block_tables(
            self.dtable, torch.tensor(self.lens if old is None else old, dtype=I32, device=DEV),
            torch.tensor(new, dtype=I32, device=DEV), self.dfree, self.dnum, self.bs, rows,
            dev_error=self.err, **kw)

    def same(self):
        assert self.dtable.tolist() == self.table
        assert self.dnum.item() == len(self.free)
        assert self.dfree[:len(self.free)].tolist() == self.free

    def step(self, new, pad=0, **kw):
        rows = sum(max(0, b - a) for a, b in zip(self.lens, new)) + pad
        want = S.step(self.table, self.free, self.lens, new, self.bs, rows)
        got = self.call(new, rows, **kw)
        for g, w in zip(got, want):
            assert g.tolist() == w
        assert [g.dtype for g in got] == [I64, I64, I32, I32]
        self.lens = list(new)
        self.same()
        assert pkv.get_device_error(self.err) == 0


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("batch", [1, 2, 7, 64, 513, 2000])
def test_steps(batch, bs):
    """Prompts, decode steps, drafts given back, requests done and admitted."""
    rng = random.Random(batch + bs)
    book = Book(batch, 40, 30 * batch + 5, bs, seed=batch)
    top = 30 * bs
    for it in range(6):
        new = []
        for n in book.lens:
            kind = rng.random()
            if n == 0:
                new.append(0 if kind < 0.3 else rng.randint(1, top))
            elif kind < 0.15:
                new.append(0)
            elif kind < 0.4:
                new.append(max(0, n - rng.randint(0, 40)))
            else:
                new.append(min(top, n + rng.choice([0, 1, 1, bs, rng.randint(0, 70)])))
        book.step(new, pad=rng.choice([0, 5]))


def test_the_first_page_of_the_stack_and_full_pages():
    book = Book(3, 4, 9, 16)
    book.step([16, 17, 32])
    book.step([17, 17, 48])      # a full page goes on in a new one; nothing moves
    book.step([17, 17, 48], pad=3)
    book.step([64, 0, 64])       # one page comes from the request that is done
    assert len(book.free) == 1
    book.step([0, 0, 0])
    assert sorted(book.free) == list(range(9))


def test_giving_back_what_was_taken_restores_the_stack():
    book = Book(5, 20, 80, 16)
    book.step([30, 16, 0, 100, 7])
    free, table, lens = list(book.free), [list(x) for x in book.table], list(book.lens)
    book.step([44, 80, 33, 101, 0])
    book.step(lens)
    assert book.free == free and book.table == table


@pytest.mark.parametrize("rows", [16384, 16385, 70001])
def test_many_rows(rows):
    """Rows written by the table kernel, and by one of their own."""
    book = Book(3, 9000, 18000, 16)
    book.step([40, 0, 9])
    book.step([40, rows - 777, 786], pad=0)
    book.step([0, rows - 777 - 300, 786 + rows], pad=11)


def test_large_batch():
    book = Book(16384, 3, 30000, 32)
    rng = random.Random(3)
    book.step([rng.randint(0, 40) for _ in range(16384)])
    book.step([rng.choice([0, n, min(96, n + 1), min(96, n + 30)]) for n in book.lens])


def test_no_requests():
    book = Book(0, 4, 8, 16)
    got = book.call([], 5, old=[])
    assert got[0].tolist() == [-1] * 5 and got[1].tolist() == [0] * 5
    assert got[2].tolist() == [0] and got[3].tolist() == [0]
    book.same()


BAD = {
    "no pages": (dict(new=[20, 160, 33]), pkv.DEVERR_NO_BLOCKS),
    "negative": (dict(new=[20, -1, 33]), pkv.DEVERR_SEQLEN),
    "negative before": (dict(new=[20, 40, 33], old=[20, -5, 33]), pkv.DEVERR_SEQLEN),
    "longer than the table": (dict(new=[20, 161, 33]), pkv.DEVERR_SEQLEN),
    "rows": (dict(new=[20, 60, 34], rows=20), pkv.DEVERR_SEQLEN),
    "height": (dict(new=[20, 40, 34], num=13), pkv.DEVERR_BLOCK_ID),
    "negative height": (dict(new=[20, 40, 34], num=-1), pkv.DEVERR_BLOCK_ID | pkv.DEVERR_NO_BLOCKS),
    "too many pages": (dict(new=[20, 0, 0], num=12), pkv.DEVERR_BLOCK_ID),
    "released id": (dict(new=[20, 0, 33], spoil=1), pkv.DEVERR_BLOCK_ID),
    "free id": (dict(new=[20, 41, 80], free=-3), pkv.DEVERR_BLOCK_ID),
    "page that goes on": (dict(new=[20, 41, 33], spoil=2), pkv.DEVERR_BLOCK_ID),
}


@pytest.mark.parametrize("many", [0, 20000])
@pytest.mark.parametrize("what", sorted(BAD))
def test_nothing_moves_after_an_error(what, many):
    """12 pages, 8 of them taken: lengths 20, 40, 33; nothing changes but the outputs."""
    kw, bits = BAD[what]
    book = Book(3, 10, 12, 16)
    book.step([20, 40, 33])
    if "spoil" in kw:
        book.dtable[1, kw["spoil"]] = 12 if kw["spoil"] == 1 else -1
    if "free" in kw:
        book.dfree[len(book.free) - 1] = kw["free"]
    if "num" in kw:
        book.dnum.fill_(kw["num"])
    before = [x.clone() for x in (book.dtable, book.dfree, book.dnum)]
    rows = kw.get("rows", 200 + many)
    got = book.call(kw["new"], rows, old=kw.get("old"))
    assert pkv.get_device_error(book.err) == bits
    with pytest.raises(pkv.PkvError, match="OUT_OF_RANGE"):
        pkv.get_device_error(book.err, raise_on_error=True)
    for a, b in zip(before, (book.dtable, book.dfree, book.dnum)):
        assert torch.equal(a, b)
    assert bool((got[0] == -1).all()) and bool((got[1] == 0).all())
    assert got[2].tolist() == [0] * 4 and got[3].tolist() == [0] * 4


def test_lengths_beyond_32_bits_in_sum():
    """Sums of lengths and of pages are kept in 64 bits."""
    book = Book(300, 1 << 16, 600, 16)
    book.call([1 << 20] * 300, 8, old=[0] * 300)
    assert pkv.get_device_error(book.err, clear=True) & (pkv.DEVERR_SEQLEN | pkv.DEVERR_NO_BLOCKS)
    book.call([0] * 300, 8, old=[1 << 20] * 300)   # 19.7 million pages to give back
    assert pkv.get_device_error(book.err) == pkv.DEVERR_BLOCK_ID
    book.same()


@pytest.mark.parametrize("batch,old,new,bits", [
    (3, 1 << 29, 1 << 29, 0), (4, 1 << 29, 1 << 29, pkv.DEVERR_SEQLEN),      # 2^31
    (9, 1 << 29, 1 << 29, pkv.DEVERR_SEQLEN),                               # 2^32 + 2^29
    (8, 0, 1 << 29, pkv.DEVERR_SEQLEN | pkv.DEVERR_NO_BLOCKS),              # 2^32 tokens
    (8, 1 << 29, 0, pkv.DEVERR_BLOCK_ID),                                   # 2^28 pages back
])
def test_sums_that_pass_32_bits(batch, old, new, bits):
    """Lengths of which each is in range and the sum of all is not: of the keys alone
    (nothing grows, no page moves), of the tokens, of the pages."""
    table = torch.full((batch, 1 << 25), -1, dtype=I32, device=DEV)
    free = torch.arange(40, dtype=I32, device=DEV)
    num, err = torch.tensor([40], dtype=I32, device=DEV), torch.zeros(1, dtype=I32, device=DEV)
    lens = [torch.full((batch,), x, dtype=I32, device=DEV) for x in (old, new)]
    got = pkv.update_block_tables(table, *lens, free, num, 16, 8, dev_error=err)
    assert pkv.get_device_error(err) == bits
    assert got[0].tolist() == [-1] * 8 and got[1].tolist() == [0] * 8
    assert got[2].tolist() == [0] * (batch + 1)
    assert got[3].tolist() == [0 if bits else (new * r) for r in range(batch + 1)]
    assert num.item() == 40 and free.tolist() == list(range(40)) and bool((table == -1).all())


def test_outputs_given_and_streams():
    book = Book(4, 8, 20, 16)
    outs = dict(slot_mapping=torch.full((9,), 5, dtype=I64, device=DEV),
                positions=torch.full((9,), 5, dtype=I64, device=DEV),
                cu_seq_lens_q=torch.full((5,), 5, dtype=I32, device=DEV),
                cu_seq_lens_k=torch.full((5,), 5, dtype=I32, device=DEV))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = book.call([3, 0, 2, 1], 9, stream=s, **outs)
    s.synchronize()
    assert all(a is b for a, b in zip(got, outs.values()))
    want = S.step(book.table, book.free, [0] * 4, [3, 0, 2, 1], 16, 9)
    assert [g.tolist() for g in got] == list(map(list, want))
    book.same()


def test_in_a_graph():
    """Captured once, replayed while the lengths change in place."""
    book = Book(6, 10, 60, 16)
    old, new = (torch.zeros(6, dtype=I32, device=DEV) for _ in range(2))
    args = (book.dtable, old, new, book.dfree, book.dnum, 16, 64)
    new.fill_(0)
    pkv.update_block_tables(*args, dev_error=book.err)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pkv.update_block_tables(*args, dev_error=book.err)
    lens = [0] * 6
    for to in ([5, 0, 17, 9, 1, 16], [6, 1, 18, 10, 2, 17], [0, 2, 19, 0, 3, 18], [8, 3, 20, 4, 0, 19]):
        old.copy_(torch.tensor(lens))
        new.copy_(torch.tensor(to))
        graph.replay()
        want = S.step(book.table, book.free, lens, to, 16, 64)
        assert [g.tolist() for g in got] == list(map(list, want))
        book.same()
        lens = to
    assert pkv.get_device_error(book.err) == 0
