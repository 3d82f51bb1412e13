"""The sparse step's C entry points refuse what they document as refused, before any
CUDA call (CPU only; the pointers are fake, so these run only where no GPU is present)."""
import math

import pytest

import paged_kv_cache_attention_gb300 as pkv
from test_fp8_abi_cpu import FAKE, INVALID, LAUNCHED, OK, UNSUPPORTED, _check, _desc, nogpu


def _tables(bt=FAKE, mb=8, old=FAKE, new=FAKE, batch=4, free=FAKE, nb=64, num=FAKE, bs=16,
            slots=FAKE, pos=FAKE, rows=10, cuq=FAKE, cuk=FAKE):
    return pkv.load_library().pkv_update_block_tables(bt, mb, old, new, batch, free, nb, num, bs,
                                                      slots, pos, rows, cuq, cuk, None, None)


@nogpu
@pytest.mark.parametrize("kw,expected", [
    (dict(), LAUNCHED), (dict(batch=0, bt=None, old=None, new=None), LAUNCHED),
    (dict(rows=0, slots=None, pos=None), LAUNCHED), (dict(mb=0, bt=None), LAUNCHED),
    (dict(batch=16384), LAUNCHED), (dict(batch=16385), UNSUPPORTED), (dict(batch=-1), INVALID),
    (dict(mb=-1), INVALID), (dict(nb=0), INVALID), (dict(nb=-5), INVALID),
    (dict(nb=1 << 27), UNSUPPORTED), (dict(nb=(1 << 27) - 1), LAUNCHED),
    (dict(rows=-1), INVALID), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(bs=0), INVALID), (dict(bs=8), UNSUPPORTED), (dict(bs=64), UNSUPPORTED),
    (dict(bs=32), LAUNCHED), (dict(mb=1 << 26), LAUNCHED), (dict(mb=(1 << 26) + 1), UNSUPPORTED),
    (dict(bt=None), INVALID), (dict(old=None), INVALID), (dict(new=None), INVALID),
    (dict(free=None), INVALID), (dict(num=None), INVALID), (dict(slots=None), INVALID),
    (dict(pos=None), INVALID), (dict(cuq=None), INVALID), (dict(cuk=None), INVALID),
    (dict(bt=FAKE + 2), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(pos=FAKE + 4), INVALID),
    (dict(num=FAKE + 1), INVALID), (dict(cuk=FAKE + 2), INVALID),
])
def test_tables(kw, expected):
    _check(_tables(**kw), expected)


SHAPES = [(dict(nb=0), INVALID), (dict(bs=0), INVALID), (dict(hkv=0), INVALID), (dict(d=0), INVALID),
          (dict(d=72), UNSUPPORTED), (dict(d=512), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
          (dict(bs=64), UNSUPPORTED), (dict(nb=1 << 27), UNSUPPORTED),
          (dict(nb=1 << 26, hkv=64), UNSUPPORTED)]
POOLS = SHAPES + [(dict(dtype=pkv.PKV_F32), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
                  (dict(layout=2), UNSUPPORTED), (dict(dtype=pkv.PKV_BF16), LAUNCHED)]


def _bounds(desc=None, k=FAKE, ks=FAKE, b=FAKE, s=FAKE, slots=FAKE, n=10):
    return pkv.load_library().pkv_update_page_bounds(k, ks, desc or _desc(), b, s, slots, n, None,
                                                     None)


@nogpu
@pytest.mark.parametrize("pool,expected", POOLS)
def test_bounds_pools(pool, expected):
    _check(_bounds(_desc(**pool)), expected)


@nogpu
@pytest.mark.parametrize("kw,expected", [
    (dict(), LAUNCHED), (dict(n=0, slots=None), OK), (dict(n=-1), INVALID),
    (dict(n=1 << 22), LAUNCHED), (dict(n=(1 << 22) + 1), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(ks=None), INVALID), (dict(b=None), INVALID),
    (dict(s=None), INVALID), (dict(slots=None), INVALID), (dict(k=FAKE + 8), INVALID),
    (dict(b=FAKE + 8), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(s=FAKE + 1), LAUNCHED),
    (dict(desc=_desc(dtype=pkv.PKV_BF16), ks=None), LAUNCHED),
])
def test_bounds_arguments(kw, expected):
    _check(_bounds(**kw), expected)


def _select(pages=FAKE, top_k=8, q=FAKE, b=FAKE, s=FAKE, nb=64, bs=16, hkv=8, d=128, bt=FAKE, mb=8,
            lens=FAKE, max_seqlen=100, cu=None, batch=4, total=4, hq=32, first=1, recent=1):
    return pkv.load_library().pkv_select_pages(pages, top_k, q, b, s, nb, bs, hkv, d, bt, mb, lens,
                                               max_seqlen, cu, batch, total, hq, first, recent, None,
                                               None)


ROWS = [
    (dict(batch=0, total=0), OK), (dict(cu=FAKE, total=0), OK), (dict(batch=0, cu=FAKE), OK),
    (dict(batch=-1), INVALID), (dict(total=-1, cu=FAKE), INVALID), (dict(total=5), INVALID),
    (dict(total=5, cu=FAKE), LAUNCHED), (dict(hq=0), INVALID), (dict(hq=33), INVALID),
    (dict(hq=128), LAUNCHED), (dict(hq=136), UNSUPPORTED), (dict(top_k=0), INVALID),
    (dict(top_k=16384), LAUNCHED), (dict(top_k=16385), UNSUPPORTED),
    (dict(cu=FAKE, total=(1 << 24) + 1), UNSUPPORTED), (dict(mb=0), INVALID), (dict(mb=-1), INVALID),
    (dict(q=None), INVALID), (dict(pages=None), INVALID), (dict(bt=None), INVALID),
    (dict(lens=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(pages=FAKE + 2), INVALID),
    (dict(cu=FAKE + 2), INVALID), (dict(lens=FAKE + 1), INVALID), (dict(bt=FAKE + 2), INVALID),
]


@nogpu
@pytest.mark.parametrize("shape,expected", SHAPES)
def test_select_shapes(shape, expected):
    _check(_select(**shape), expected)


@nogpu
@pytest.mark.parametrize("kw,expected", ROWS + [
    (dict(), LAUNCHED), (dict(first=-1), INVALID), (dict(recent=0), INVALID),
    (dict(first=7), LAUNCHED), (dict(first=8), INVALID), (dict(recent=9), INVALID),
    (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID),
    (dict(max_seqlen=-1), INVALID), (dict(max_seqlen=0), LAUNCHED),
    (dict(max_seqlen=262144 * 16), LAUNCHED), (dict(max_seqlen=262144 * 16 + 1), UNSUPPORTED),
    (dict(max_seqlen=262144 * 32, bs=32, d=256, hq=128), LAUNCHED),
    (dict(max_seqlen=2 ** 31 - 1), UNSUPPORTED), (dict(b=None), INVALID), (dict(s=None), INVALID),
    (dict(b=FAKE + 8), INVALID),
])
def test_select_arguments(kw, expected):
    _check(_select(**kw), expected)


def _sparse(out=FAKE, q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, desc=None, bt=FAKE, mb=8, lens=FAKE,
            cu=None, batch=4, total=4, pages=FAKE, top_k=8, sink=None, hq=32, scale=0.1, lse=None):
    return pkv.load_library().pkv_paged_sparse_attention(
        out, q, k, v, ks, vs, desc or _desc(), bt, mb, lens, cu, batch, total, pages, top_k, sink, hq,
        scale, lse, None, None)


@nogpu
@pytest.mark.parametrize("pool,expected", POOLS)
def test_sparse_pools(pool, expected):
    _check(_sparse(desc=_desc(**pool), hq=64), expected)


@nogpu
@pytest.mark.parametrize("kw,expected", ROWS + [
    (dict(), LAUNCHED), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=-1.0), LAUNCHED), (dict(out=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
    (dict(desc=_desc(dtype=pkv.PKV_BF16), ks=None, vs=None), LAUNCHED),
    (dict(out=FAKE + 8), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(ks=FAKE + 8), INVALID), (dict(vs=FAKE + 4), INVALID), (dict(sink=FAKE + 2), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(sink=FAKE, lse=FAKE), LAUNCHED),
])
def test_sparse_arguments(kw, expected):
    _check(_sparse(**kw), expected)
