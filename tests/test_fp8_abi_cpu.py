"""The 8-bit cache's, the tree attention's and the fused norm's C entry points
refuse what they document as refused, before any CUDA call (CPU only; the
pointers are fake, so these run only where no GPU is present)."""
import math

import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv

nogpu = pytest.mark.skipif(torch.cuda.is_available(),
                           reason="fake-pointer validation tests run without a GPU only")
FAKE = 0x10000
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
LAUNCHED = "valid: only the missing device stops it"


def _desc(nb=64, bs=16, hkv=8, d=128, dtype=pkv.PKV_E4M3, layout=0):
    return pkv.CacheDesc(nb, bs, hkv, d, dtype, layout)


def _check(st, expected):
    if expected is LAUNCHED:
        assert st not in (OK, INVALID, UNSUPPORTED, WORKSPACE)
    else:
        assert st == expected


# what is wrong with a pool, whatever the call; the calls that also take plain
# pools accept more dtypes
POOLS = [
    (dict(nb=0), INVALID), (dict(bs=0), INVALID), (dict(hkv=0), INVALID), (dict(d=0), INVALID),
    (dict(d=72), UNSUPPORTED), (dict(d=512), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(bs=64), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(layout=2), UNSUPPORTED),
    (dict(nb=1 << 27), UNSUPPORTED),            # pool rows beyond int32
    (dict(nb=1 << 26, hkv=64), UNSUPPORTED),    # (page, head) pairs beyond int32
]
PLAIN = [(dict(dtype=pkv.PKV_BF16), UNSUPPORTED), (dict(dtype=pkv.PKV_F32), UNSUPPORTED)]


# ---------------------------------------------------------------- write
def _write(desc=None, key=FAKE, value=FAKE, ks=1024, vs=1024, dtype=1, kc=FAKE, vc=FAKE,
           ksc=FAKE, vsc=FAKE, slots=FAKE, n=10):
    return pkv.load_library().pkv_reshape_and_cache_fp8(
        key, value, ks, vs, dtype, kc, vc, ksc, vsc, slots, n, desc or _desc(), None, None)


@nogpu
@pytest.mark.parametrize("pool,expected", POOLS + PLAIN)
def test_write_pools(pool, expected):
    assert _write(_desc(**pool)) == expected


@nogpu
@pytest.mark.parametrize("kw,expected", [
    (dict(), LAUNCHED),
    (dict(n=0, key=None, slots=None), OK),
    (dict(n=-1), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED),
    (dict(ks=1023), INVALID), (dict(vs=1020), INVALID),       # shorter than a token
    (dict(ks=1028), INVALID), (dict(vs=1025), INVALID),       # not 16-byte multiples
    (dict(ks=1028, dtype=0), LAUNCHED),                        # 4 floats are 16 bytes
    (dict(ks=1 << 33, vs=1 << 33), LAUNCHED),
    (dict(key=None), INVALID), (dict(value=None), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(ksc=None), INVALID), (dict(vsc=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(key=FAKE + 8), INVALID), (dict(vc=FAKE + 4), INVALID), (dict(slots=FAKE + 4), INVALID),
    (dict(ksc=FAKE + 1), LAUNCHED),                            # the write's scales: any address
])
def test_write_arguments(kw, expected):
    _check(_write(**kw), expected)


# ---------------------------------------------------------------- gather
def _gather(desc=None, key=FAKE, value=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, bt=FAKE,
            max_blocks=8, cu=FAKE, batch=4, total=100):
    return pkv.load_library().pkv_gather_cache_fp8(
        key, value, kc, vc, ksc, vsc, desc or _desc(), bt, max_blocks, cu, batch, total, None, None)


@nogpu
@pytest.mark.parametrize("pool,expected", POOLS + PLAIN)
def test_gather_pools(pool, expected):
    assert _gather(_desc(**pool)) == expected


@nogpu
@pytest.mark.parametrize("kw,expected", [
    (dict(), LAUNCHED),
    (dict(batch=0), OK), (dict(total=0, key=None, value=None), OK),
    (dict(batch=-1), INVALID), (dict(total=-1), INVALID), (dict(max_blocks=0), INVALID),
    (dict(total=(1 << 30) + 1), UNSUPPORTED),
    (dict(key=None), INVALID), (dict(bt=None), INVALID), (dict(cu=None), INVALID),
    (dict(ksc=None), INVALID), (dict(value=FAKE + 2), INVALID), (dict(cu=FAKE + 2), INVALID),
])
def test_gather_arguments(kw, expected):
    _check(_gather(**kw), expected)


# ---------------------------------------------------------------- decode
def _decode(desc=None, out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, bt=FAKE,
            max_blocks=8, sl=FAKE, max_seqlen=128, batch=4, hq=32, window=-1, scale=0.1, part=0,
            ws=FAKE, ws_bytes=1 << 40):
    return pkv.load_library().pkv_paged_decode_fp8(
        out, q, kc, vc, ksc, vsc, desc or _desc(), bt, max_blocks, sl, max_seqlen, None, None,
        batch, hq, window, scale, part, None, ws, ws_bytes, None, None)


@nogpu
@pytest.mark.parametrize("pool,expected", POOLS + PLAIN)
def test_decode_pools(pool, expected):
    assert _decode(_desc(**pool), hq=64) == expected


@nogpu
@pytest.mark.parametrize("kw,expected", [
    (dict(), LAUNCHED),
    (dict(batch=0, q=None), OK),
    (dict(batch=-1), INVALID), (dict(batch=65536), INVALID),
    (dict(hq=0), INVALID), (dict(hq=12), INVALID), (dict(hq=256), UNSUPPORTED),
    (dict(max_seqlen=-1), INVALID), (dict(max_blocks=0), INVALID), (dict(window=-2), INVALID),
    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(part=-16), INVALID), (dict(part=24), INVALID), (dict(part=1 << 15), INVALID),
    (dict(part=16, max_seqlen=1 << 21), UNSUPPORTED),          # partitions beyond the grid
    (dict(part=16, max_seqlen=1 << 21, window=100), LAUNCHED),  # a window leaves a few
    (dict(max_seqlen=(1 << 30) + 1, window=100), UNSUPPORTED),  # 32-bit partition bounds
    (dict(max_seqlen=1 << 30, window=100), LAUNCHED),
    (dict(ws=None), LAUNCHED),                                  # one partition needs none
    (dict(max_seqlen=4096, ws=None), WORKSPACE),
    (dict(max_seqlen=4096, ws=FAKE + 16), WORKSPACE),
    (dict(max_seqlen=4096, ws_bytes=4096), WORKSPACE),
    (dict(out=None), INVALID), (dict(ksc=None), INVALID), (dict(sl=None), INVALID),
    (dict(ksc=FAKE + 8), INVALID), (dict(q=FAKE + 8), INVALID), (dict(kc=FAKE + 1), INVALID),
])
def test_decode_arguments(kw, expected):
    _check(_decode(**kw), expected)


@nogpu
def test_decode_workspace_is_enough_for_any_partition_it_may_choose():
    # partition_size 0: what the size function gives for 0 suffices
    for batch, seqlen in ((1, 600), (4, 4096), (512, 131072), (65535, 8192)):
        need = pkv.paged_decode_workspace_size(batch, 32, 128, seqlen, 0)
        _check(_decode(batch=batch, max_seqlen=seqlen, ws_bytes=need), LAUNCHED)


# ---------------------------------------------------------------- norm + rope + write
def _norm(desc=None, query=FAKE, key=FAKE, value=FAKE, qs=4096, ks=1024, vs=1024, dtype=1,
          qo=FAKE, ko=FAKE, qos=4096, kos=1024, kc=FAKE, ksc=FAKE, vsc=FAKE, pos=FAKE, slots=FAKE,
          n=10, hq=32, qw=FAKE, kw=FAKE, eps=1e-6, table=FAKE, max_pos=4096, rd=128):
    return pkv.load_library().pkv_qk_norm_rope_reshape_and_cache(
        query, key, value, qs, ks, vs, dtype, qo, ko, qos, kos, kc, FAKE, ksc, vsc, pos, slots, n,
        hq, desc or _desc(), qw, kw, 1, eps, table, max_pos, rd, 1, None, None)


@nogpu
@pytest.mark.parametrize("pool,expected", POOLS + [
    (dict(dtype=pkv.PKV_BF16), LAUNCHED),
    (dict(dtype=pkv.PKV_F32), INVALID),         # bf16 rows into a float32 pool
])
def test_norm_pools(pool, expected):
    _check(_norm(_desc(**pool)), expected)


@nogpu
@pytest.mark.parametrize("kw,expected", [
    (dict(), LAUNCHED),
    (dict(n=0, key=None), OK),
    (dict(n=-1), INVALID), (dict(hq=-1), INVALID), (dict(max_pos=0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=0.0), LAUNCHED),
    (dict(dtype=2), UNSUPPORTED),
    (dict(rd=0), INVALID), (dict(rd=144), INVALID), (dict(rd=31), INVALID),
    (dict(rd=24), UNSUPPORTED), (dict(rd=16), LAUNCHED),
    (dict(hq=1 << 18, qs=1 << 25, qos=1 << 25), UNSUPPORTED),   # a q row beyond 2^24
    (dict(qs=4095), INVALID), (dict(qos=4088), INVALID), (dict(ks=1020), INVALID),
    (dict(vs=1030), INVALID), (dict(kos=1), INVALID),
    (dict(query=None, qo=None, qw=None, hq=0, qs=0, qos=0), LAUNCHED),
    (dict(query=None), INVALID), (dict(qo=None), INVALID), (dict(qw=None), INVALID),
    (dict(kw=None), INVALID), (dict(ko=None), INVALID), (dict(pos=None), INVALID),
    (dict(table=None), INVALID), (dict(ksc=None), INVALID), (dict(vsc=None), INVALID),
    (dict(table=FAKE + 8), INVALID), (dict(qw=FAKE + 4), INVALID), (dict(kw=FAKE + 4), INVALID),
    (dict(pos=FAKE + 4), INVALID), (dict(kc=FAKE + 8), INVALID),
])
def test_norm_arguments(kw, expected):
    _check(_norm(**kw), expected)


@nogpu
def test_norm_ignores_scales_of_a_plain_pool():
    _check(_norm(_desc(dtype=pkv.PKV_BF16), ksc=None, vsc=None), LAUNCHED)


# ---------------------------------------------------------------- tree attention
def _tree(desc=None, out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, bt=FAKE, max_blocks=8,
          cu=FAKE, sl=FAKE, max_q=16, max_seqlen=128, total_q=64, mask=FAKE, words=1, depth=FAKE,
          alibi=None, batch=4, hq=32, window=-1, scale=0.1, part=0, ws=FAKE, ws_bytes=1 << 40):
    return pkv.load_library().pkv_paged_tree_attention(
        out, q, kc, vc, ksc, vsc, desc or _desc(), bt, max_blocks, cu, sl, max_q, max_seqlen,
        total_q, mask, words, depth, None, alibi, batch, hq, window, scale, part, None, ws,
        ws_bytes, None, None)


@nogpu
@pytest.mark.parametrize("pool,expected", POOLS + [
    (dict(dtype=pkv.PKV_BF16), LAUNCHED), (dict(dtype=pkv.PKV_F32), UNSUPPORTED)])
def test_tree_pools(pool, expected):
    _check(_tree(_desc(**pool), hq=64), expected)


@nogpu
@pytest.mark.parametrize("kw,expected", [
    (dict(), LAUNCHED),
    (dict(batch=0, q=None), OK), (dict(total_q=0, out=None), OK), (dict(max_q=0), OK),
    (dict(batch=-1), INVALID), (dict(batch=65536), INVALID), (dict(hq=0), INVALID),
    (dict(hq=30), INVALID), (dict(hq=256), UNSUPPORTED),
    (dict(max_q=257, words=5), UNSUPPORTED), (dict(max_q=256, words=4), LAUNCHED),
    (dict(max_q=65, words=1), INVALID), (dict(max_q=-1), INVALID),
    (dict(max_seqlen=-1), INVALID), (dict(max_seqlen=(1 << 30) + 1), UNSUPPORTED),
    (dict(total_q=-1), INVALID), (dict(total_q=(1 << 24) + 1), UNSUPPORTED),
    (dict(max_blocks=0), INVALID), (dict(window=-2), INVALID), (dict(scale=math.inf), INVALID),
    (dict(part=-128), INVALID), (dict(part=100), INVALID), (dict(part=256), LAUNCHED),
    (dict(depth=None), LAUNCHED), (dict(depth=None, window=64), INVALID),
    (dict(depth=None, alibi=FAKE), INVALID),
    (dict(mask=None), INVALID), (dict(cu=None), INVALID), (dict(sl=None), INVALID),
    (dict(ksc=None), INVALID), (dict(vsc=FAKE + 8), INVALID), (dict(mask=FAKE + 4), INVALID),
    (dict(q=FAKE + 8), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE), (dict(ws_bytes=256), WORKSPACE),
])
def test_tree_arguments(kw, expected):
    _check(_tree(**kw), expected)


@nogpu
def test_tree_ignores_scales_of_a_plain_pool():
    _check(_tree(_desc(dtype=pkv.PKV_BF16), ksc=None, vsc=FAKE + 1), LAUNCHED)


def test_tree_workspace_size():
    size = pkv.paged_tree_attention_workspace_size
    # two partials of 128 rows (lse and D outputs, float32) per CTA, and a
    # place on the line of work per request and two words
    ctas = 152 // 8 * 8
    assert size(4, 32, 8, 128, 8) >= 2 * ctas * 128 * 129 * 4 + (4 + 2) * 8
    # two row tiles share a CTA; more do not need more
    assert size(4, 32, 8, 128, 64) > size(4, 32, 8, 128, 32)
    assert size(4, 32, 8, 128, 256) == size(4, 32, 8, 128, 64)
    # head size 256 takes one
    assert size(4, 32, 8, 256, 256) == size(4, 32, 8, 256, 8)
    # more kv heads than CTAs: one group
    assert size(1, 200, 200, 64, 8) >= 2 * 200 * 128 * 65 * 4
    # nothing to do
    assert size(0, 32, 8, 128, 8) == size(4, 4, 8, 128, 8) == size(4, 32, 8, 128, -1) == 256
