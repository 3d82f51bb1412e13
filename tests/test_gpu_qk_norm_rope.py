"""qk_norm_rope_reshape_and_cache on the GPU against the 64-bit definition."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def bound(ref, mag, dtype):
    """Half a step of the type; in fp32: the sum of squares adds at most 8 + 5
    terms deep, the mean, eps, root, reciprocal, two products of the norm and
    two of the rotation round once each (2^-24): under 24 roundings of the
    magnitudes an output adds, and as much of the half step again where the
    rounded value sits next to a border."""
    return HALF[dtype] * ref.abs() + 24 * 2.0 ** -24 * mag * 1.01 + 1e-37


def pool_shape(nb, bs, hkv, d, layout):
    return (nb, bs, hkv, d) if layout == "NHD" else (nb, hkv, bs, d)


def run(tokens, hq, hkv, d, rd, neox=True, dtype=BF16, fp8=False, layout="NHD", bs=16,
        in_place=False, w32=True, eps=1e-6, seed=0, size=1.0, maxpos=500):
    g = torch.Generator().manual_seed(seed + tokens + d)
    qkv = (torch.randn(tokens, hq + 2 * hkv, d, generator=g) * size *
           torch.exp2(2 * torch.randn(tokens, hq + 2 * hkv, 1, generator=g))).to(dtype)
    qw, kw = (1 + 0.3 * torch.randn(2, d, generator=g)).to(F32 if w32 else dtype)
    pos = torch.randint(0, maxpos, (tokens,), generator=g)
    nb = (tokens + bs - 1) // bs + 2
    slots = torch.randperm(nb * bs, generator=g)[:tokens]
    slots[2::5] = -1
    table = pkv.rope_cos_sin_table(maxpos, rd)
    dev = qkv.to(DEV)
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    shape = pool_shape(nb, bs, hkv, d, layout)
    if fp8:
        pools = [torch.full(shape, 0x11, dtype=U8, device=DEV).view(R.E4M3) for _ in range(2)]
        scales = [torch.full((nb, hkv, bs), 77, dtype=U8, device=DEV) for _ in range(2)]
    else:
        pools, scales = [torch.full(shape, 3.0, dtype=dtype, device=DEV) for _ in range(2)], [None, None]
    qo = None if in_place else torch.empty(tokens, hq, d, dtype=dtype, device=DEV)
    ko = None if in_place else torch.empty(tokens, hkv, d, dtype=dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.qk_norm_rope_reshape_and_cache(
        q if hq else None, k, v, pools[0], pools[1], pos.to(DEV), slots.to(DEV), table,
        qw.to(DEV) if hq else None, kw.to(DEV), eps=eps, rotary_dim=rd, is_neox_style=neox,
        query_out=qo if hq else None, key_out=ko, k_scale=scales[0], v_scale=scales[1],
        layout=layout, dev_error=err)
    assert pkv.get_device_error(err) == 0
    got_q, got_k = (q, k) if in_place else (qo, ko)
    tab = table.cpu()
    for got, x, w in ((got_q, qkv[:, :hq], qw), (got_k, qkv[:, hq:hq + hkv], kw)):
        ref, mag = R.norm_rope(x, w, eps, tab, pos, rd, neox)
        R.assert_within(got, ref, bound(ref, mag, dtype), "rotated")
    assert R.same_bits(v, qkv[:, hq + hkv:])  # the value is only read
    if not in_place:
        assert R.same_bits(dev, qkv)
    keep = slots >= 0
    s = slots[keep]
    b, o = s // bs, s % bs
    for x, pool, scale in ((got_k.cpu(), pools[0], scales[0]),
                           (qkv[:, hq + hkv:], pools[1], scales[1])):
        if fp8:
            codes, byte = R.quantise(x)
            want, src = torch.full(shape, 0x11, dtype=U8), codes
            wantb = torch.full((nb, hkv, bs), 77, dtype=U8)
            wantb[b, :, o] = byte[keep]
            assert torch.equal(scale.cpu(), wantb)
            have = pool.view(U8).cpu()
        else:
            want, src, have = torch.full(shape, 3.0, dtype=dtype), x, pool.cpu()
        if layout == "NHD":
            want[b, o] = src[keep]
        else:
            want[b, :, o] = src[keep]
        assert R.same_bits(have, want)


@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("d,rd", [(64, 64), (64, 32), (80, 80), (96, 64), (112, 16), (128, 128),
                                  (128, 48), (256, 256), (256, 64)])
def test_head_sizes(d, rd, fp8, neox):
    run(37, 4, 2, d, rd, neox, fp8=fp8)


@pytest.mark.parametrize("dtype,fp8,w32", [(BF16, False, False), (F32, False, True),
                                           (F32, True, True), (BF16, True, False)])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("tokens,hq,hkv", [(1, 1, 1), (2, 32, 8), (7, 3, 1), (301, 8, 8),
                                           (19, 0, 2), (1000, 64, 8)])
def test_tokens_heads_types(tokens, hq, hkv, layout, dtype, fp8, w32):
    run(tokens, hq, hkv, 128, 128, dtype=dtype, fp8=fp8, layout=layout, bs=32, w32=w32)


@pytest.mark.parametrize("fp8", [True, False])
def test_in_place(fp8):
    run(50, 8, 2, 128, 64, fp8=fp8, in_place=True)


def test_sizes_of_the_values():
    run(40, 4, 2, 128, 128, size=1e-6, fp8=True)        # eps dominates
    run(40, 4, 2, 128, 128, size=1e4, fp8=True)
    run(40, 4, 2, 64, 64, size=0.0, fp8=True)           # zero rows stay zero
    run(40, 4, 2, 64, 64, dtype=F32, size=1e-3, eps=1e-5)


def test_bad_positions_and_slots_are_skipped():
    t, hq, hkv, d = 9, 2, 1, 64
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(t, h, d, generator=g).to(BF16).to(DEV) for h in (hq, hkv, hkv))
    q0, k0 = q.clone(), k.clone()
    table = pkv.rope_cos_sin_table(64, d)
    w = torch.ones(d, device=DEV)
    pos = torch.tensor([0, 1, 64, 3, -1, 5, 6, 7, 8], device=DEV)
    slots = torch.tensor([0, 1, 2, 16, 4, 5, 6, 1 << 33, -1], device=DEV)
    kc, vc = (torch.full((1, 16, hkv, d), 3.0, dtype=BF16, device=DEV) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.qk_norm_rope_reshape_and_cache(q, k, v, kc, vc, pos, slots, table, w, w, dev_error=err)
    assert pkv.get_device_error(err) == pkv.DEVERR_POSITION | pkv.DEVERR_SLOT
    for t_ in (2, 4):                                    # untouched tokens
        assert R.same_bits(q[t_], q0[t_]) and R.same_bits(k[t_], k0[t_])
    written = [0, 1, 5, 6]
    for i in range(16):
        if i in written:
            assert R.same_bits(kc[0, i], k[i]) and R.same_bits(vc[0, i], v[i])
        else:
            assert bool((kc[0, i] == 3.0).all()) and bool((vc[0, i] == 3.0).all())


def test_the_fused_write_equals_the_separate_calls():
    """Quantising in the fused call gives the bits of reshape_and_cache_fp8 on
    its rotated key; captured and replayed, the same bits again."""
    t, hq, hkv, d, bs = 65, 8, 2, 128, 16
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(t, h, d, generator=g).to(BF16).to(DEV) for h in (hq, hkv, hkv))
    table = pkv.rope_cos_sin_table(4096, d)
    qw, kw = torch.randn(2, d, generator=g).to(DEV)
    pos = torch.randint(0, 4096, (t,), generator=g).to(DEV)
    slots = torch.randperm(6 * bs, generator=g)[:t].to(DEV)

    def pools():
        return [torch.zeros(6, bs, hkv, d, dtype=U8, device=DEV).view(R.E4M3) for _ in range(2)] + \
            [torch.zeros(6, hkv, bs, dtype=U8, device=DEV) for _ in range(2)]

    a, b = pools(), pools()
    qo, ko = torch.empty_like(q), torch.empty_like(k)

    def fused(p):
        pkv.qk_norm_rope_reshape_and_cache(q, k, v, p[0], p[1], pos, slots, table, qw, kw,
                                           query_out=qo, key_out=ko, k_scale=p[2], v_scale=p[3])
    fused(a)
    want = (qo.clone(), ko.clone())
    pkv.reshape_and_cache_fp8(ko, v, *b, slots)
    for x, y in zip(a, b):
        assert R.same_bits(x, y)
    c = pools()
    qo.zero_()
    ko.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fused(c)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(c + [qo, ko], a + list(want)):
        assert R.same_bits(x, y)
