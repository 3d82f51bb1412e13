"""A prompt over the 8-bit cache, as a server runs it: the chunk's rows are
quantised into the pages, the requests' rows are read back, and the chunk attends
over them causally."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, I32 = torch.bfloat16, torch.int32


@pytest.mark.parametrize("layout,bs", [("NHD", 16), ("HND", 32)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64), (2, 1, 256)])
def test_write_read_back_and_prefill(hq, hkv, d, layout, bs):
    g = torch.Generator().manual_seed(d + bs)
    lens, chunk = [70, 5, 300, 129, 40], [30, 5, 129, 1, 0]   # whole and continued prompts
    nb = sum((n + bs - 1) // bs for n in lens) + 3
    pools = R.Pools(nb, bs, hkv, d, layout, True, g)
    table, slots = R.paged(lens, bs, nb, g)
    kc, vc, ks, vs = pools.device(DEV)
    total, rows = sum(lens), sum(chunk)
    q, = torch.randn(1, rows, hq, d, generator=g).to(BF16)
    new = torch.randn(2, rows, hkv, d, generator=g).to(BF16)
    at = torch.cat([s[n - m:] for s, n, m in zip(slots, lens, chunk)])
    cu_q = torch.tensor([0] + torch.tensor(chunk).cumsum(0).tolist(), dtype=I32, device=DEV)
    cu_k = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=I32, device=DEV)
    sink = torch.randn(hq, generator=g)
    err = torch.zeros(1, dtype=I32, device=DEV)

    def step(out):
        pkv.reshape_and_cache_fp8(new[0].to(DEV), new[1].to(DEV), kc, vc, ks, vs, at.to(DEV),
                                  dev_error=err, layout=layout)
        k, v = pkv.gather_cache_fp8(kc, vc, ks, vs, table.to(DEV), cu_k, total, dev_error=err,
                                    layout=layout)
        pkv.varlen_prefill_contiguous(q.to(DEV), k, v, cu_q, cu_k, max(chunk), max(lens),
                                      sink=sink.to(DEV), out=out, dev_error=err)
        return k, v

    out = torch.full((rows, hq, d), 7.0, dtype=BF16, device=DEV)
    k, v = step(out)
    assert pkv.get_device_error(err) == 0
    # what the pages hold: the old rows, and the chunk's as the format rounds them
    codes, byte = R.quantise(new)
    for i in range(2):
        pools.codes[i][at // bs, :, at % bs] = codes[i]
        pools.byte[i][at // bs, :, at % bs] = byte[i]
    want = pools.at(torch.cat(slots))
    assert torch.equal(k.cpu().to(torch.float64), want[0])
    assert torch.equal(v.cpu().to(torch.float64), want[1])
    row = 0
    for i, (n, m) in enumerate(zip(lens, chunk)):
        kk, vv = pools.at(slots[i])
        keep = torch.arange(n)[None] <= (n - m + torch.arange(m))[:, None]
        ref, _, absv, smax = R.attend(q[row:row + m], kk, vv, keep, d ** -0.5, sink)
        # bf16 weights: half a step is 2^-8
        R.assert_within(out[row:row + m], ref, R.out_bound(ref, absv, smax, d, 2.0 ** -8),
                        f"out {i}")
        row += m
    again = torch.zeros_like(out)
    step(again)
    assert R.same_bits(out, again)
