"""One tensor as key and value of the fused norm, rotation and write: the pools get
the normed key and the value as it was, and the tensor the key."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("neox", [False, True])
@pytest.mark.parametrize("tokens,hq,hkv,d", [(1, 2, 1, 64), (70, 8, 3, 128), (300, 20, 20, 256),
                                             (1500, 40, 40, 64)])
def test_key_is_value(tokens, hq, hkv, d, neox, dtype, fp8):
    g = torch.Generator().manual_seed(tokens + d)
    bs = 16
    nb = (tokens + bs - 1) // bs + 1
    q = torch.randn(tokens, hq, d, generator=g).to(dtype).to(DEV)
    x = torch.randn(tokens, hkv, d, generator=g).to(dtype).to(DEV)
    table = pkv.rope_cos_sin_table(2048, d)
    w = torch.randn(2, d, generator=g).to(DEV)
    pos = torch.randint(0, 2048, (tokens,), generator=g).to(DEV)
    slots = torch.randperm(nb * bs, generator=g)[:tokens].to(DEV)

    def call(key, value, **kw):
        pools = [torch.zeros(nb, bs, hkv, d, dtype=torch.uint8, device=DEV).view(R.E4M3)
                 if fp8 else torch.zeros(nb, bs, hkv, d, dtype=dtype, device=DEV)
                 for _ in range(2)]
        scales = [torch.zeros(nb, hkv, bs, dtype=torch.uint8, device=DEV) if fp8 else None
                  for _ in range(2)]
        pkv.qk_norm_rope_reshape_and_cache(q.clone(), key, value, *pools, pos, slots, table, w[0],
                                           w[1], is_neox_style=neox, k_scale=scales[0],
                                           v_scale=scales[1], **kw)
        return pools + [s for s in scales if s is not None]

    key = x.clone()
    want = call(key, x.clone())
    both = x.clone()
    for got, out in ((call(both, both), both), (call(x.clone(), v := x.clone(), key_out=v), v)):
        assert R.same_bits(out, key)
        for a, b in zip(got, want):
            assert R.same_bits(a, b)
