"""Reading back nothing needs no pages (CPU only; fake pointers)."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv

FAKE = 0x10000
OK, INVALID = 0, 1


@pytest.mark.skipif(torch.cuda.is_available(),
                    reason="fake-pointer validation tests run without a GPU only")
@pytest.mark.parametrize("batch,total,max_blocks,expected", [
    (3, 0, 0, OK), (0, 0, 0, OK), (0, 5, 0, OK), (3, 1, 0, INVALID), (3, 0, -1, INVALID)])
def test_gather(batch, total, max_blocks, expected):
    desc = pkv.CacheDesc(64, 16, 8, 128, pkv.PKV_E4M3, 0)
    assert pkv.load_library().pkv_gather_cache_fp8(
        FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, desc, FAKE, max_blocks, FAKE, batch, total, None,
        None) == expected
