"""The partition that paged_decode_fp8 chooses, seen through the workspace it asks
for (CPU only; the pointers are fake, so this runs only where no GPU is present)."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv

nogpu = pytest.mark.skipif(torch.cuda.is_available(),
                           reason="fake-pointer validation tests run without a GPU only")
FAKE = 0x10000
WORKSPACE = 3


def asks_for(batch, max_seqlen, window, nbytes):
    """Whether a workspace of nbytes is too small."""
    desc = pkv.CacheDesc(64, 16, 8, 128, pkv.PKV_E4M3, 0)
    st = pkv.load_library().pkv_paged_decode_fp8(
        FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, desc, FAKE, 1 << 16, FAKE, max_seqlen, None, None,
        batch, 32, window, 0.1, 0, None, FAKE, nbytes, None, None)
    assert st in (WORKSPACE, 4), st   # 4: valid, only the device is missing
    return st == WORKSPACE


def chosen(batch, max_seqlen, window):
    """The partitions (of 512, 1024 and 1536) whose workspace is just enough."""
    got = []
    for p in (512, 1024, 1536):
        need = pkv.paged_decode_workspace_size(batch, 32, 128, max_seqlen, p, window)
        if not asks_for(batch, max_seqlen, window, need) and \
                asks_for(batch, max_seqlen, window, need - 1):
            got.append(p)
    return got


@nogpu
@pytest.mark.parametrize("batch,max_seqlen,window,want", [
    (64, 4096, -1, 512), (8, 131072, -1, 1536), (128, 8192, -1, 1024),
    # the keys that a window leaves decide, not the sequences' lengths
    (64, 32768, 4095, 512), (16, 131072, 4095, 512), (128, 32768, 8191, 1024),
    (128, 32768, 16383, 1536), (8, 131072, 1 << 30, 1536), (8, 131072, (1 << 31) - 1, 1536),
    (64, 32768, 0, 512),
])
def test_partition(batch, max_seqlen, window, want):
    assert want in chosen(batch, max_seqlen, window)
