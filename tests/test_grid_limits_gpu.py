"""Batches beyond what a grid holds are refused before a launch: the number of
CTAs was an int32 that wrapped around.  (The plans are real, the buffers small:
nothing may be launched.)"""
import numpy as np
import pytest
import torch

from test_kv4_gpu import binding

pytestmark = pytest.mark.gpu

UNSUPPORTED = 2


def test_eviction_of_more_rows_than_a_grid_holds():
    b = binding()
    batch, Hkv = 1 << 20, 1 << 12                       # 2^32 rows: 0 in 32 bits
    zeros, table = np.zeros(batch + 1, dtype=np.int32), torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = b.Plan(zeros, zeros, table, zeros[:batch], Hkv, Hkv, 64, 16, num_pages=1)
    p = torch.zeros(1024, dtype=torch.uint8, device="cuda").data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    for call in ("attn_evict_kv", "attn_evict_kv4"):
        for out in (p, None):
            status = getattr(b.load_library(), call)(plan.handle, p, p, 4, 1, p, out, 1, p, p, stream)
            assert status == UNSUPPORTED, call


def test_key_weights_of_more_tiles_than_a_grid_holds():
    b = binding()
    pages, Hkv, batch = 1 << 16, 1 << 12, 8            # 8 x 65536 tiles of 128 keys, times 4096 heads: 2^31
    qo, kv = np.arange(batch + 1, dtype=np.int32) * 2, np.arange(batch + 1, dtype=np.int32) * pages
    table = torch.zeros(batch * pages, dtype=torch.int32, device="cuda")
    plan = b.Plan(qo, kv, table, np.full(batch, 128, dtype=np.int32), Hkv, Hkv, 64, 128, num_pages=1)
    p = torch.zeros(1024, dtype=torch.uint8, device="cuda").data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    lib = b.load_library()
    assert lib.attn_key_weights(plan.handle, p, p, p, None, 0.0, 0, p, stream) == UNSUPPORTED
    assert lib.attn_key_weights_kv4(plan.handle, p, p, 1.0, p, None, 0.0, 0, p, stream) == UNSUPPORTED
