"""The paged calls at sizes whose launches would pass 2^32 threads in one
dimension, which no launch may."""
import pytest
import torch

from gpu_util import need_gpu
import indexer_top_kv_amd as ech

pytestmark = pytest.mark.gpu


def test_evict_in_place_of_wide_rows():
    """520 sequences of rows of 1 MiB, one wave column of 128 bytes each: 2^32
    threads and more. Token 1 is the heavier one and takes token 0's place."""
    need_gpu()
    B, width = 520, 1 << 18
    i32 = dict(dtype=torch.int32, device='cuda')
    pool = torch.arange(2 * B, **i32).view(-1, 1).expand(-1, width).contiguous()
    pool[:, -1] += 1 << 20
    table = torch.arange(2 * B, **i32).view(B, 2)
    acc = torch.tensor([[1.0, 2.0]], device='cuda').repeat(B, 1)
    n = torch.full((B,), 2, **i32)
    kept, n_out = torch.empty((B, 1), **i32), torch.empty(B, **i32)
    ech.ech_paged_evict(acc, n, 2, 1, 0, 0, kept, n_out, pool=pool, src_table=table, dst_table=table, page_size=1)
    want = (torch.arange(2 * B, **i32) | 1).view(-1, 1)
    assert torch.all(kept == 1) and torch.all(n_out == 1)
    assert torch.equal(pool[:, :-1], want.expand(-1, width - 1)) and torch.equal(pool[:, -1:], want + (1 << 20))
