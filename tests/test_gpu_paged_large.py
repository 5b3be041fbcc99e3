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


def test_append_of_many_rows():
    """2^26 rows and a few: a wave each would be 2^32 threads and more. The last
    rows belong to a sequence whose pages are in descending order."""
    need_gpu()
    T, few, page = (1 << 26) + 37, 29, 1 << 20
    i32 = dict(dtype=torch.int32, device='cuda')
    n_pg = -(-(T - few) // page)
    rows = torch.arange(T, **i32).view(-1, 1) * torch.tensor([1, 3, 5, 7], **i32)
    pool = torch.full(((n_pg + 1) * page, 4), -1, **i32)
    table = torch.full((2, n_pg), -1, **i32)
    table[0, 0] = n_pg
    table[1] = torch.arange(n_pg - 1, -1, -1, **i32)
    row0, n = torch.tensor([0, few, T], **i32), torch.tensor([few, T - few], **i32)
    status = torch.zeros(1, **i32)
    ech.ech_paged_append(pool, table, page, row0, n, rows, status)
    assert int(status.item()) == 0
    assert torch.equal(pool[n_pg * page:n_pg * page + few], rows[:few]) and torch.all(pool[n_pg * page + few:] == -1)
    for j in range(n_pg):
        at, mine = (n_pg - 1 - j) * page, rows[few + j * page:few + (j + 1) * page]
        assert torch.equal(pool[at:at + len(mine)], mine), j
        assert torch.all(pool[at + len(mine):at + page] == -1)
