"""The accepted rows' move (ech_paged_accept) and copies of pages
(ech_paged_copy): rows go where they belong bit for bit, and nothing else
changes."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, need_gpu
import indexer_top_kv_amd as ech

pytestmark = pytest.mark.gpu


class Batch:
    def __init__(self, rows, ctx, page, width=576, seed=0, dtype=np.int16):
        r = self.r = np.random.default_rng(seed)
        self.B, self.page, self.rows = len(rows), page, list(rows)
        self.row0 = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.seq_len = np.array([n + c for n, c in zip(rows, ctx)], np.int32)
        self.max_len = int(self.seq_len.max())
        npg = -(-max(self.max_len, 1) // page)
        self.table = r.permutation(self.B * npg + 3)[:self.B * npg].reshape(self.B, npg).astype(np.int32)
        self.pool = r.integers(-30000, 30000, ((self.B * npg + 3) * page, width)).astype(dtype)
        self.kept = [sorted(r.choice(n, int(r.integers(0, n + 1)), replace=False).tolist()) if n else [] for n in rows]
        self.most = max([1] + [len(k) for k in self.kept])

    def run(self, pool=None, in_place=False, kept=None, n_kept=None, max_rows=None, max_len=None):
        pool = dev(self.pool) if pool is None else pool
        lens = dev(self.seq_len)
        out = lens if in_place else torch.full_like(lens, -5)
        if kept is None:
            kept = np.full((self.B, self.most), -1, np.int32)
            for b, x in enumerate(self.kept):
                kept[b, :len(x)] = x
        ech.ech_paged_accept(pool, dev(self.table), self.page, dev(self.row0), lens, dev(kept),
                             dev(np.array([len(x) for x in self.kept], np.int32) if n_kept is None else n_kept),
                             max(self.rows) if max_rows is None else max_rows, self.max_len if max_len is None else max_len, out)
        torch.cuda.synchronize()
        return pool.cpu().numpy(), out.cpu().numpy()


SHAPES = [
    # rows, ctx, page, width
    ([1], [0], 1, 576),
    ([8], [999], 64, 576),
    ([5, 0, 3, 1], [0, 12, 7, 100], 4, 576),
    ([60] * 9, [700 + 5 * i for i in range(9)], 24, 576),
    ([256, 255], [3, 64], 16, 576),
    ([17, 9], [30, 31], 1, 8),                                  # one piece a row
    ([12, 30], [5, 6], 7, 576 * 5),                             # rows of more pieces than a workgroup has threads
    ([2] * 1000, [3] * 1000, 2, 64),
]


@pytest.mark.parametrize('in_place', [False, True])
@pytest.mark.parametrize('rows,ctx,page,width', SHAPES)
def test_accept_against_oracle(rows, ctx, page, width, in_place):
    need_gpu()
    c = Batch(rows, ctx, page, width, seed=sum(rows) + page)
    want = c.pool.copy()
    lens = oracle.drafts.accept(want, c.table, page, c.row0, c.seq_len, c.kept)
    got, out = c.run(in_place=in_place)
    np.testing.assert_array_equal(out, lens)
    np.testing.assert_array_equal(got, want)


def test_accept_cuts_what_is_not_the_steps():
    """Counts beyond the rows and the list are cut; rows past the last, negative
    ones, rows that would move on, and rows without a page stay."""
    need_gpu()
    c = Batch([6, 6, 6, 6], [10, 10, 10, 10], 4, seed=3)
    c.table[3, 3] = -1                                          # tokens 12 .. 15 of the last
    c.most = 4
    kept = np.array([[0, 2, 9, 5], [-7, 3, 2 ** 31 - 1, -2 ** 31], [1, 1, 2, 3], [0, 2, 4, 5]], np.int32)
    got, out = c.run(kept=kept, n_kept=np.array([99, 2, -3, 4], np.int32))
    want = c.pool.copy()
    at = [oracle.paged.slots(c.table[b], 4, len(want), 16) for b in range(4)]
    src = c.pool.copy()
    want[at[0][11]], want[at[0][13]] = src[at[0][12]], src[at[0][15]]
    want[at[1][11]] = src[at[1][13]]
    np.testing.assert_array_equal(out, [14, 12, 10, 14])
    np.testing.assert_array_equal(got, want)                    # of the last: 12 to 11, 14 to 12, 15 to 13: no page on a side
    # lengths cut at the host's bound and at the table; fewer rows than the offsets say
    _, out = c.run(max_len=12, kept=kept, n_kept=np.array([1, 2, 0, 0], np.int32))
    np.testing.assert_array_equal(out, [7, 8, 6, 6])
    _, out = c.run(max_rows=1, kept=kept, n_kept=np.array([4, 4, 4, 4], np.int32))
    np.testing.assert_array_equal(out, [11, 11, 11, 11])
    c.seq_len[:] = [2, 0, 6, -4]
    got, out = c.run(kept=kept, n_kept=np.array([1, 0, 3, 2], np.int32))
    np.testing.assert_array_equal(out, [0, 0, 3, 0])
    np.testing.assert_array_equal(got[at[0]], c.pool[at[0]])


@pytest.mark.parametrize('page,width,dtype', [(64, 576, np.int16), (1, 576, np.int16), (24, 8, np.int16), (7, 600, np.int16),
                                              (100, 4, np.int32), (3, 5000, np.int16)])
@pytest.mark.parametrize('partial', [False, True])
def test_copy(page, width, dtype, partial):
    need_gpu()
    for n in (1, 5, 40):
        r = np.random.default_rng(n + page)
        pool = r.integers(-30000, 30000, (100 * page, width)).astype(dtype)
        perm = r.permutation(100).astype(np.int32)
        src, dst = perm[:n], perm[50:50 + n]
        if n > 1:
            src[1] = src[0]                                     # one page copied twice
        rows = r.integers(-1, page + 3, n).astype(np.int32) if partial else None
        want = pool.copy()
        for i in range(n):
            k = page if rows is None else min(max(int(rows[i]), 0), page)
            want[dst[i] * page:dst[i] * page + k] = pool[src[i] * page:src[i] * page + k]
        p = dev(pool)
        ech.ech_paged_copy(p, page, dev(src), dev(dst), None if rows is None else dev(rows))
        torch.cuda.synchronize()
        np.testing.assert_array_equal(p.cpu().numpy(), want)


def test_copy_pages_that_are_none():
    """Pages outside the pool are not copied; the page that its end cuts, up to there."""
    need_gpu()
    r = np.random.default_rng(1)
    pool = r.integers(-30000, 30000, (10 * 8 + 3, 16)).astype(np.int16)
    src = np.array([0, -1, 11, 10, 2 ** 31 - 1, 3, -2 ** 31, 5], np.int32)
    dst = np.array([11, 1, 2, 4, 6, -1, 7, 10], np.int32)
    p = dev(pool)
    ech.ech_paged_copy(p, 8, dev(src), dev(dst))
    torch.cuda.synchronize()
    want = pool.copy()
    want[32:35], want[80:83] = pool[80:83], pool[40:43]
    np.testing.assert_array_equal(p.cpu().numpy(), want)
    ech.ech_paged_copy(p, 8, dev(src[:0]), dev(dst[:0]))


def test_copies_behind_4_gib_of_pool():
    need_gpu()
    page, width = 64, 576
    n_pages = (5 << 30) // (page * width * 2)
    pool = torch.zeros((n_pages * page, width), dtype=torch.int16, device='cuda')
    pool[-page:] = torch.arange(page, dtype=torch.int16, device='cuda').view(-1, 1)
    src, dst = (torch.tensor(x, dtype=torch.int32, device='cuda') for x in ([n_pages - 1, n_pages - 1], [0, n_pages - 3]))
    ech.ech_paged_copy(pool, page, src, dst)
    assert torch.equal(pool[:page], pool[-page:]) and torch.equal(pool[-3 * page:-2 * page], pool[-page:])
    table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32, device='cuda')
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device='cuda')  # noqa: E731
    ech.ech_paged_accept(pool, table, page, i32([0, 70]), i32([100]), i32([[3, 69]]), i32([2]), 70, 128, i32([0]))
    assert int(pool[-page + 30, 5]) == 33 and int(pool[-page + 31, 5]) == 99 - 64


def test_accept_and_copy_in_a_graph():
    """Captured, replayed several times on new contents, against the eager calls."""
    need_gpu()
    c = Batch([12, 9, 30], [40, 50, 3], 16, seed=4)
    k = np.full((c.B, c.most), -1, np.int32)
    for b, x in enumerate(c.kept):
        k[b, :len(x)] = x
    t = [dev(x) for x in (c.table, c.row0, c.seq_len, k, np.array([len(x) for x in c.kept], np.int32))]
    free = [p for p in range(len(c.pool) // 16) if p not in set(c.table.reshape(-1).tolist())]
    src, dst = dev(c.table[:, 0].copy()), dev(np.array(free[:3], np.int32))
    pool, out = dev(c.pool), torch.zeros_like(t[2])

    def calls():
        ech.ech_paged_accept(pool, t[0], 16, t[1], t[2], t[3], t[4], 30, c.max_len, out)
        ech.ech_paged_copy(pool, 16, src, dst)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        calls()
    for rep in range(4):
        fresh = torch.randint(-30000, 30000, pool.shape, dtype=torch.int16, device='cuda')
        pool.copy_(fresh)
        calls()
        torch.cuda.synchronize()
        want = pool.clone()
        pool.copy_(fresh)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool, want) and not torch.equal(pool, fresh)
        assert out.tolist() == [int(n) - r + len(x) for n, r, x in zip(c.seq_len, c.rows, c.kept)]
