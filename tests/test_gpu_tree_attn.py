"""Attention of drafted rows that form trees (ech_paged_tree_attn) against the
oracle. Tolerances are those of test_gpu_paged.py: the arithmetic is the same,
only the set of tokens differs."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, need_gpu
import indexer_top_kv_amd as ech
from test_gpu_paged import SCALE, Case, check_attn

pytestmark = pytest.mark.gpu


def trees(kind, rows, seed):
    """Parents of every sequence's rows, one after another."""
    r = np.random.default_rng(seed)
    out = []
    for n in rows:
        for i in range(n):
            if i == 0:
                out.append(-1)
            elif kind == 'random':
                out.append(int(r.integers(0, i)))
            elif kind == 'chain':
                out.append(i - 1)
            elif kind == 'star':
                out.append(0)
            elif kind == 'forest':                     # several rows follow the cached tokens
                out.append(int(r.integers(-1, i)))
            elif kind == 'binary':
                out.append((i - 1) // 2)
    return np.array(out, np.int32).reshape(-1)


class TreeCase(Case):
    def __init__(self, rows, ctx, H, page, window=0, sink=0, kind='random', **kw):
        super().__init__(rows, ctx, H, page, window, sink, **kw)
        lead = int(self.row0[0])
        self.parent = np.concatenate([np.full(lead, 5, np.int32), trees(kind, rows, kw.get('seed', 0) + 1),
                                      np.full(self.T - int(self.row0[-1]), -7, np.int32)])

    def attn(self, q=None, pool=None, table=None, out=None, lse=None, stream=None, ws=None, scale=SCALE, parent=None):
        out = torch.full((self.T, self.H, 512), 7.0, dtype=torch.bfloat16, device='cuda') if out is None else out
        lse = torch.full((self.T, self.H), 7.0, dtype=torch.float32, device='cuda') if lse is None else lse
        ws = self.ws(ech.ech_paged_tree_attn_ws_bytes, self.B, self.T, self.H, self.max_rows, self.max_len, self.window,
                     self.sink) if ws is None else ws
        ech.ech_paged_tree_attn(dev(self.q) if q is None else q, dev(self.pool) if pool is None else pool,
                                dev(self.table) if table is None else table, self.page, dev(self.row0),
                                dev(self.seq_len), dev(self.parent if parent is None else parent), self.max_rows,
                                self.max_len, scale, out, lse, window=self.window, n_sink=self.sink, ws=ws,
                                stream=stream)
        torch.cuda.synchronize()
        return out.float().cpu().numpy(), lse.cpu().numpy()

    def ref(self, table=None, pool=None, scale=SCALE, parent=None):
        return oracle.drafts.attention(self.q, self.pool if pool is None else pool,
                                       self.table if table is None else table, self.page, self.row0, self.seq_len,
                                       self.parent if parent is None else parent, scale, self.window, self.sink)


SHAPES = [
    # rows, ctx, H, page, window, sink, kind
    ([1], [0], 1, 1, 0, 0, 'random'),
    ([1], [0], 16, 64, 0, 0, 'random'),
    ([8], [999], 16, 64, 0, 0, 'random'),
    ([2], [37], 16, 64, 0, 0, 'forest'),                        # at most 32 queries
    ([32], [100], 1, 16, 0, 0, 'random'),
    ([16], [63], 1, 7, 0, 0, 'forest'),
    ([5, 0, 3], [0, 31, 700], 4, 24, 0, 0, 'binary'),
    ([12, 1, 0, 7], [300, 2, 9, 65], 128, 16, 0, 0, 'random'),
    ([64], [500], 16, 64, 0, 0, 'random'),                      # a tree over several steps
    ([33, 65], [31, 1], 8, 24, 0, 0, 'forest'),
    ([256], [10], 1, 16, 0, 0, 'random'),                       # the largest tree
    ([256], [0], 2, 48, 0, 0, 'chain'),
    ([200, 100], [64, 77], 3, 1, 0, 0, 'star'),
    ([9], [4000], 32, 64, 0, 0, 'binary'),                      # split over spans
    ([3], [2500], 5, 31, 0, 0, 'star'),
    # windows and first tokens
    ([8], [1000], 2, 64, 128, 4, 'random'),
    ([24], [200], 1, 16, 3, 0, 'chain'),                        # a line longer than the window
    ([40, 17], [300, 5], 16, 24, 5, 9, 'random'),               # first tokens inside the tree
    ([64], [2], 4, 16, 4, 20, 'forest'),
    ([70], [0], 8, 16, 1, 0, 'binary'),                         # a row sees itself only
    ([16, 0, 5], [3000, 10, 90], 64, 32, 100, 33, 'random'),
    ([128], [700], 2, 64, 31, 130, 'random'),
    ([256], [300], 1, 24, 90, 2, 'chain'),
    ([6], [2000], 128, 64, 4096, 4, 'random'),                  # a window longer than the sequence
    # tiles of 128 queries: more than 256 of 32
    ([64, 60, 0, 64, 90], [100, 3, 9, 31, 200], 64, 16, 0, 0, 'random'),
    ([70, 64, 64], [500, 0, 64], 63, 24, 0, 0, 'forest'),
    ([256], [333], 40, 64, 0, 0, 'chain'),
    ([256], [31], 33, 7, 0, 0, 'binary'),
    ([100, 100], [700, 30], 64, 16, 90, 5, 'random'),
    ([250], [40], 48, 16, 30, 60, 'chain'),                     # first tokens inside the tree
    ([128, 80], [400, 64], 48, 24, 1, 0, 'random'),
    ([256, 200], [20, 150], 128, 16, 0, 0, 'random'),           # and more of these than CUs
    ([256, 200], [300, 50], 100, 64, 40, 3, 'forest'),
    # of 32, as many rounds as they are used for, and more
    ([16, 9, 16, 16], [3000, 3800, 3500, 2900], 16, 64, 0, 0, 'random'),
    ([16, 16, 16, 16, 16, 16, 16, 16], [6400] * 8, 16, 64, 0, 0, 'star'),
]


@pytest.mark.parametrize('rows,ctx,H,page,window,sink,kind', SHAPES)
def test_against_oracle(rows, ctx, H, page, window, sink, kind):
    need_gpu()
    c = TreeCase(rows, ctx, H, page, window, sink, kind, seed=sum(rows) * 7 + H)
    check_attn(c.attn(), c.ref(), c.max_len, f'{rows} {ctx} {kind}')


@pytest.mark.parametrize('rows,ctx,H,window,sink', [([12, 30], [500, 3], 16, 0, 0), ([7], [900], 4, 60, 5), ([50], [90], 32, 17, 3)])
def test_a_chain_is_the_causal_call(rows, ctx, H, window, sink):
    """Up to the order of sums: the two choose their forms by rules of their own."""
    need_gpu()
    c = TreeCase(rows, ctx, H, 16, window, sink, 'chain', seed=9)
    ref = Case.ref(c)
    check_attn(c.attn(), ref, c.max_len)
    check_attn(Case.attn(c), ref, c.max_len)


def test_rows_of_no_sequence_and_parents_that_are_none():
    """Rows before the first and behind the last sequence stay as they were;
    parents that do not precede their row count as none."""
    need_gpu()
    for ctx, H, more in ((40, 16, 0), (1500, 16, 0), (5, 1, 0), (50, 128, 80)):
        c = TreeCase([9, 4 + more], [ctx, 3], H, 16, seed=3, lead=2, tail=3)
        bad = c.parent.copy()
        bad[2:15] = [0, 1, 2, -5, 4, 2 ** 31 - 1, -2 ** 31, 300, 3, 0, 0, 2, 9]
        check_attn(c.attn(parent=bad), c.ref(parent=bad), c.max_len, f'{ctx}')


@pytest.mark.parametrize('rows,H', [([6], 4), ([40], 16), ([150], 64)])
def test_values_that_are_not_finite_outside_of_a_line(rows, H):
    """Infinities and NaN in rows of other branches, and in rows without a page,
    stay out of a row's output; in its own line they reach it."""
    need_gpu()
    c = TreeCase(rows, [50], H, 8, kind='binary', seed=4)
    at = oracle.paged.slots(c.table[0], 8, c.n_slots, int(c.seq_len[0]))
    pool = c.pool.copy()
    pool[at[50 + 2], 7], pool[at[50 + 4], 600 % 512] = 0x7f80, 0x7fc0        # rows 2 and 4
    out, lse = c.attn(pool=dev(pool))
    hit = [i for i in range(rows[0]) if {2, 4} & set(oracle.drafts.line(c.parent, i))]
    free = [i for i in range(rows[0]) if i not in hit]
    o, l, a, mag = c.ref(pool=np.where((pool & 0x7f80) == 0x7f80, 0, pool).astype(np.uint16))
    de = 576 * 2.0 ** -24 * mag + 8 * 2.0 ** -24 * (1 + mag)
    bound = (2.0 ** -8 * (1 + 2.0 ** -8) + 2 * de + 2 * c.max_len * 2.0 ** -24)[..., None] * a + 2.0 ** -8 * np.abs(o)
    assert len(hit) > 1 and len(free) > 1
    assert np.all(np.abs(out[free] - o[free]) <= bound[free])
    assert not np.isfinite(out[hit]).all(axis=(1, 2)).any()


@pytest.mark.parametrize('rows,H', [([20, 12], 16), ([100, 60], 60)])
def test_absent_pages_and_short_lengths(rows, H):
    """Nodes whose page is missing count as absent; a length below the number
    of rows leaves rows without a slot."""
    need_gpu()
    c = TreeCase(rows, [30, 40], H, 8, seed=6)
    table = c.table.copy()
    table[0, 4], table[0, 5], table[1, 2] = -1, c.n_slots, 2 ** 31 - 1
    check_attn(c.attn(table=dev(table)), c.ref(table=table), c.max_len)
    c.seq_len[:] = [7, 0]
    check_attn(c.attn(), c.ref(), c.max_len)


@pytest.mark.parametrize('rows,H', [([5], 4), ([9], 16), ([100], 128)])
def test_pages_behind_4_gib_of_pool(rows, H):
    """The cached rows and the tree at the end of a pool of more than 2^32 bytes."""
    need_gpu()
    c = TreeCase(rows, [70], H, 16, seed=8)
    n = 5 * 2 ** 30 // (16 * 1152)
    pool = torch.zeros((n * 16, 576), dtype=torch.int16, device='cuda')
    small = dev(c.pool)
    far = n - len(c.pool) // 16
    pool[far * 16:] = small
    check_attn(c.attn(pool=pool, table=dev(c.table + far)), c.ref(), c.max_len)


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    need_gpu()
    cs = [TreeCase([30, 12], [700, 40], 32, 16, seed=s) for s in (11, 12)]
    streams = [torch.cuda.Stream() for _ in cs]
    bufs = []
    for c in cs:
        bufs.append([dev(x) for x in (c.q, c.pool, c.table, c.row0, c.seq_len, c.parent)] + [
            torch.empty((c.T, c.H, 512), dtype=torch.bfloat16, device='cuda'), torch.empty((c.T, c.H), device='cuda'),
            c.ws(ech.ech_paged_tree_attn_ws_bytes, c.B, c.T, c.H, c.max_rows, c.max_len, 0, 0)])
    torch.cuda.synchronize()
    for _ in range(5):
        for c, b, s in zip(cs, bufs, streams):
            ech.ech_paged_tree_attn(b[0], b[1], b[2], c.page, b[3], b[4], b[5], c.max_rows, c.max_len, SCALE, b[6], b[7], ws=b[8],
                                    stream=s)
    torch.cuda.synchronize()
    for c, b in zip(cs, bufs):
        check_attn((b[6].float().cpu().numpy(), b[7].cpu().numpy()), c.ref(), c.max_len)


def test_strided_queries():
    """Rows and heads of a wider tensor."""
    need_gpu()
    for rows, H in (([12], 16), ([3], 8), ([200], 48)):
        c = TreeCase(rows, [100], H, 16, seed=13)
        wide = torch.full((c.T, H + 2, 640), float('nan'), dtype=torch.bfloat16, device='cuda')
        wide[:, 1:-1, 8:584] = dev(c.q).view(torch.bfloat16)
        check_attn(c.attn(q=wide[:, 1:-1, 8:584]), c.ref(), c.max_len)
