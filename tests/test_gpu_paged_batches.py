"""The resident paged cache in large, cut and concurrent batches: more
sequences than one plan covers, more tiles than CUs, more rows or tokens than
the bounds name, tables and lengths that are wrong, empty calls, two calls at
once. Tolerances as in test_gpu_paged.py."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wk
from gpu_util import dev, host, need_gpu
import indexer_top_kv_amd as ech
from test_gpu_paged import SCALE, Case, check_attn, weight_bound

pytestmark = pytest.mark.gpu


class Ragged(Case):
    """A batch whose sequences hold only the pages of their own lengths."""

    def __init__(self, rows, ctx, H, page, window=0, sink=0, seed=0, lead=0, tail=0):
        r = self.r = np.random.default_rng(seed)
        self.B, self.H, self.page, self.window, self.sink = len(rows), H, page, window, sink
        self.row0 = (lead + np.concatenate([[0], np.cumsum(rows)])).astype(np.int32)
        self.T = int(self.row0[-1]) + tail
        self.rows = list(rows)
        self.seq_len = np.array([n + c for n, c in zip(rows, ctx)], np.int32)
        self.max_len = int(self.seq_len.max())
        held = -(-self.seq_len // page)
        n_pages = int(held.sum()) + 2
        perm = r.permutation(n_pages)
        self.table = np.full((self.B, max(int(held.max()), 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.n_slots = n_pages * page
        self.pool = wk.to_bf16_bits(r.standard_normal((self.n_slots, 576)).astype(np.float32))
        self.q = wk.to_bf16_bits(r.standard_normal((self.T, H, 576)).astype(np.float32))


def check_both(c, decay=0.5):
    """Attention and received weight of a batch."""
    ref = c.ref()
    got = c.attn()
    check_attn(got, ref, c.max_len)
    lse32 = np.nan_to_num(ref[1], nan=0.0, neginf=-np.inf).astype(np.float32)
    acc_in = c.r.random((c.B, c.max_len + 1)).astype(np.float32)
    w = c.weight(lse32, acc_in, decay)
    want = oracle.paged.received(c.q, lse32, c.pool, c.table, c.page, c.row0, c.seq_len, SCALE, acc_in, decay, c.window,
                                 c.sink)
    mag = ref[3][~np.isnan(ref[3])]
    bound = weight_bound(c, want, acc_in, decay, mag)
    for b in range(c.B):
        n = int(c.seq_len[b])
        err = np.abs(w[b, :n] - want[b, :n])
        assert np.all(err <= bound[b, :n]), (b, float((err / bound[b, :n]).max()))
        assert np.all(w[b, n:] == 7.0)


def many(B, most, long_at=(), long=0, rows=(0, 1), seed=0):
    r = np.random.default_rng(seed)
    n = r.choice(rows, B)
    ctx = r.integers(0, most, B)
    for b in long_at:
        ctx[b] = long
    return n.tolist(), ctx.tolist()


@pytest.mark.parametrize('H,rows,window,sink', [(16, (0, 1), 0, 0), (16, (0, 1), 30, 3), (5, (0, 1, 3), 0, 0), (32, (1,), 0, 0),
                                                (32, (0, 1), 64, 0), (64, (0, 1, 2), 0, 0), (64, (0, 2), 20, 5),
                                                (40, (0, 1, 4), 0, 0), (40, (4,), 33, 1)])
def test_more_sequences_than_a_plan_covers(H, rows, window, sink):
    """B > 256: a tile (or sequence) per workgroup, single tokens and several.
    Two sequences are long, one of them maybe without new rows: their sums
    leave in more than one piece."""
    need_gpu()
    n, ctx = many(300, 90, (7, 299), 2500, rows, seed=H + window)
    n[7], n[299] = 0, max(rows)
    check_both(Ragged(n, ctx, H, 16, window, sink, seed=H, lead=1, tail=2))


@pytest.mark.parametrize('window,sink', [(0, 0), (100, 10)])
def test_more_tiles_than_cus(window, sink):
    """A tile per workgroup, the last first; a sequence without rows between."""
    need_gpu()
    check_both(Ragged([150, 0, 1, 121], [100, 300, 77, 260], 128, 48, window, sink, seed=window, tail=1))


@pytest.mark.parametrize('B', [255, 256, 257])
def test_around_the_plans_size(B):
    need_gpu()
    n, ctx = many(B, 200, (0,), 1500, (1,), seed=B)
    check_both(Ragged(n, ctx, 24, 32, seed=B))
    check_both(Ragged(n, ctx, 128, 32, seed=B))


@pytest.mark.parametrize('H', [4, 64])
def test_bounds_below_what_the_batch_holds(H):
    """Of a sequence with more than max_rows rows the first max_rows are
    computed, and lengths past max_len are cut there; nothing else is written."""
    need_gpu()
    c = Case([5, 2, 9], [200, 40, 90], H, 16, seed=H)
    for most in (3, 1):
        full = Case([5, 2, 9], [200, 40, 90], H, 16, seed=H)
        ref = [x.copy() for x in full.ref()]
        for b in range(3):
            for x in ref:
                x[c.row0[b] + most:c.row0[b + 1]] = np.nan
        c.rows = [most]
        check_attn(c.attn(), ref, c.max_len, f'max_rows {most}')
    c = Case([5, 2, 9], [200, 40, 90], H, 16, seed=H + 1)
    c.max_len = 70                               # sequences of 205, 42 and 99 tokens
    cut = np.minimum(c.seq_len, 70)
    ref = oracle.paged.attention(c.q, c.pool, c.table, 16, c.row0, cut, SCALE)
    check_attn(c.attn(), ref, 70)
    w = c.weight(np.nan_to_num(ref[1]).astype(np.float32), np.zeros((3, 300), np.float32), 1.0)
    for b in range(3):
        assert np.all(w[b, cut[b]:] == 7.0) and np.all(np.isfinite(w[b, :cut[b]]))


@pytest.mark.parametrize('H,rows', [(16, [2, 1, 1]), (128, [3, 1, 4]), (8, [1, 40, 3])])
def test_wrong_tables_and_lengths_stay_inside(H, rows):
    """Row offsets out of order and out of range, negative and huge lengths,
    pages far outside the pool: every call returns, and only the buffers' own
    places are written (a canary before and behind)."""
    need_gpu()
    c = Case(rows, [100, 0, 700], H, 16, seed=H)
    r = np.random.default_rng(H)
    i32 = np.iinfo(np.int32)
    for trial in range(4):
        row0 = r.choice([i32.min, -5, 0, 1, 2, c.T, c.T + 9, i32.max], 4).astype(np.int32)
        lens = r.choice([i32.min, -1, 0, 50, 700, i32.max], 3).astype(np.int32)
        table = np.where(r.random(c.table.shape) < 0.3, r.choice([i32.min, -1, i32.max, c.n_slots // 16], c.table.shape),
                         c.table).astype(np.int32)
        c.row0, c.seq_len = row0, lens
        out = torch.full((c.T + 2, H, 512), 7.0, dtype=torch.bfloat16, device='cuda')
        lse = torch.full((c.T + 2, H), 7.0, dtype=torch.float32, device='cuda')
        c.attn(table=dev(table), out=out[1:-1], lse=lse[1:-1])
        assert bool((out[0] == 7).all() and (out[-1] == 7).all() and (lse[0] == 7).all() and (lse[-1] == 7).all())
        t0, c.table = c.table, table
        acc = torch.full((5, c.max_len), 7.0, dtype=torch.float32, device='cuda')
        c.weight(np.zeros((c.T, H), np.float32), np.zeros((3, c.max_len), np.float32), 1.0, acc_out=acc[1:-1])
        assert bool((acc[0] == 7).all() and (acc[-1] == 7).all())
        pool = torch.full((c.n_slots + 2, 576), 7, dtype=torch.int16, device='cuda')
        x = torch.zeros((c.T, 576), dtype=torch.int16, device='cuda')
        ech.ech_paged_append(pool[1:-1], dev(table), 16, dev(row0), dev(lens), x)
        kept = torch.full((5, 40), -9, dtype=torch.int32, device='cuda')
        lo = torch.empty(3, dtype=torch.int32, device='cuda')
        a = torch.rand((3, c.max_len), device='cuda')
        tb = dev(table)
        ech.ech_paged_evict(a, dev(lens), c.max_len, 40, 3, 7, kept[1:-1], lo, acc_out=a, pool=pool[1:-1], src_table=tb,
                            dst_table=tb if trial % 2 else dev(c.r.permutation(table.reshape(-1)).reshape(table.shape)),
                            page_size=16)
        torch.cuda.synchronize()
        assert bool((kept[0] == -9).all() and (kept[-1] == -9).all())
        assert bool((pool[0] == 7).all() and (pool[-1] == 7).all())
        np.testing.assert_array_equal(host(lo), np.clip(lens.astype(np.int64), 0, 40))
        c.table = t0


def test_calls_with_nothing_to_do():
    """No rows at all: attention writes nothing, the weights only decay,
    acc_in None counts as zeros, an append does nothing."""
    need_gpu()
    c = Case([0, 0], [100, 33], 16, 16, 0, 0, seed=2)
    assert ech.ech_paged_attn_ws_bytes(2, 0, 16, 0, c.max_len) == 0
    c.attn()
    acc = c.r.random((2, 100)).astype(np.float32)
    for window in (0, 20):
        c.window = window
        got = c.weight(np.zeros((0, 16), np.float32), acc, 0.25)
        for b, n in enumerate(c.seq_len):
            np.testing.assert_array_equal(got[b, :n], acc[b, :n] * np.float32(0.25))
            assert np.all(got[b, n:] == 7.0)
        out = torch.full((2, 100), 7.0, dtype=torch.float32, device='cuda')
        ech.ech_paged_weight(torch.empty((0, 16, 576), dtype=torch.bfloat16, device='cuda'),
                             torch.empty((0, 16), device='cuda'), dev(c.pool), dev(c.table), 16, dev(c.row0),
                             dev(c.seq_len), 0, 100, SCALE, None, out, window=window)
        torch.cuda.synchronize()
        for b, n in enumerate(c.seq_len):
            assert bool((out[b, :n] == 0).all() and (out[b, n:] == 7).all())
    for H, rows in ((16, [1, 1]), (64, [40, 3])):       # acc_in None is a running sum of zeros, in both forms
        c = Case(rows, [200, 9], H, 16, seed=3)
        lse = np.nan_to_num(c.ref()[1]).astype(np.float32)
        want = c.weight(lse, np.zeros((2, c.max_len), np.float32), 1.0)
        out = torch.full((2, c.max_len), 7.0, dtype=torch.float32, device='cuda')
        ech.ech_paged_weight(dev(c.q), dev(lse), dev(c.pool), dev(c.table), 16, dev(c.row0), dev(c.seq_len), c.max_rows,
                             c.max_len, SCALE, None, out,
                             ws=c.ws(ech.ech_paged_weight_ws_bytes, 2, c.T, H, c.max_rows, c.max_len))
        np.testing.assert_array_equal(host(out), want)


def test_two_calls_at_once():
    """Two streams, a workspace each, shared inputs: both as alone."""
    need_gpu()
    c = Case([1, 1, 1], [3000, 700, 50], 16, 64, seed=8)
    d = Case([90, 3], [600, 30], 64, 24, seed=9)
    want = [x.attn() for x in (c, d)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args, outs = [], []
    for x in (c, d):
        args.append([dev(v) for v in (x.q, x.pool, x.table, x.row0, x.seq_len)])
        outs.append((torch.empty((x.T, x.H, 512), dtype=torch.bfloat16, device='cuda'),
                     torch.empty((x.T, x.H), device='cuda'),
                     x.ws(ech.ech_paged_attn_ws_bytes, x.B, x.T, x.H, x.max_rows, x.max_len)))
    torch.cuda.synchronize()
    for _ in range(8):
        for x, (q, pool, table, row0, lens), (o, l, ws), s in zip((c, d), args, outs, streams):
            ech.ech_paged_attn(q, pool, table, x.page, row0, lens, x.max_rows, x.max_len, SCALE, o, l, ws=ws, stream=s)
    torch.cuda.synchronize()
    for (o, l, _), (wo, wl) in zip(outs, want):
        np.testing.assert_array_equal(o.float().cpu().numpy(), wo)
        np.testing.assert_array_equal(host(l), wl)


def test_pages_of_the_largest_size_and_a_pool_that_ends_inside_one():
    need_gpu()
    c = Case([3], [400], 16, 16, seed=12)
    c.page, c.table = 1 << 20, np.array([[0]], np.int32)
    check_attn(c.attn(), c.ref(), c.max_len)             # the pool's rows end inside the page, behind the last token
    c.pool = c.pool[:200].copy()
    c.n_slots = 200                                      # and before it: tokens from 200 on are absent
    check_attn(c.attn(), c.ref(), c.max_len)


@pytest.mark.parametrize('L', [4096, 4097, 16384, 16385])
def test_evict_at_the_forms_ends_with_room_to_spare(L):
    """Rows of exactly a form's most tokens, and keep beyond max_len."""
    need_gpu()
    from test_gpu_paged import check_evict, run_evict
    r = np.random.default_rng(L)
    acc = r.random((2, L)).astype(np.float32)
    for keep, lens in ((L + 700, [L, L - 1]), (L - 1, [L, 5]), (1, [L, 1])):
        lens = np.array(lens, np.int32)
        check_evict(run_evict(acc, lens, keep, 0, 0), acc, lens, keep, 0, 0)
        check_evict(run_evict(acc, lens, keep, 0, 0, in_place=True), acc, lens, keep, 0, 0)


@pytest.mark.parametrize('T,H', [(1, 16), (1, 1), (7, 1)])
def test_strides_of_single_rows_and_heads_do_not_matter(T, H):
    """A dimension of one has no stride worth checking: a row or a head cut
    from a tensor whose rows or heads are oddly spaced."""
    need_gpu()
    c = Case([T], [300], H, 16, seed=T + H)
    want = c.attn()
    if T == 1:
        q = torch.as_strided(dev(c.q).view(torch.bfloat16), (1, H, 576), (1, 576, 1))
    else:
        q = torch.as_strided(dev(c.q).view(torch.bfloat16), (T, 1, 576), (576, 3, 1))
    got = c.attn(q=q)
    np.testing.assert_array_equal(got[0], want[0])
    acc = np.zeros((1, c.max_len), np.float32)
    np.testing.assert_array_equal(c.weight(want[1], acc, 1.0, q=q), c.weight(want[1], acc, 1.0))


@pytest.mark.parametrize('rows,ctx,H', [([1], [900], 16), ([1, 40], [10, 400], 64), ([300], [0], 128)])
def test_attention_without_lse(rows, ctx, H):
    need_gpu()
    c = Case(rows, ctx, H, 16, seed=H)
    want, _ = c.attn()
    out = torch.full((c.T, H, 512), 7.0, dtype=torch.bfloat16, device='cuda')
    ech.ech_paged_attn(dev(c.q), dev(c.pool), dev(c.table), 16, dev(c.row0), dev(c.seq_len), c.max_rows, c.max_len,
                       SCALE, out, ws=c.ws(ech.ech_paged_attn_ws_bytes, c.B, c.T, H, c.max_rows, c.max_len))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out.float().cpu().numpy(), want)


@pytest.mark.parametrize('scale', [0.0, -0.03])
def test_scales_of_zero_and_below(scale):
    need_gpu()
    for rows, H in (([2, 1], 16), ([20, 3], 64)):
        c = Case(rows, [300, 70], H, 16, seed=H)
        ref = c.ref(scale=scale)
        check_attn(c.attn(scale=scale), ref, c.max_len, f'scale {scale}')


def test_every_call_beyond_32_bit_offsets():
    """Pages behind the pool's first 4 GiB give what the same pages of a small
    pool give."""
    need_gpu()
    page, n_pages = 64, 65600                    # 4.2M rows, 4.8 GB
    r = np.random.default_rng(77)
    big = torch.zeros((n_pages * page, 576), dtype=torch.int16, device='cuda')
    base = n_pages - 60
    for rows, H in (([1, 3], 16), ([40, 7], 64)):
        c = Case(rows, [500, 90], H, page, seed=H, extra_pages=0)
        n_tab = c.table.size                     # the small pool's second half takes the moved rows
        c.pool, c.n_slots = np.concatenate([c.pool, np.zeros_like(c.pool)]), 2 * c.n_slots
        assert n_tab * page * 2 == c.n_slots
        x = dev(wk.to_bf16_bits(r.standard_normal((c.T, 576)).astype(np.float32)).view(np.int16))
        lse = torch.zeros((c.T, H), device='cuda')
        got = []
        for pool, first in ((dev(c.pool.view(np.int16)), 0), (big, base)):
            table = dev(c.table + first)
            if first:
                big[first * page:first * page + c.n_slots] = dev(c.pool.view(np.int16))
            ech.ech_paged_append(pool, table, page, dev(c.row0), dev(c.seq_len), x)
            acc = torch.zeros((2, c.max_len), device='cuda')
            ech.ech_paged_weight(dev(c.q), lse, pool, table, page, dev(c.row0), dev(c.seq_len), c.max_rows, c.max_len,
                                 SCALE, None, acc, ws=c.ws(ech.ech_paged_weight_ws_bytes, 2, c.T, H, c.max_rows, c.max_len))
            n, kept, lo = dev(c.seq_len), torch.empty((2, 200), dtype=torch.int32, device='cuda'), torch.empty_like(dev(c.seq_len))
            ech.ech_paged_evict(acc, n, c.max_len, 200, 4, 30, kept, lo, pool=pool, src_table=table,
                                dst_table=table + n_tab, page_size=page)      # to the pages behind
            ech.ech_paged_evict(acc, n, c.max_len, 200, 4, 30, kept, n, pool=pool, src_table=table, dst_table=table,
                                page_size=page)                                                  # and in place
            torch.cuda.synchronize()
            got.append((host(acc), host(kept), pool[first * page:first * page + c.n_slots].clone()))
        for small, large in zip(*got):
            assert np.array_equal(small, large) if isinstance(small, np.ndarray) else torch.equal(small, large)


def test_captured_chunks_and_evictions_share_a_workspace():
    """Two graphs, of chunks under no limit and under a window, with one
    workspace between them, each ending in an eviction (rows of one workgroup
    and long rows, in place and to other pages): replayed in turn, with eager
    work between, every replay equals the eager calls."""
    need_gpu()
    sides = []
    for k, (rows, ctx, H, window, L) in enumerate((([70, 5], [900, 30], 64, 0, 1000), ([40, 9], [300, 600], 128, 100, 20000))):
        c = Case(rows, ctx, H, 16, window, 4, seed=50 + k)
        c.pool = np.concatenate([c.pool, c.pool])
        t = dict(q=dev(c.q), table=dev(c.table), far=dev(c.table + len(c.pool) // 32), row0=dev(c.row0), n=dev(c.seq_len),
                 pool=dev(c.pool.view(np.int16)), pool0=dev(c.pool.view(np.int16)),
                 acc0=torch.rand((2, L), device='cuda'), acc=torch.empty((2, L), device='cuda'),
                 out=torch.zeros((c.T, H, 512), dtype=torch.bfloat16, device='cuda'), lse=torch.zeros((c.T, H), device='cuda'),
                 kept=torch.empty((2, 200), dtype=torch.int32, device='cuda'), lens=torch.empty(2, dtype=torch.int32, device='cuda'))
        sides.append((c, t, L))
    need = [max(ech.ech_paged_attn_ws_bytes(c.B, c.T, c.H, c.max_rows, L, c.window, c.sink),
                ech.ech_paged_weight_ws_bytes(c.B, c.T, c.H, c.max_rows, L), ech.ech_paged_evict_ws_bytes(c.B, L, 200))
            for c, _, L in sides]
    ws = torch.full((max(need),), 0xff, dtype=torch.uint8, device='cuda')

    def step(c, t, L):
        t['pool'].copy_(t['pool0'])
        t['acc'].copy_(t['acc0'])
        ech.ech_paged_attn(t['q'], t['pool'], t['table'], 16, t['row0'], t['n'], c.max_rows, L, SCALE, t['out'], t['lse'],
                           window=c.window, n_sink=c.sink, ws=ws)
        ech.ech_paged_weight(t['q'], t['lse'], t['pool'], t['table'], 16, t['row0'], t['n'], c.max_rows, L, SCALE, t['acc'],
                             t['acc'], decay=0.5, window=c.window, n_sink=c.sink, ws=ws)
        ech.ech_paged_evict(t['acc'], t['n'], L, 200, 4, 50, t['kept'], t['lens'], acc_out=t['acc'], pool=t['pool'],
                            src_table=t['table'], dst_table=t['table'] if c.window else t['far'], page_size=16, ws=ws)

    names = ('out', 'lse', 'acc', 'kept', 'lens', 'pool')
    want, graphs = [], []
    for c, t, L in sides:
        step(c, t, L)
        torch.cuda.synchronize()
        want.append({k: t[k].clone() for k in names})
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(c, t, L)
        graphs.append(g)
    for i in range(5):
        for (c, t, L), w, g in zip(sides, want, graphs):
            for k in names:
                t[k].zero_()
            g.replay()
            torch.cuda.synchronize()
            for k in names:
                a, b = t[k], w[k]
                if k == 'acc':          # what lies behind the sequences is the caller's
                    a, b = a[:, :200], b[:, :200]
                assert torch.equal(a, b), (i, k)
            y = torch.arange(4096, device='cuda', dtype=torch.float32)
            assert float((y * 2).sum().item()) == 4096 * 4095
