"""The resident paged cache (ech_paged_append / _attn / _weight / _evict)
against the oracle.

Tolerances, derived from the arithmetic. A score is a sum of 576 exact bf16
products in fp32: it is off by at most d = 576 * 2^-24 * sum|q k| * scale, and
the base-2 argument and exponential add a few 2^-24 of its size, taken as
8 * 2^-24 * (1 + sum|q k| * scale). So a weight is off by a factor within
1 +- 2 (d + e) (its own score and the denominator's), and by a bf16 rounding,
2^-8, in the value product; sums over n tokens in fp32 add n * 2^-24. The
output is rounded to bf16, 2^-8 of itself. With a[c] = sum_t p_t |v_t[c]|:
    |out - ref| <= (2^-8 (1 + 2^-8) + 2 (d + e) + 2 n 2^-24) a + 2^-8 |ref|
    |lse - ref| <= d + e + n 2^-24 + 2^-23 |ref|
A received weight sums w_rh = exp(s - lse) over n (row, head) pairs, the lse
taken as given: |acc - ref| <= sum w (d + e) + n 2^-24 acc + 2^-23 |acc|.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle.numerics import bf16_to_f64
import workloads as wk
from gpu_util import dev, host, need_gpu
import indexer_top_kv_amd as ech

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(192.0)
U = 2.0 ** -24


class Case:
    """A batch: rows and context length per sequence, pages shuffled."""

    def __init__(self, rows, ctx, H, page, window=0, sink=0, seed=0, lead=0, tail=0, extra_pages=3, q_scale=1.0):
        r = self.r = np.random.default_rng(seed)
        self.B, self.H, self.page, self.window, self.sink = len(rows), H, page, window, sink
        self.row0 = (lead + np.concatenate([[0], np.cumsum(rows)])).astype(np.int32)
        self.T = int(self.row0[-1]) + tail
        self.rows = list(rows)
        self.seq_len = np.array([n + c for n, c in zip(rows, ctx)], np.int32)
        self.max_len = int(self.seq_len.max())
        npg = -(-max(self.max_len, 1) // page)
        n_pages = self.B * npg + extra_pages
        self.table = r.permutation(n_pages)[:self.B * npg].reshape(self.B, npg).astype(np.int32)
        self.n_slots = n_pages * page
        self.pool = wk.to_bf16_bits(r.standard_normal((self.n_slots, 576)).astype(np.float32))
        self.q = wk.to_bf16_bits((q_scale * r.standard_normal((self.T, H, 576))).astype(np.float32))

    @property
    def max_rows(self):
        return max(self.rows)

    def ws(self, fn, *a):
        n = fn(*a)
        return torch.full((n,), 0xff, dtype=torch.uint8, device='cuda') if n else None   # NaN patterns

    def attn(self, q=None, pool=None, table=None, out=None, lse=None, stream=None, ws=None, scale=SCALE):
        out = torch.full((self.T, self.H, 512), 7.0, dtype=torch.bfloat16, device='cuda') if out is None else out
        lse = torch.full((self.T, self.H), 7.0, dtype=torch.float32, device='cuda') if lse is None else lse
        ws = self.ws(ech.ech_paged_attn_ws_bytes, self.B, self.T, self.H, self.max_rows, self.max_len, self.window,
                     self.sink) if ws is None else ws
        ech.ech_paged_attn(dev(self.q) if q is None else q, dev(self.pool) if pool is None else pool,
                           dev(self.table) if table is None else table, self.page, dev(self.row0), dev(self.seq_len),
                           self.max_rows, self.max_len, scale, out, lse, window=self.window, n_sink=self.sink, ws=ws,
                           stream=stream)
        torch.cuda.synchronize()
        return out.float().cpu().numpy(), lse.cpu().numpy()

    def ref(self, table=None, pool=None, scale=SCALE):
        return oracle.paged.attention(self.q, self.pool if pool is None else pool,
                                      self.table if table is None else table, self.page, self.row0, self.seq_len,
                                      scale, self.window, self.sink)

    def weight(self, lse, acc_in, decay, acc_out=None, q=None):
        acc_out = torch.full((self.B, acc_in.shape[1]), 7.0, dtype=torch.float32, device='cuda') if acc_out is None else acc_out
        ws = self.ws(ech.ech_paged_weight_ws_bytes, self.B, self.T, self.H, self.max_rows, self.max_len)
        ech.ech_paged_weight(dev(self.q) if q is None else q, dev(lse), dev(self.pool), dev(self.table), self.page,
                             dev(self.row0), dev(self.seq_len), self.max_rows, self.max_len, SCALE,
                             acc_in if isinstance(acc_in, torch.Tensor) else dev(acc_in), acc_out, decay=decay,
                             window=self.window, n_sink=self.sink, ws=ws)
        torch.cuda.synchronize()
        return acc_out.cpu().numpy()


def check_attn(got, ref, n, tag=''):
    out, lse = got
    o, l, a, mag = ref
    mine = ~np.isnan(l)
    assert np.all(out[~mine] == 7.0) and np.all(lse[~mine] == 7.0), f'{tag}: rows of no sequence were written'
    de = 576 * U * mag + 8 * U * (1 + mag)
    bound = (2.0 ** -8 * (1 + 2.0 ** -8) + 2 * de + 2 * n * U)[..., None] * a + 2.0 ** -8 * np.abs(o)
    err = np.abs(out - o)
    bad = mine[..., None] & ~(err <= bound)
    assert not bad.any(), (tag, int(bad.sum()), float(np.nanmax(np.where(bad, err / np.maximum(bound, 1e-30), 0))),
                           np.argwhere(bad)[:4].tolist())
    empty = mine & np.isneginf(l)
    assert np.all(out[empty] == 0) and np.all(np.isneginf(lse[empty])), tag
    fin = mine & np.isfinite(l)
    assert np.all(np.abs(lse[fin] - l[fin]) <= (de + n * U)[fin] + 2 * U * np.abs(l[fin])), tag


SHAPES = [
    # rows, ctx, H, page, window, sink
    ([1], [0], 1, 1, 0, 0),                                   # one token, nothing before it
    ([1], [0], 16, 64, 0, 0),
    ([1], [999], 16, 64, 0, 0),
    ([1, 1, 1], [30, 31, 32], 128, 16, 0, 0),                 # around a step's end
    ([1, 0, 1, 0], [5, 100, 700, 0], 32, 7, 0, 0),            # sequences without new rows
    ([5, 1, 33], [0, 64, 130], 24, 24, 0, 0),                 # tiles that span rows, odd heads
    ([130], [0], 1, 1, 0, 0),                                 # a prompt's first chunk, one head
    ([9, 17], [100, 1], 128, 100, 0, 0),
    ([40], [1500], 8, 48, 0, 0),
    ([3], [2500], 5, 31, 0, 0),                               # few queries, many spans
    ([2, 1, 4], [4000, 10, 300], 16, 64, 0, 0),
    # windows and first tokens
    ([1], [1000], 16, 64, 128, 4),
    ([1, 1], [4000, 90], 64, 32, 100, 33),
    ([70], [200], 16, 16, 1, 0),                              # a row sees itself only
    ([64], [300], 4, 24, 17, 3),
    ([20, 3, 50], [500, 0, 40], 16, 24, 64, 64),
    ([33], [700], 32, 64, 31, 130),                           # more first tokens than the window
    ([200], [0], 2, 16, 50, 0),
    ([1], [2000], 128, 64, 4096, 4),                          # a window longer than the sequence
]


@pytest.mark.parametrize('rows,ctx,H,page,window,sink', SHAPES)
def test_attention_against_oracle(rows, ctx, H, page, window, sink):
    need_gpu()
    c = Case(rows, ctx, H, page, window, sink, seed=sum(rows) * 7 + H)
    check_attn(c.attn(), c.ref(), c.max_len, f'{rows} {ctx}')


def test_attention_rows_of_no_sequence():
    """Rows before the first and behind the last sequence stay as they were,
    with and without spans."""
    need_gpu()
    for ctx in (40, 1500):
        c = Case([2, 1], [ctx, 3], 16, 16, seed=3, lead=2, tail=3)
        check_attn(c.attn(), c.ref(), c.max_len)


def test_attention_absent_pages():
    """Negative and too large table entries, and the pool's end inside a page:
    those tokens are absent; a sequence without any page sees nothing."""
    need_gpu()
    c = Case([3, 1, 2], [200, 90, 1000], 16, 16, seed=4)
    t = c.table.copy()
    t[0, 2] = -1
    t[0, 5] = 2 ** 31 - 1
    t[1, :] = -7
    t[2, 60] = c.n_slots // 16
    check_attn(c.attn(table=dev(t)), c.ref(table=t), c.max_len, 'absent')
    pool = c.pool[:c.n_slots - 5]                       # the last page ends early
    t = c.table.copy()
    t[0, 1] = c.n_slots // 16 - 1
    check_attn(c.attn(table=dev(t), pool=dev(pool)), c.ref(table=t, pool=pool), c.max_len, 'short pool')


def test_attention_lengths_beyond_the_table():
    """More rows than tokens (their positions are negative: they see nothing)."""
    need_gpu()
    c = Case([6, 2], [0, 50], 16, 8, seed=5)
    c.seq_len[0] = 3
    check_attn(c.attn(), c.ref(), c.max_len)


@pytest.mark.parametrize('window,sink', [(0, 0), (20, 2)])
def test_attention_infinities_and_nan_out_of_sight(window, sink):
    """Slots that no query sees hold NaN and infinities (free pages, the end of
    the last page, slot 0); later tokens of the same chunk hold them too: only
    the rows that see them are not finite."""
    need_gpu()
    c = Case([70, 1], [45, 333], 2, 16, window, sink, seed=6)
    used = np.zeros(c.n_slots, bool)
    for b in range(c.B):
        used[oracle.paged.slots(c.table[b], 16, c.n_slots, int(c.seq_len[b]))] = True
    clean = c.pool.copy()
    junk = np.array([0x7f80, 0xff80, 0x7fc0, 0xffff], np.uint16)
    c.pool[~used] = junk[c.r.integers(0, 4, (int((~used).sum()), 576))]
    check_attn(c.attn(), c.ref(pool=clean), c.max_len, 'free slots')
    bad_t = 45 + 50                                     # a token of the chunk, seen by rows from position 95 on
    s = oracle.paged.slots(c.table[0], 16, c.n_slots, int(c.seq_len[0]))[bad_t]
    for what in (0x7fc0, 0x7f80):
        c.pool[s, 100:103] = what
        out, lse = c.attn()
        o, l, a, mag = c.ref(pool=clean)
        p = 45 + np.arange(70)
        hit = np.zeros(c.T, bool)
        hit[:70] = (p >= bad_t) & ((window == 0) | (bad_t > p - window))
        if what == 0x7fc0:
            assert not np.isfinite(out[hit]).all(axis=(1, 2)).any()
        out[hit], lse[hit] = 7.0, 7.0
        for x in (o, l, a, mag):
            x[hit] = np.nan
        check_attn((out, lse), (o, l, a, mag), c.max_len, hex(what))


def test_attention_peaked_and_flat():
    need_gpu()
    c = Case([4, 1], [300, 2000], 16, 64, seed=7, q_scale=6.0)
    check_attn(c.attn(scale=0.5), c.ref(scale=0.5), c.max_len, 'peaked')
    c.q[:] = 0
    check_attn(c.attn(), c.ref(), c.max_len, 'flat')
    # the maximum grows through the sequence, step by step
    c = Case([3], [900], 16, 64, seed=8)
    f = wk.to_bf16_bits(np.ones(576, np.float32))
    c.q[:] = f
    sl = oracle.paged.slots(c.table[0], 64, c.n_slots, int(c.seq_len[0]))
    c.pool[sl] = wk.to_bf16_bits((np.linspace(-3, 3, len(sl))[:, None] * np.ones(576)).astype(np.float32))
    check_attn(c.attn(), c.ref(), c.max_len, 'growing')


def test_attention_strided_queries_and_equal_values():
    """q as a view into a larger tensor (rows and heads strided) gives the bits
    of a dense q; the order of pages does not matter to the result's bits."""
    need_gpu()
    c = Case([5, 1], [130, 1500], 16, 16, seed=9)
    o1, l1 = c.attn()
    big = torch.zeros((c.T, c.H, 1024), dtype=torch.int16, device='cuda')
    big[:, :, 64:640] = dev(c.q)
    o2, l2 = c.attn(q=big[:, :, 64:640])
    np.testing.assert_array_equal(o1, o2)
    np.testing.assert_array_equal(l1, l2)
    byhead = dev(c.q).transpose(0, 1).contiguous().transpose(0, 1)
    o2, l2 = c.attn(q=byhead)
    np.testing.assert_array_equal(o1, o2)
    # another placement of the same rows
    perm = c.r.permutation(c.n_slots // 16)
    pool = c.pool.reshape(-1, 16 * 576)[np.argsort(perm)].reshape(-1, 576)
    o2, l2 = c.attn(pool=dev(pool), table=dev(perm[c.table].astype(np.int32)))
    np.testing.assert_array_equal(o1, o2)
    np.testing.assert_array_equal(l1, l2)


def test_attention_shared_pages():
    """Two sequences read the same prompt pages."""
    need_gpu()
    c = Case([1, 2], [640, 650], 16, 64, seed=10)
    c.table[1, :10] = c.table[0, :10]
    check_attn(c.attn(), c.ref(), c.max_len)


def test_attention_through_sel_slot_is_sparse_attention():
    """page_size 1 with sel_slot as the table: the attention of ech_sparse_attn."""
    need_gpu()
    r = np.random.default_rng(12)
    B, H, k, C = 3, 64, 512, 2000
    q = wk.to_bf16_bits(r.standard_normal((B, H, 576)).astype(np.float32))
    cache = wk.to_bf16_bits(r.standard_normal((C, 576)).astype(np.float32))
    sel = np.stack([r.choice(C, k, replace=False) for _ in range(B)]).astype(np.int32)
    sel[1, 400:] = -1
    out = torch.zeros((B, H, 512), dtype=torch.bfloat16, device='cuda')
    lse = torch.zeros((B, H), dtype=torch.float32, device='cuda')
    row0 = dev(np.arange(B + 1, dtype=np.int32))
    n = dev(np.full(B, k, np.int32))
    ws = torch.empty(ech.ech_paged_attn_ws_bytes(B, B, H, 1, k), dtype=torch.uint8, device='cuda')
    ech.ech_paged_attn(dev(q), dev(cache), dev(sel), 1, row0, n, 1, k, SCALE, out, lse, ws=ws)
    o, l = oracle.sparse_attention(q, cache, sel, SCALE)
    ref = oracle.paged.attention(q, cache, sel, 1, np.arange(B + 1), np.full(B, k), SCALE)
    np.testing.assert_allclose(ref[0], o, rtol=1e-12, atol=1e-14)
    check_attn((out.float().cpu().numpy(), host(lse)), ref, k)


def test_attention_beyond_32_bit_offsets():
    """Slots whose byte offset passes 2^32 (and 2^31 values)."""
    need_gpu()
    page, n_pages = 64, 60000                            # 3.84M rows, 4.4 GB
    pool = torch.zeros((n_pages * page, 576), dtype=torch.bfloat16, device='cuda')
    r = np.random.default_rng(13)
    pages = np.array([[n_pages - 1, 0, n_pages - 2, n_pages // 2, n_pages - 3]], np.int32)
    n, H, rows = 300, 16, 3
    x = wk.to_bf16_bits(r.standard_normal((n, 576)).astype(np.float32))
    small = np.zeros((5 * page, 576), np.uint16)
    small[:n] = x
    bits = pool.view(torch.int16)
    seq_len, row0 = dev(np.array([n], np.int32)), dev(np.array([0, n], np.int32))
    ech.ech_paged_append(bits, dev(pages), page, row0, seq_len, dev(x))
    for j in range(5):
        got = host(bits[int(pages[0, j]) * page:(int(pages[0, j]) + 1) * page]).view(np.uint16)
        np.testing.assert_array_equal(got, small[j * page:(j + 1) * page])
    q = wk.to_bf16_bits(r.standard_normal((rows, H, 576)).astype(np.float32))
    out = torch.zeros((rows, H, 512), dtype=torch.bfloat16, device='cuda')
    lse = torch.zeros((rows, H), dtype=torch.float32, device='cuda')
    ws = torch.empty(ech.ech_paged_attn_ws_bytes(1, rows, H, rows, n), dtype=torch.uint8, device='cuda')
    r0 = np.array([0, rows], np.int32)
    ech.ech_paged_attn(dev(q), pool, dev(pages), page, dev(r0), seq_len, rows, n, SCALE, out, lse, ws=ws)
    ref = oracle.paged.attention(q, small, np.arange(5)[None], page, r0, np.array([n]), SCALE)
    check_attn((out.float().cpu().numpy(), host(lse)), ref, n)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize('rows,ctx,page,lead,tail', [([1], [0], 1, 0, 0), ([1] * 70, list(range(70)), 16, 0, 0),
                                                     ([130, 0, 1, 7], [5, 9, 63, 64], 24, 3, 5)])
def test_append(rows, ctx, page, lead, tail):
    need_gpu()
    c = Case(rows, ctx, 1, page, seed=20 + page, lead=lead, tail=tail)
    x = c.r.integers(0, 2 ** 16, (c.T, 576)).astype(np.uint16)
    want = c.pool.copy()
    oracle.paged.append(want, c.table, page, c.row0, c.seq_len, x)
    pool = dev(c.pool)
    status = torch.zeros(1, dtype=torch.int32, device='cuda')
    ech.ech_paged_append(pool, dev(c.table), page, dev(c.row0), dev(c.seq_len), dev(x), status)
    np.testing.assert_array_equal(host(pool).view(np.uint16), want)
    assert int(status.item()) == 0
    # rows as a strided view, a pool of another row width and type
    wide = torch.zeros((c.T, 600), dtype=torch.int16, device='cuda')
    wide[:, 24:] = dev(x)
    pool = dev(c.pool)
    ech.ech_paged_append(pool, dev(c.table), page, dev(c.row0), dev(c.seq_len), wide[:, 24:])
    np.testing.assert_array_equal(host(pool).view(np.uint16), want)
    p8 = torch.zeros((c.n_slots, 16), dtype=torch.uint8, device='cuda')
    x8 = torch.randint(0, 256, (c.T, 16), dtype=torch.uint8, device='cuda')
    ech.ech_paged_append(p8, dev(c.table), page, dev(c.row0), dev(c.seq_len), x8)
    want8 = np.zeros((c.n_slots, 16), np.uint8)
    oracle.paged.append(want8, c.table, page, c.row0, c.seq_len, host(x8))
    np.testing.assert_array_equal(host(p8), want8)


def test_append_without_pages():
    """Positions without a page, past the table, and negative ones: not
    written, flagged; the others land."""
    need_gpu()
    c = Case([4, 6, 2], [30, 0, 0], 1, 8, seed=23)
    t = c.table.copy()
    t[0, 4] = -1                          # positions 32, 33 of sequence 0
    c.seq_len[1] = 4                      # two rows at negative positions
    c.seq_len[2] = t.shape[1] * 8 + 1     # one past the table
    x = c.r.integers(0, 2 ** 16, (c.T, 576)).astype(np.uint16)
    want = c.pool.copy()
    assert oracle.paged.append(want, t, 8, c.row0, c.seq_len, x)
    pool = dev(c.pool)
    status = torch.zeros(1, dtype=torch.int32, device='cuda')
    ech.ech_paged_append(pool, dev(t), 8, dev(c.row0), dev(c.seq_len), dev(x), status)
    np.testing.assert_array_equal(host(pool).view(np.uint16), want)
    assert int(status.item()) == ech.ST_FULL


# ------------------------------------------------------------------ received weight
def weight_bound(c, ref, acc_in, decay, mag):
    de = 576 * U * mag + 8 * U * (1 + mag)
    got = ref - acc_in * float(np.float32(decay))
    n = c.max_rows * c.H
    return got * de.max(initial=0) * 1.01 + n * U * np.abs(got) + 2 * U * (np.abs(ref) + np.abs(acc_in)) + 1e-30


@pytest.mark.parametrize('rows,ctx,H,page,window,sink', SHAPES)
def test_weight_against_oracle(rows, ctx, H, page, window, sink):
    need_gpu()
    c = Case(rows, ctx, H, page, window, sink, seed=31 + sum(rows) + H)
    _, lse, _, mag = c.ref()
    lse32 = lse.astype(np.float32)
    acc_in = c.r.random((c.B, c.max_len + 5)).astype(np.float32)
    got = c.weight(lse32, acc_in, 0.75)
    ref = oracle.paged.received(c.q, lse32, c.pool, c.table, page, c.row0, c.seq_len, SCALE, acc_in, 0.75, window, sink)
    bound = weight_bound(c, ref, acc_in, 0.75, mag[~np.isnan(mag)])
    for b in range(c.B):
        n = int(c.seq_len[b])
        err = np.abs(got[b, :n] - ref[b, :n])
        assert np.all(err <= bound[b, :n]), (b, float((err / bound[b, :n]).max()))
        assert np.all(got[b, n:] == 7.0), 'entries past the length were written'
    # each (row, head) that sees something hands out 1
    total = sum(int(np.isfinite(lse[c.row0[b]:c.row0[b + 1]]).sum()) for b in range(c.B))
    zero = c.weight(lse32, np.zeros_like(acc_in), 1.0)
    s = sum(float(zero[b, :int(c.seq_len[b])].sum(dtype=np.float64)) for b in range(c.B))
    assert abs(s - total) <= 1e-3 * max(total, 1)


def test_weight_in_place_absent_pages_and_nan():
    """acc_out is acc_in; tokens without a page receive nothing; NaN in rows
    out of sight does not spread; the same call gives the same bits."""
    need_gpu()
    c = Case([9, 1], [300, 77], 16, 16, 40, 3, seed=33)
    t0 = c.table.copy()
    c.table[0, 18] = -1
    _, lse, _, mag = c.ref()
    lse32 = lse.astype(np.float32)
    acc_in = c.r.random((c.B, c.max_len)).astype(np.float32)
    ref = oracle.paged.received(c.q, lse32, c.pool, c.table, 16, c.row0, c.seq_len, SCALE, acc_in, 1.0, 40, 3)
    bound = weight_bound(c, ref, acc_in, 1.0, mag)
    unseen = oracle.paged.slots(t0[0], 16, c.n_slots, 309)[100]          # between the first tokens and every window
    c.pool[unseen] = 0x7fc0
    a = dev(acc_in)
    got = c.weight(lse32, a, 1.0, acc_out=a)
    again = c.weight(lse32, acc_in, 1.0)
    for b in range(c.B):
        n = int(c.seq_len[b])
        assert np.all(np.abs(got[b, :n] - ref[b, :n]) <= bound[b, :n])
        np.testing.assert_array_equal(got[b, :n], again[b, :n])


# ------------------------------------------------------------------ eviction
def run_evict(acc, lens, keep, sink, recent, pool=None, src=None, dst=None, page=1, in_place=False, len_in_place=None):
    B, L = acc.shape
    kept = torch.full((B, keep), -9, dtype=torch.int32, device='cuda')
    a = dev(acc)
    n = dev(lens)
    ao = a if in_place else torch.full_like(a, 5.0)
    lo = n if (in_place if len_in_place is None else len_in_place) else torch.full_like(n, -3)
    nb = ech.ech_paged_evict_ws_bytes(B, L, keep)
    ws = torch.full((nb,), 0xff, dtype=torch.uint8, device='cuda') if nb else None
    ech.ech_paged_evict(a, n, L, keep, sink, recent, kept, lo, acc_out=ao, pool=pool, src_table=src, dst_table=dst,
                        page_size=page, ws=ws)
    torch.cuda.synchronize()
    return host(kept), host(lo), host(ao)


def check_evict(got, acc, lens, keep, sink, recent):
    kept, lo, ao = got
    for b, ref in enumerate(oracle.paged.evict(acc, lens, keep, sink, recent)):
        assert lo[b] == len(ref)
        np.testing.assert_array_equal(kept[b, :len(ref)], ref, err_msg=f'sequence {b}')
        assert np.all(kept[b, len(ref):] == -1)
        np.testing.assert_array_equal(ao[b, :len(ref)], acc[b, ref])
        assert np.all(ao[b, len(ref):] == 0)


EVICT = [
    # lens, keep, sink, recent
    ([1], 1, 0, 0), ([0, 5, 3], 4, 0, 0), ([2], 1, 1, 0), ([2], 1, 0, 1), ([100, 64, 65], 64, 4, 16),
    ([1000, 1025, 3, 700], 512, 4, 100), ([5000], 17, 0, 0), ([5000, 4999], 4000, 1000, 1500),
    ([20011], 9001, 16, 512), ([300], 200, 100, 100), ([70000, 131], 4096, 4, 0), ([16384, 16385], 8192, 0, 0),
    ([4096, 4097, 1], 1, 0, 0), ([24577, 8191, 8193], 30000, 9, 9), ([24577, 8191, 8193], 8192, 8000, 100),
]


@pytest.mark.parametrize('lens,keep,sink,recent', EVICT)
@pytest.mark.parametrize('kind', ['spread', 'ties', 'zeros', 'odd'])
def test_evict_selection(lens, keep, sink, recent, kind):
    need_gpu()
    r = np.random.default_rng(sum(lens) + keep)
    lens = np.array(lens, np.int32)
    shape = (len(lens), max(int(lens.max()), 1) + 3)
    if kind == 'spread':
        acc = np.exp(3 * r.standard_normal(shape))
    elif kind == 'ties':
        acc = r.integers(0, 4, shape) * 0.25
    elif kind == 'zeros':
        acc = np.where(r.random(shape) < 0.95, 0.0, r.random(shape)) * np.where(r.random(shape) < 0.5, 1, -1)
    else:
        acc = r.standard_normal(shape)
        acc[r.random(shape) < 0.1] = np.inf
        acc[r.random(shape) < 0.1] = -np.inf
        acc[r.random(shape) < 0.05] = np.nan
        acc[r.random(shape) < 0.05] = -np.nan
    acc = acc.astype(np.float32)
    check_evict(run_evict(acc, lens, keep, sink, recent), acc, lens, keep, sink, recent)
    check_evict(run_evict(acc, lens, keep, sink, recent, in_place=True), acc, lens, keep, sink, recent)
    if max(lens) > 16384:                  # blocks of a long row: each output in place by itself
        check_evict(run_evict(acc, lens, keep, sink, recent, in_place=True, len_in_place=False), acc, lens, keep, sink, recent)
        check_evict(run_evict(acc, lens, keep, sink, recent, len_in_place=True), acc, lens, keep, sink, recent)


@pytest.mark.parametrize('page,row', [(1, 576), (16, 576), (24, 576), (100, 24)])
@pytest.mark.parametrize('within', [False, True])
def test_evict_moves_rows(page, row, within):
    """Kept rows land in the destination's pages (or move together in place);
    every other slot keeps its bytes."""
    need_gpu()
    r = np.random.default_rng(page + row)
    lens = np.array([700, 300, 0, 513], np.int32)
    keep, B, L = 300, 4, 700
    npg = -(-L // page)
    n_pages = 2 * B * npg + 2
    perm = r.permutation(n_pages).astype(np.int32)
    src = perm[:B * npg].reshape(B, npg)
    dst = src if within else perm[B * npg:2 * B * npg].reshape(B, npg).copy()
    pool = r.integers(0, 2 ** 16, (n_pages * page, row)).astype(np.uint16)
    acc = r.random((B, L)).astype(np.float32)
    want = pool.copy()
    for b, ref in enumerate(oracle.paged.evict(acc, lens, keep, 4, 50)):
        s = oracle.paged.slots(src[b], page, len(pool), L)[ref]
        d = oracle.paged.slots(dst[b], page, len(pool), len(ref))
        want[d] = pool[s]
    p, st = dev(pool), dev(src)
    got = run_evict(acc, lens, keep, 4, 50, pool=p, src=st, dst=st if within else dev(dst), page=page)
    check_evict(got, acc, lens, keep, 4, 50)
    np.testing.assert_array_equal(host(p).view(np.uint16), want)


# ------------------------------------------------------------------ streams, graphs, refusals
def test_other_stream_and_captured_replays():
    """A captured append + attention + weight follows lengths, rows and pages
    that change in place; every replay equals the eager calls, with eager work
    between the replays. And the calls run on a stream that is not current."""
    need_gpu()
    c = Case([1, 1, 1], [400, 1200, 33], 16, 16, seed=40)
    npg = c.table.shape[1] + 2
    table = dev(np.resize(c.r.permutation(3 * npg), (3, npg)).astype(np.int32))
    pool = dev(wk.to_bf16_bits(c.r.standard_normal((3 * npg * 16, 576)).astype(np.float32)))
    q, row0, n = dev(c.q), dev(c.row0), dev(c.seq_len)
    x = dev(wk.to_bf16_bits(c.r.standard_normal((3, 576)).astype(np.float32)))
    cap = c.max_len + 16
    out = torch.zeros((3, 16, 512), dtype=torch.bfloat16, device='cuda')
    lse = torch.zeros((3, 16), dtype=torch.float32, device='cuda')
    acc = torch.zeros((3, cap), dtype=torch.float32, device='cuda')
    ws = torch.empty(max(16, ech.ech_paged_attn_ws_bytes(3, 3, 16, 1, cap)), dtype=torch.uint8, device='cuda')
    ww = torch.empty(max(16, ech.ech_paged_weight_ws_bytes(3, 3, 16, 1, cap)), dtype=torch.uint8, device='cuda')

    def step(p, o, l, a, stream=None):
        ech.ech_paged_append(p, table, 16, row0, n, x, stream=stream)
        ech.ech_paged_attn(q, p, table, 16, row0, n, 1, cap, SCALE, o, l, ws=ws, stream=stream)
        ech.ech_paged_weight(q, l, p, table, 16, row0, n, 1, cap, SCALE, a, a, decay=0.5, ws=ww, stream=stream)

    step(pool.clone(), out, lse, acc.clone())
    torch.cuda.synchronize()
    p_g, a_g = pool.clone(), acc.clone()
    p_e, a_e, o_e, l_e = pool.clone(), acc.clone(), torch.zeros_like(out), torch.zeros_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(p_g, out, lse, a_g)
    side = torch.cuda.Stream()
    for i in range(4):
        n.add_(1 if i else 0)
        x.copy_(dev(wk.to_bf16_bits(c.r.standard_normal((3, 576)).astype(np.float32))))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        step(p_e, o_e, l_e, a_e, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(p_g, p_e) and torch.equal(out, o_e) and torch.equal(lse, l_e) and torch.equal(a_g, a_e), i
        y = torch.arange(4096, device='cuda', dtype=torch.float32)
        assert float((y * 2).sum().item()) == 4096 * 4095


def test_refusals_on_the_gpu():
    need_gpu()
    c = Case([1], [100], 16, 16, seed=41)
    with pytest.raises(ech.EchError):       # a workspace too small
        c.attn(ws=torch.empty(8, dtype=torch.uint8, device='cuda')) if ech.ech_paged_attn_ws_bytes(
            1, 1, 16, 1, c.max_len) else (_ for _ in ()).throw(ech.EchError('none needed', -1))
    with pytest.raises(ValueError):         # q's innermost values must be dense
        c.attn(q=dev(c.q).repeat(1, 1, 2)[:, :, ::2])
    with pytest.raises(ech.EchError):       # head stride not a multiple of 8
        big = torch.zeros((1, 16, 580), dtype=torch.int16, device='cuda')
        c.attn(q=big[:, :, :576])
    with pytest.raises(TypeError):
        c.attn(pool=dev(c.pool).to(torch.float16))
    with pytest.raises(ValueError):
        c.attn(table=dev(c.table).expand(2, -1))
    with pytest.raises(ech.EchError):
        c.attn(scale=float('nan'))


def test_a_workspace_too_small_is_refused_on_the_gpu():
    """Every call that needs a workspace at these sizes refuses one that is a
    byte short, missing or not aligned, and leaves its outputs as they were."""
    need_gpu()
    c = Case([1], [1000], 16, 16, seed=41)
    need = ech.ech_paged_attn_ws_bytes(1, 1, 16, 1, c.max_len)
    assert need > 8
    out = torch.full((1, 16, 512), 7.0, dtype=torch.bfloat16, device='cuda')
    lse = torch.full((1, 16), 7.0, dtype=torch.float32, device='cuda')
    room = torch.empty(need + 256, dtype=torch.uint8, device='cuda')
    for ws in (room[:8], room[:need - 1], room[16:16 + need]):
        with pytest.raises(ech.EchError):
            c.attn(out=out, lse=lse, ws=ws)
    args = (dev(c.pool).view(torch.int16), dev(c.table), c.page, dev(c.row0), dev(c.seq_len), 1, c.max_len, SCALE)
    with pytest.raises(ech.EchError):
        ech.ech_paged_attn(dev(c.q), *args, out, lse)
    torch.cuda.synchronize()
    assert torch.all(out == 7.0) and torch.all(lse == 7.0)
    c.attn(out=out, lse=lse, ws=room[:need])
    assert not torch.any(out == 7.0)
    # received weight of a chunk, in parts; eviction of a long row
    T, ml = 512, 200
    q = torch.zeros((T, 16, 576), dtype=torch.bfloat16, device='cuda')
    need = ech.ech_paged_weight_ws_bytes(1, T, 16, T, ml)
    assert need > 8
    acc = torch.full((1, ml), 7.0, device='cuda')
    for ws in (None, room[:8], torch.empty(need - 1, dtype=torch.uint8, device='cuda')):
        with pytest.raises(ech.EchError):
            ech.ech_paged_weight(q, torch.zeros((T, 16), device='cuda'), dev(c.pool), dev(c.table), c.page,
                                 torch.tensor([0, T], dtype=torch.int32, device='cuda'), dev(c.seq_len), T, ml, SCALE, None,
                                 acc, ws=ws)
    n, keep = 20000, 64
    need = ech.ech_paged_evict_ws_bytes(1, n, keep)
    assert need > 8
    w = torch.zeros((1, n), device='cuda')
    kept, n_out = (torch.full(s, 7, dtype=torch.int32, device='cuda') for s in ((1, keep), (1,)))
    for ws in (None, room[:8], torch.empty(need - 1, dtype=torch.uint8, device='cuda')):
        with pytest.raises(ech.EchError):
            ech.ech_paged_evict(w, torch.tensor([n], dtype=torch.int32, device='cuda'), n, keep, 0, 0, kept, n_out, ws=ws)
    torch.cuda.synchronize()
    assert torch.all(acc == 7.0) and torch.all(kept == 7) and torch.all(n_out == 7)


def inf_case(rows, ctx, H, page, window, sink, seed, one):
    """Infinities in rows that some queries see and others do not, in few value
    columns or behind them, and in slots that none sees (slot 0 among them): a
    score of +inf or NaN makes all of a query's output NaN, one of -inf a weight
    of 0, whose product with an infinite value is NaN in that column alone."""
    c = Case(rows, ctx, H, page, window, sink, seed=seed)
    used = np.zeros(c.n_slots, bool)
    for b in range(c.B):
        sl = oracle.paged.slots(c.table[b], page, c.n_slots, int(c.seq_len[b]))
        used[sl] = True
        n, own = int(c.seq_len[b]), c.rows[b]
        # cached tokens, and some of the sequence's own rows
        at = np.unique(np.concatenate([c.r.integers(0, n, 2), n - 1 - c.r.integers(0, max(own, 1), 2)]))
        for t in at[-1:] if one else at:
            cols = c.r.integers(0, 500, 1) if one else c.r.integers(0, 576, 2)
            c.pool[sl[t], cols] = c.r.choice(np.array([0x7f80, 0xff80], np.uint16))
    c.pool[~used] = 0x7fc0
    return c


@pytest.mark.parametrize('rows,ctx,H,page,window,sink', [
    ([40], [300], 2, 16, 0, 0), ([70, 33], [45, 333], 4, 16, 0, 0), ([70, 33], [45, 333], 4, 16, 20, 3),
    ([1, 1, 1], [77, 1000, 40], 16, 24, 0, 0), ([1, 1], [500, 2001], 32, 16, 0, 0), ([2, 1, 2], [90, 700, 63], 16, 16, 30, 2),
    ([3], [50], 8, 16, 0, 0), ([1], [3000], 128, 16, 0, 0), ([300], [10], 128, 16, 0, 0)])
def test_attention_infinities_in_sight(rows, ctx, H, page, window, sink):
    need_gpu()
    whole = columns = 0
    for seed in range(8):
        c = inf_case(rows, ctx, H, page, window, sink, seed, one=seed >= 4)
        with np.errstate(invalid='ignore'):
            o, l, _, _ = c.ref()
        out, lse = c.attn()
        assert np.array_equal(np.isnan(out), np.isnan(o)), seed
        assert np.array_equal(np.isnan(lse), np.isnan(l)) and np.isfinite(l[~np.isnan(l)]).all(), seed
        # the columns that are finite: the bound of check_attn with the largest finite value and products
        clean = np.where((c.pool & 0x7f80) == 0x7f80, np.uint16(0), c.pool)
        de = np.max(c.ref(pool=clean)[3]) * 576 * U
        de += 8 * U * (1 + de / (576 * U))
        vmax, fin = np.abs(bf16_to_f64(clean[:, :512])).max(), np.isfinite(o)
        bound = (2.0 ** -8 * (1 + 2.0 ** -8) + 2 * de + 2 * c.max_len * U) * vmax + 2.0 ** -8 * np.abs(o[fin])
        assert np.all(np.abs(out[fin] - o[fin]) <= bound), seed
        fin = np.isfinite(l)
        assert np.all(np.abs(lse[fin] - l[fin]) <= de + c.max_len * U + 2 * U * np.abs(l[fin])), seed
        whole += int(np.isnan(o).all(axis=2).sum())
        columns += int((np.isnan(o).any(axis=2) & ~np.isnan(o).all(axis=2)).sum())
    assert whole and columns


@pytest.mark.parametrize('H,rows', [(16, 1), (128, 1), (16, 5)])
def test_attention_spans_whose_scores_are_all_minus_infinity(H, rows):
    """Tokens 0 .. 1999 hold -inf in value column 5, where every query is
    positive: whole spans of a split sequence weigh nothing, and column 5 is NaN
    by their 0 x -inf. A sequence of nothing else: out 0 (NaN in that column),
    lse -inf."""
    need_gpu()
    c = Case([rows, rows], [2500, 300], H, 16, seed=7)
    c.q[..., 5] = 0x3f80
    for b, n in ((0, 2000), (1, 300 + rows)):
        c.pool[oracle.paged.slots(c.table[b], 16, c.n_slots, n), 5] = 0xff80
    with np.errstate(invalid='ignore'):
        o, l, a, mag = c.ref()
    clean = np.where((c.pool & 0x7f80) == 0x7f80, np.uint16(0), c.pool)
    out, lse = c.attn()
    first, second = slice(0, rows), slice(rows, 2 * rows)
    assert np.isnan(out[first, :, 5]).all() and np.isnan(o[first, :, 5]).all()
    rest = np.arange(512) != 5
    assert np.array_equal(np.isnan(out[first][..., rest]), np.isnan(o[first][..., rest])) and np.isfinite(l[first]).all()
    mag = c.ref(pool=clean)[3]
    for x in (o, a, out):                   # check_attn takes NaN in lse for rows of no sequence
        x[first, :, 5] = 0.0
    check_attn((out[first], lse[first]), (o[first], l[first], a[first], mag[first]), c.max_len)
    assert np.isnan(out[second, :, 5]).all() and np.all(out[second][..., rest] == 0) and np.all(np.isneginf(lse[second]))


@pytest.mark.parametrize('rows,ctx,H,page,window,sink', [
    ([1, 1, 1], [77, 1000, 40], 16, 24, 0, 0), ([2, 1, 2], [90, 700, 63], 16, 16, 30, 2), ([70, 33], [45, 333], 4, 16, 0, 0),
    ([70, 33], [45, 333], 4, 16, 20, 3), ([1], [3000], 128, 16, 0, 0)])
def test_weight_infinities_in_sight(rows, ctx, H, page, window, sink):
    """Sums are NaN where the formula's are: tokens that a row with an lse of NaN
    sees, or one with scores of -inf alone; a single score of -inf adds nothing."""
    need_gpu()
    for seed in range(4, 8):
        c = inf_case(rows, ctx, H, page, window, sink, seed, one=True)
        if seed == 7:                       # a sequence whose scores are all -inf
            c.q[:rows[0], :, 5] = 0x3f80
            c.pool[oracle.paged.slots(c.table[0], page, c.n_slots, int(c.seq_len[0])), 5] = 0xff80
        out, lse = c.attn()
        if seed == 7:
            assert np.isneginf(lse[:rows[0]]).any()
        acc = np.ones((c.B, c.max_len), np.float32)
        with np.errstate(invalid='ignore'):
            ref = oracle.paged.received(c.q, lse, c.pool, c.table, page, c.row0, c.seq_len, SCALE, acc, 0.5, window, sink)
        got = c.weight(lse, acc, 0.5)
        for b, n in enumerate(c.seq_len):
            assert np.array_equal(np.isnan(got[b, :n]), np.isnan(ref[b, :n])), (seed, b)
