"""PagedLayer: append, attention, received weight and eviction as a model's
layer calls them, step after step, against the oracle run the same way: the
oracle keeps each sequence's rows as a plain list. Tolerances as in
test_gpu_paged.py; the kept tokens have to be exactly those that the layer's own
weights rank first."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wk
from gpu_util import dev, host, need_gpu
from indexer_top_kv_amd.pipeline import PagedLayer
from test_gpu_paged import U, check_attn

pytestmark = pytest.mark.gpu
SCALE = 1.0 / np.sqrt(192.0)


class Model:
    """The oracle's side: rows of every sequence in order, and their weights."""

    def __init__(self, B):
        self.rows = [np.zeros((0, 576), np.uint16) for _ in range(B)]

    def dense(self):
        """(pool, table, lengths) with one page per sequence."""
        n = max(max(len(r) for r in self.rows), 1)
        pool = np.zeros((len(self.rows) * n, 576), np.uint16)
        for b, r in enumerate(self.rows):
            pool[b * n:b * n + len(r)] = r
        return pool, np.arange(len(self.rows))[:, None], n, np.array([len(r) for r in self.rows])


def run(layer, steps, seed, window, sink):
    r = np.random.default_rng(seed)
    B, H = layer.B, layer.H
    m = Model(B)
    acc = np.zeros((B, layer.max_len))
    slack_err = np.zeros((B, layer.max_len))
    trimmed = 0
    for i, counts in enumerate(steps):
        T = sum(counts)
        q = wk.to_bf16_bits(r.standard_normal((T, H, 576)).astype(np.float32))
        x = wk.to_bf16_bits(r.standard_normal((T, 576)).astype(np.float32))
        row0 = np.concatenate([[0], np.cumsum(counts)])
        Tn = layer.place(counts)
        assert Tn == T
        out, lse = layer.launch(dev(q).view(torch.bfloat16), dev(x).view(torch.bfloat16))
        got = out.float().cpu().numpy(), host(lse)
        for b in range(B):
            m.rows[b] = np.concatenate([m.rows[b], x[row0[b]:row0[b + 1]]])
        pool, table, page, lens = m.dense()
        assert np.array_equal(lens, layer.lens)
        ref = oracle.paged.attention(q, pool, table, page, row0, lens, SCALE, window, sink)
        check_attn(got, ref, int(lens.max()), f'step {i}')
        if layer.budget is None:
            continue
        L = layer.max_len
        acc = oracle.paged.received(q, got[1], pool, table, page, row0, lens, SCALE, acc, layer.decay, window, sink)
        mag = ref[3].max() if T else 0.0
        de = 576 * U * mag + 8 * U * (1 + mag)
        slack_err = slack_err * layer.decay + acc * (de * 1.01 + (layer.max_rows * H + 4) * U) + 1e-30
        a_gpu = host(layer.acc)
        for b in range(B):
            assert np.all(np.abs(a_gpu[b, :lens[b]] - acc[b, :lens[b]]) <= slack_err[b, :lens[b]]), f'step {i}'
        if layer.trim():
            trimmed += 1
            torch.cuda.synchronize()
            kept = oracle.paged.evict(a_gpu, lens, layer.budget, layer.n_sink, layer.n_recent)
            new_acc, new_err = np.zeros((B, L)), np.zeros((B, L))
            for b in range(B):
                n = len(kept[b])
                np.testing.assert_array_equal(host(layer.kept)[b, :n], kept[b])
                m.rows[b] = m.rows[b][kept[b]]
                new_acc[b, :n], new_err[b, :n] = acc[b, kept[b]], slack_err[b, kept[b]]
            acc, slack_err = new_acc, new_err
            np.testing.assert_array_equal(host(layer.seq_len), [len(k) for k in kept])
        held = layer.pages.need(layer.lens)
        assert np.array_equal(held, layer.pages.held)
        assert len(layer.pages.free) == layer.pages.n_pages - held.sum()
    assert int(layer.status.item()) == 0
    return trimmed


STEPS = [[40, 0, 7], [1, 90, 1], [0, 0, 33], [1, 1, 1], [64, 1, 0], [1, 1, 1], [1, 1, 100], [1, 1, 1], [1, 1, 1]]


@pytest.mark.parametrize('page,window,sink', [(16, 0, 0), (24, 50, 4), (1, 0, 0)])
def test_steps_without_a_budget(page, window, sink):
    need_gpu()
    layer = PagedLayer(3, 16, n_pages=3 * (-(-260 // page)), max_len=260, max_rows=100, page_size=page, window=window,
                       n_sink=sink)
    run(layer, STEPS, 1, window, sink)


@pytest.mark.parametrize('page,window,H,slack', [(16, 0, 16, 0), (7, 0, 4, 10), (16, 40, 2, 0), (64, 0, 64, 0)])
def test_steps_with_a_budget(page, window, H, slack):
    need_gpu()
    layer = PagedLayer(3, H, n_pages=3 * (-(-200 // page)), max_len=200, max_rows=100, page_size=page, window=window,
                       n_sink=3, budget=60, n_recent=20, slack=slack, decay=0.9)
    assert run(layer, STEPS, 2 + page, window, 3) >= 2


def test_captured_decode_steps_follow_the_tables():
    """The launch of a decode step captured once; place() between the replays
    moves lengths and pages, and every replay equals an eager layer's step,
    with eager work between the replays."""
    need_gpu()
    r = np.random.default_rng(5)
    mk = lambda: PagedLayer(2, 16, n_pages=80, max_len=600, max_rows=300, page_size=16, budget=500, n_recent=8)  # noqa: E731
    a, b = mk(), mk()
    bits = lambda *s: dev(wk.to_bf16_bits(r.standard_normal(s).astype(np.float32))).view(torch.bfloat16)  # noqa: E731
    q0, x0 = bits(400, 16, 576), bits(400, 576)
    for layer in (a, b):
        layer.step(q0, x0, [270, 130])
    q, x = bits(2, 16, 576), bits(2, 576)
    for layer in (a, b):                        # warm-up outside the capture, buffers of T = 2
        layer.step(q, x, [1, 1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = a.launch(q, x)
    for i in range(6):
        q.copy_(bits(2, 16, 576))
        x.copy_(bits(2, 576))
        a.place([1, 1])
        g.replay()
        o2, l2 = b.step(q, x, [1, 1])
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2) and torch.equal(a.acc, b.acc), i
        y = torch.arange(4096, device='cuda', dtype=torch.float32)
        assert float((y * 2).sum().item()) == 4096 * 4095
    assert torch.equal(a.pool, b.pool)


def test_release_and_refusals():
    need_gpu()
    layer = PagedLayer(2, 4, n_pages=8, max_len=100, max_rows=64, page_size=16, budget=50)
    z = lambda n: (torch.zeros((n, 4, 576), dtype=torch.bfloat16, device='cuda'),  # noqa: E731
                   torch.zeros((n, 576), dtype=torch.bfloat16, device='cuda'))
    layer.step(*z(64), [64, 0])                 # cut to 50: 4 pages
    assert layer.lens.tolist() == [50, 0] and len(layer.pages.free) == 4
    before = layer.pages.table.copy()
    for counts in ([65, 0], [1], [-1, 0], [0, 64 + 1], [51, 0]):
        with pytest.raises(ValueError):
            layer.place(counts)
    with pytest.raises(ValueError):
        layer.place([40, 64])                   # 6 + 4 pages of 8
    assert np.array_equal(layer.pages.table, before) and layer.lens.tolist() == [50, 0]
    with pytest.raises(ValueError):
        layer.step(*z(3), [2, 2])
    assert layer.lens.tolist() == [50, 0]       # nothing was placed
    layer.step(*z(0), [0, 0])                   # a step without rows changes nothing but the decay
    assert layer.lens.tolist() == [50, 0]
    layer.release(0)
    assert layer.lens[0] == 0
    layer.step(*z(64), [0, 64])
    with pytest.raises(ValueError):
        PagedLayer(1, 4, 4, 64, 8, n_sink=40, n_recent=30, budget=60)


def test_chunks_of_many_sizes_keep_no_buffers():
    """Only steps of at most B rows leave buffers with the layer; a chunk's
    results are its own, on another stream too."""
    need_gpu()
    r = np.random.default_rng(9)
    layer = PagedLayer(2, 16, n_pages=100, max_len=700, max_rows=64, page_size=16)
    bits = lambda *s: dev(wk.to_bf16_bits(r.standard_normal(s).astype(np.float32))).view(torch.bfloat16)  # noqa: E731
    outs = []
    side = torch.cuda.Stream()
    for T in (3, 17, 64, 40, 2, 1, 33):
        q, x = bits(T, 16, 576), bits(T, 576)
        layer.place([T, 0])
        torch.cuda.synchronize()
        got = layer.launch(q, x, stream=side)
        junk = torch.full((T, 16, 512), 3.0, dtype=torch.bfloat16, device='cuda')
        torch.cuda.synchronize()
        outs.append((got[0], got[0].clone(), junk))
    assert set(layer._bufs) == {1, 2}
    for out, was, _ in outs[:4]:
        assert torch.equal(out, was)


def test_rows_behind_the_last_sequence_are_ignored():
    """A launch of more rows than were placed (a captured one of a smaller
    batch): the placed ones' results are those of a launch without them."""
    need_gpu()
    r = np.random.default_rng(11)
    bits = lambda *s: dev(wk.to_bf16_bits(r.standard_normal(s).astype(np.float32))).view(torch.bfloat16)  # noqa: E731
    a, b = (PagedLayer(3, 16, n_pages=60, max_len=300, max_rows=64, page_size=16, budget=200) for _ in range(2))
    for counts in ([40, 0, 7], [1, 0, 1], [1, 1, 0]):
        T = sum(counts)
        q, x = bits(T + 5, 16, 576), bits(T + 5, 576)
        assert a.place(counts) == T
        out, lse = a.launch(q, x)
        want = b.step(q[:T], x[:T], counts)
        torch.cuda.synchronize()
        assert torch.equal(out[:T], want[0]) and torch.equal(lse[:T], want[1])
        assert torch.equal(a.pool, b.pool) and torch.equal(a.acc, b.acc)
    assert int(a.status.item()) == 0
    with pytest.raises(ValueError):
        a.place([5, 0, 0])
        a.launch(bits(4, 16, 576), bits(4, 576))


def test_decode_captured_for_one_row_a_sequence():
    """A launch captured after place(..., max_rows=1) gives the bits of eager
    steps, which take the same form; eager chunks and evictions run between the
    replays, and weights past a sequence's length stay 0."""
    need_gpu()
    r = np.random.default_rng(13)
    bits = lambda *s: dev(wk.to_bf16_bits(r.standard_normal(s).astype(np.float32))).view(torch.bfloat16)  # noqa: E731
    B, H = 12, 32
    a, b = (PagedLayer(B, H, n_pages=12 * 20, max_len=2000, max_rows=500, page_size=16, budget=256, n_recent=8, slack=20)
            for _ in range(2))
    q0, x0 = bits(600, H, 576), bits(600, 576)
    chunk = [250, 13, 0, 41] + [37] * 8
    n = sum(chunk)
    for layer in (a, b):
        layer.step(q0[:n], x0[:n], chunk)
    q, x = bits(B, H, 576), bits(B, 576)
    for layer in (a, b):                        # warm-up
        layer.step(q, x, [1] * B)
    a.place([1] * B, max_rows=1)
    b.place([1] * B)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = a.launch(q, x)
    g.replay()
    b.launch(q, x)
    trims = 0
    for i in range(52):
        if i in (9, 30):
            q1, x1 = bits(30, H, 576), bits(30, 576)
            for layer in (a, b):
                layer.step(q1, x1, [30] + [0] * (B - 1))
        q.copy_(bits(B, H, 576))
        x.copy_(bits(B, 576))
        a.place([1] * B, max_rows=1)
        g.replay()
        trims += int(a.trim())
        o2, l2 = b.step(q, x, [1] * B)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2) and torch.equal(a.acc, b.acc), i
        assert torch.equal(a.seq_len, b.seq_len) and torch.equal(a.table, b.table)
        for s, m in enumerate(b.lens):
            assert not torch.any(b.acc[s, int(m):]), (i, s)
        y = torch.arange(4096, device='cuda', dtype=torch.float32)
        assert float((y * 2).sum().item()) == 4096 * 4095
    assert trims >= 2 and torch.equal(a.pool, b.pool)
    with pytest.raises(ValueError):
        a.place([2] + [1] * (B - 1), max_rows=1)


@pytest.mark.parametrize('B,H,window,sink', [(32, 16, 0, 0), (6, 128, 0, 0), (32, 32, 100, 4)])
def test_decode_steps_of_a_layer_with_chunks_against_the_oracle(B, H, window, sink):
    """Decoding in a layer that also takes chunks, whose bound of rows is not a
    decoding step's: outputs, weights and evictions."""
    need_gpu()
    r = np.random.default_rng(B + H)
    layer = PagedLayer(B, H, n_pages=B * 20, max_len=300, max_rows=200, page_size=16, window=window, n_sink=sink,
                       budget=200, n_recent=window or 20, decay=0.9)
    steps = [[int(n) for n in r.integers(0, 200, B)]] + [[1] * B] * 2 + [[0, 1] * (B // 2), [30] + [1] * (B - 1), [1] * B]
    run(layer, steps, 17, window, sink)


@pytest.mark.parametrize('window,sink,budget,slack', [(40, 3, 60, 0), (20, 0, 20, 7), (1, 2, 30, 0)])
def test_window_of_the_model_survives_evictions(window, sink, budget, slack):
    """With n_recent = window - 1 every row attends as if nothing had been
    evicted: the oracle keeps all rows at their own positions."""
    need_gpu()
    r = np.random.default_rng(window)
    B, H = 3, 16
    layer = PagedLayer(B, H, n_pages=B * 13, max_len=200, max_rows=100, page_size=16, window=window, n_sink=sink,
                       budget=budget, n_recent=window - 1, slack=slack)
    m, trimmed = Model(B), 0
    for i, counts in enumerate(STEPS):
        T = sum(counts)
        q = wk.to_bf16_bits(r.standard_normal((T, H, 576)).astype(np.float32))
        x = wk.to_bf16_bits(r.standard_normal((T, 576)).astype(np.float32))
        row0 = np.concatenate([[0], np.cumsum(counts)])
        before = layer.lens.sum() + T
        out, lse = layer.step(dev(q).view(torch.bfloat16), dev(x).view(torch.bfloat16), counts)
        trimmed += int(layer.lens.sum() < before)
        for b in range(B):
            m.rows[b] = np.concatenate([m.rows[b], x[row0[b]:row0[b + 1]]])
        pool, table, page, lens = m.dense()
        ref = oracle.paged.attention(q, pool, table, page, row0, lens, SCALE, window, sink)
        check_attn((out.float().cpu().numpy(), host(lse)), ref, int(lens.max()), f'step {i}')
    assert trimmed >= 2 and lens.max() > budget + 40


def test_decoding_keeps_one_workspace():
    """Growing contexts and counts ask for workspaces of many sizes: the layer
    keeps the largest, and those that a captured launch holds, whose replays
    still give an eager step's bits."""
    need_gpu()
    r = np.random.default_rng(19)
    bits = lambda *s: dev(wk.to_bf16_bits(r.standard_normal(s).astype(np.float32))).view(torch.bfloat16)  # noqa: E731
    B, H = 6, 16
    a, b = (PagedLayer(B, H, n_pages=6 * 200, max_len=3000, max_rows=400, page_size=16, budget=3000) for _ in range(2))
    q, x = bits(B, H, 576), bits(B, 576)
    for layer in (a, b):
        layer.step(q, x, [1] * B)
    a.place([1] * B, max_rows=1)
    b.place([1] * B)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = a.launch(q, x)
    g.replay()
    b.launch(q, x)
    first, sizes = a._ws, set()
    for i in range(12):
        n = 220
        q1, x1 = bits(n, H, 576), bits(n, 576)
        for layer in (a, b):
            layer.step(q1, x1, [n, 0, 0, 0, 0, 0])          # a chunk: a workspace of its own
            for counts in ([6, 0, 0, 0, 0, 0], [0, 2, 1, 0, 1, 2], [3, 1, 0, 0, 0, 0]):
                T = sum(counts)
                layer.step(q1[:T], x1[:T], counts)
                sizes.add(layer._ws_bytes(T, *layer._bounds(False)))
        a.place([1] * B, max_rows=1)
        g.replay()
        o2, l2 = b.step(q, x, [1] * B)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2) and torch.equal(a.acc, b.acc), i
    assert len(sizes) > 2 and a._ws.numel() >= max(sizes)
    assert a._held[0] is first and len(a._held) == 1 and not b._held
