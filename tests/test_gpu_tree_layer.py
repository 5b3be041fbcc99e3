"""Steps of drafts as a model makes them: two layers with the same sequences
take the rows of trees or chains (PagedLayer.draft), the target's logits decide
(DraftStep), the accepted rows stay, sequences fork and end, ordinary steps come
between. The oracle keeps every sequence's rows as a plain list. Tolerances of the
attention as in test_gpu_paged.py; what is kept, and the rows themselves, have to
be equal."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wk
from gpu_util import dev, host, need_gpu
from indexer_top_kv_amd.pipeline import DraftStep, PagedLayer
from test_gpu_tree_attn import trees
from test_gpu_paged import SCALE, check_attn
from test_gpu_paged_layer import Model
from test_gpu_paged_streams import WAIT

pytestmark = pytest.mark.gpu
V = 3000


def rows_of(layer, b):
    """The rows that a layer holds of sequence b, from its pool."""
    at = oracle.paged.slots(host(layer.table)[b], layer.pages.page_size, layer.pool.shape[0], int(layer.lens[b]))
    assert (at >= 0).all()
    return host(layer.pool.view(torch.int16)).view(np.uint16)[at]


def some(r, *shape):
    return wk.to_bf16_bits(r.standard_normal(shape).astype(np.float32))


def check_layer(layer, m):
    assert np.array_equal(layer.lens, [len(x) for x in m.rows])
    assert np.array_equal(host(layer.seq_len), layer.lens)
    for b in range(layer.B):
        np.testing.assert_array_equal(rows_of(layer, b), m.rows[b])
    pages = [p for b in range(layer.B) for p in layer.pages.table[b, :layer.pages.held[b]].tolist()]
    assert len(set(pages)) + len(layer.pages.free) == layer.pages.n_pages and not set(pages) & set(layer.pages.free)
    assert len(pages) - len(set(pages)) == layer.pages.more.sum()


def draft_step(layers, models, ds, r, counts, kind, drawn=False, seed=0):
    T, row0 = sum(counts), np.concatenate([[0], np.cumsum(counts)])
    parent = trees(kind, counts, seed) if kind else None
    for layer, m in zip(layers, models):
        q, x = some(r, T, layer.H, 576), some(r, T, 576)
        before = [y.copy() for y in m.rows]
        for b in range(layer.B):
            m.rows[b] = np.concatenate([m.rows[b], x[row0[b]:row0[b + 1]]])
        out, lse = layer.draft(dev(q).view(torch.bfloat16), dev(x).view(torch.bfloat16), None if parent is None else dev(parent), counts)
        pool, table, page, lens = m.dense()
        args = (q, pool, table, page, row0, lens)
        ref = (oracle.paged.attention(*args, SCALE, layer.window, layer.n_sink) if parent is None else
               oracle.drafts.attention(*args, parent, SCALE, layer.window, layer.n_sink))
        check_attn((out.float().cpu().numpy(), host(lse)), ref, int(lens.max()))
        m.rows, m.step = before, x
    logits = (2 * r.standard_normal((T, V))).astype(np.float32)
    first = np.repeat(row0[:-1], counts)
    before = first + (np.arange(T) - first - 1 if parent is None else parent).clip(0)
    tokens = np.where(r.random(T) < 0.7, logits.argmax(1)[before], r.integers(0, V, T)).astype(np.int32)
    draft = None
    if drawn:
        q = np.exp(logits + 0.5 * r.standard_normal((T, V)))
        draft = (q / q.sum(1, keepdims=True)).astype(np.float32)
    u, temp = r.random(T).astype(np.float32), r.choice([0.0, 0.3, 1.0], layers[0].B).astype(np.float32)
    opt = lambda x: None if x is None else dev(x)  # noqa: E731
    got = ds.finish(dev(logits), dev(tokens), dev(u), parent=opt(parent), draft=opt(draft), temperature=dev(temp))
    kept, nxt, near = oracle.drafts.verify(logits, tokens, row0, u, ds.most, parent, draft, temp)
    assert min(near) > 1e-9
    assert got.counts.tolist() == [len(k) for k in kept] and got.next_token.tolist() == nxt
    assert got.kept.tolist() == [k + [-1] * (ds.most - len(k)) for k in kept]
    for m in models:
        for b, k in enumerate(kept):
            m.rows[b] = np.concatenate([m.rows[b], m.step[row0[b]:row0[b + 1]][k]])
    return kept


@pytest.mark.parametrize('page,window,sink', [(16, 0, 0), (7, 20, 3), (1, 0, 0)])
def test_steps_of_drafts_between_others(page, window, sink):
    need_gpu()
    r = np.random.default_rng(page)
    B, H = 4, 16
    layers = [PagedLayer(B, H, n_pages=-(-1400 // page), max_len=400, max_rows=120, page_size=page, window=window, n_sink=sink)
              for _ in range(2)]
    models, ds = [Model(B) for _ in layers], DraftStep(layers, 9)

    def plain(counts):
        for layer, m in zip(layers, models):
            q, x = some(r, sum(counts), H, 576), some(r, sum(counts), 576)
            row0 = np.concatenate([[0], np.cumsum(counts)])
            layer.step(dev(q).view(torch.bfloat16), dev(x).view(torch.bfloat16), counts)
            for b in range(B):
                m.rows[b] = np.concatenate([m.rows[b], x[row0[b]:row0[b + 1]]])

    kept = []
    plain([40, 0, 90, 0])
    for i, (counts, kind, drawn) in enumerate([([8, 0, 12, 0], 'random', False), ([1, 0, 30, 0], 'binary', False),
                                               ([6, 0, 5, 0], None, True), ([20, 0, 3, 0], 'star', False)]):
        kept += draft_step(layers, models, ds, r, counts, kind, drawn, seed=i)
        for layer, m in zip(layers, models):
            check_layer(layer, m)
    for layer, m in zip(layers, models):                        # samples of sequence 2's prompt go on by themselves
        layer.fork(2, [1, 3])
        m.rows[1], m.rows[3] = m.rows[2].copy(), m.rows[2].copy()
        check_layer(layer, m)
        assert page == 1 or layer.pages.more.sum() > 0
    for i, (counts, kind) in enumerate([([3, 9, 17, 2], 'random'), ([4, 4, 4, 4], None), ([1, 1, 64, 11], 'random')]):
        kept += draft_step(layers, models, ds, r, counts, kind, seed=50 + i)
        for layer, m in zip(layers, models):
            check_layer(layer, m)
    for layer, m in zip(layers, models):                        # the prompt's first holder ends; its samples stay
        layer.release(2)
        m.rows[2] = np.zeros((0, 576), np.uint16)
        check_layer(layer, m)
    plain([1, 1, 33, 1])
    kept += draft_step(layers, models, ds, r, [2, 40, 9, 5], 'random', seed=70)
    for layer, m in zip(layers, models):
        check_layer(layer, m)
        for b in (1, 3, 0, 2):
            layer.release(b)
        assert len(layer.pages.free) == layer.pages.n_pages and not layer.pages.more.any()
    lengths = [len(k) for k in kept if k]
    assert max(lengths) > 3 and min(lengths) == 1


def test_fork_with_a_budget_copies():
    """Evictions in place move rows: forked sequences of such a layer share none,
    and go on with the weights that the first had."""
    need_gpu()
    r = np.random.default_rng(3)
    layer = PagedLayer(3, 16, n_pages=60, max_len=300, max_rows=100, page_size=16, budget=60, n_recent=10, slack=10)
    q, x = (dev(some(r, *s)).view(torch.bfloat16) for s in ((65, 16, 576), (65, 576)))
    layer.step(q, x, [65, 0, 0])
    layer.fork(0, 2)
    assert not layer.pages.more.any() and layer.lens.tolist() == [65, 0, 65]
    np.testing.assert_array_equal(rows_of(layer, 2), rows_of(layer, 0))
    assert torch.equal(layer.acc[2], layer.acc[0]) and layer.acc[0, :65].min() > 0
    q, x = (dev(some(r, *s)).view(torch.bfloat16) for s in ((7, 16, 576), (7, 576)))
    q, x = torch.cat([q, q]), torch.cat([x, x])                 # the same rows: the same evictions
    layer.step(q, x, [7, 0, 7])
    assert layer.lens.tolist() == [60, 0, 60]
    np.testing.assert_array_equal(rows_of(layer, 2), rows_of(layer, 0))
    assert torch.equal(layer.acc[2], layer.acc[0])
    with pytest.raises(ValueError, match='budget'):
        layer.draft(q[:2], x[:2], None, [1, 0, 1])


def test_captured_draft_launch():
    """A launch of trees captured once, replayed for steps placed with the same
    bound; on another stream than the eager calls."""
    need_gpu()
    r = np.random.default_rng(5)
    layers = [PagedLayer(2, 32, n_pages=80, max_len=500, max_rows=300, page_size=16) for _ in range(2)]
    a, b = layers                                               # a replays, b runs eagerly
    q, x = (dev(some(r, *s)).view(torch.bfloat16) for s in ((90, 32, 576), (90, 576)))
    for layer in layers:
        layer.step(q, x, [50, 40])
    q, x, parent = torch.empty((20, 32, 576), dtype=torch.bfloat16, device='cuda'), torch.empty((20, 576), dtype=torch.bfloat16, device='cuda'), \
        torch.empty(20, dtype=torch.int32, device='cuda')
    q.zero_(), x.zero_(), parent.fill_(-1)
    with pytest.raises(ValueError):
        a.place([10, 10], drafts=True)
        with torch.cuda.graph(torch.cuda.CUDAGraph()):          # made for any step: 300 rows a sequence
            torch.zeros(1, device='cuda')
            a.launch(q, x, parent=parent)
    a.accept(torch.zeros((2, 1), dtype=torch.int32, device='cuda'), torch.zeros(2, dtype=torch.int32, device='cuda'), [0, 0])
    a.place([10, 10], max_rows=16, drafts=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = a.launch(q, x, parent=parent)
    a.accept(torch.zeros((2, 1), dtype=torch.int32, device='cuda'), torch.zeros(2, dtype=torch.int32, device='cuda'), [0, 0])
    for step, counts in enumerate([[10, 10], [4, 16], [16, 0], [1, 9]]):
        T = sum(counts)
        q.copy_(dev(some(r, 20, 32, 576)).view(torch.bfloat16))
        x.copy_(dev(some(r, 20, 576)).view(torch.bfloat16))
        par = trees('random', counts, step)
        parent[:T].copy_(dev(par))
        a.place(counts, max_rows=16, drafts=True)
        g.replay()
        eager = b.draft(q[:T], x[:T], parent[:T].clone(), counts)
        n = max(int(a.lens.max()), 1)
        # the same arithmetic in spans of another number: both are within the bounds that test_gpu_paged.py derives
        assert torch.allclose(out[:T].float(), eager[0].float(), rtol=2.0 ** -6, atol=2.0 ** -6) and n < 500
        assert torch.allclose(lse[:T], eager[1], rtol=1e-5, atol=1e-4)
        kept = torch.tensor([[0, counts[0] - 1], [0, -1]], dtype=torch.int32, device='cuda')
        keep = [min(2, counts[0]), min(1, counts[1])]
        n_kept = torch.tensor(keep, dtype=torch.int32, device='cuda')
        for layer in layers:
            layer.accept(kept, n_kept, keep)
        for s in range(2):
            np.testing.assert_array_equal(rows_of(a, s), rows_of(b, s))


def test_calls_on_several_streams():
    """draft, finish, fork and release from changing streams give what one
    stream gives."""
    need_gpu()
    mk = lambda: [PagedLayer(3, 16, n_pages=200, max_len=600, max_rows=80, page_size=16) for _ in range(2)]  # noqa: E731
    got = []
    for streams in ([None], [torch.cuda.Stream(), None, torch.cuda.Stream()]):
        r, layers = np.random.default_rng(7), mk()
        ds, turn = DraftStep(layers, 6), 0
        log = []

        def on():
            nonlocal turn
            turn += 1
            s = streams[turn % len(streams)]
            return torch.cuda.stream(s)
        for i in range(12):
            counts = [int(n) for n in r.integers(0, 30, 3)]
            T = sum(counts)
            ins = [[dev(some(r, *s)).view(torch.bfloat16) for s in ((T, 16, 576), (T, 576))] for _ in layers]
            parent = dev(trees('random', counts, i))
            logits, u = dev((3 * r.standard_normal((T, V))).astype(np.float32)), dev(r.random(T).astype(np.float32))
            tokens = logits.argmax(1).to(torch.int32).roll(1)
            torch.cuda.synchronize()
            for layer, (q, x) in zip(layers, ins):
                with on():
                    layer.draft(q, x, parent, counts)
            with on():
                res = ds.finish(logits, tokens, u, parent=parent)
            log += [res.counts.tolist(), res.kept.tolist(), res.next_token.tolist()]
            if i == 6:
                for layer in layers:
                    with on():
                        layer.release(1)
                    with on():
                        layer.fork(0, 1)
        torch.cuda.synchronize()
        got.append((log, [rows_of(layer, b) for layer in layers for b in range(3)]))
    assert got[0][0] == got[1][0]
    for x, y in zip(got[0][1], got[1][1]):
        np.testing.assert_array_equal(x, y)


def test_a_step_without_rows():
    """No sequence brings a row: nothing changes, nothing is kept."""
    need_gpu()
    layer = PagedLayer(2, 16, n_pages=20, max_len=100, max_rows=40, page_size=16)
    x = dev(some(np.random.default_rng(1), 5, 576)).view(torch.bfloat16)
    layer.step(torch.zeros((5, 16, 576), dtype=torch.bfloat16, device='cuda'), x, [5, 0])
    none = dict(dtype=torch.int32, device='cuda')
    out, lse = layer.draft(torch.zeros((0, 16, 576), dtype=torch.bfloat16, device='cuda'), x[:0], torch.zeros(0, **none), [0, 0])
    assert out.shape == (0, 16, 512)
    got = DraftStep([layer], 3).finish(torch.zeros((0, 50), device='cuda'), torch.zeros(0, **none), torch.zeros(0, device='cuda'),
                                       parent=torch.zeros(0, **none))
    assert got.counts.tolist() == [0, 0] and got.next_token.tolist() == [-1, -1] and (got.kept == -1).all()
    assert layer.lens.tolist() == [5, 0] and host(layer.seq_len).tolist() == [5, 0]


def test_buffers_made_on_a_stream_that_is_busy():
    """A DraftStep's buffers may be memory that the stream it was made on still
    writes: the first finish on another stream comes behind that."""
    need_gpu()
    layer = PagedLayer(1, 16, n_pages=20, max_len=100, max_rows=40, page_size=16)
    r, side, ended = np.random.default_rng(3), torch.cuda.Stream(), torch.cuda.Event()
    q, x = (dev(some(r, *s)).view(torch.bfloat16) for s in ((3, 16, 576), (3, 576)))
    logits = torch.zeros((3, 50), device='cuda')
    logits[:, 7] = 100.
    tokens, u = torch.full((3,), 7, dtype=torch.int32, device='cuda'), torch.full((3,), 0.5, device='cuda')
    layer.draft(q, x, None, [3])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        old = torch.empty(64, dtype=torch.int32, device='cuda')
        torch.cuda._sleep(WAIT)
        old.fill_(-7)
        del old
        ds = DraftStep([layer], 4)
        ended.record()
    got = ds.finish(logits, tokens, u)
    assert ended.query()
    assert got.counts.tolist() == [3] and got.kept.tolist() == [[0, 1, 2, -1]] and got.next_token.tolist() == [7]
    np.testing.assert_array_equal(rows_of(layer, 0), host(x.view(torch.int16)).view(np.uint16))
