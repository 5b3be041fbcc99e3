"""Steps of drafts at the limits of their calls (DraftStep, PagedLayer.accept):
what is kept, the rows and the next tokens have to be the oracle's."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, host, need_gpu
from indexer_top_kv_amd.pipeline import DraftStep, PagedLayer
from test_gpu_paged import SCALE, check_attn
from test_gpu_paged_layer import Model
from test_gpu_tree_attn import trees
from test_gpu_tree_layer import rows_of, some

pytestmark = pytest.mark.gpu


def long_chains(drawn, seed=1):
    """Chains that pass 256 rows: tokens, logits, draft, u and temperatures of three sequences."""
    r = np.random.default_rng(seed)
    counts, V = [300, 257, 4], 100
    T, row0 = sum(counts), np.concatenate([[0], np.cumsum(counts)])
    x = r.standard_normal((T, V)).astype(np.float32)
    x[np.arange(T), r.integers(0, V, T)] += 30.0           # all but certain: whole chains pass
    tokens = np.concatenate([[3], x.argmax(1)[:-1]]).astype(np.int32)
    q = None
    if drawn:
        q = np.exp(0.9 * x.astype(np.float64))
        q = (q / q.sum(1, keepdims=True)).astype(np.float32)
    return counts, row0, x, tokens, q, r.random(T).astype(np.float32), np.array([0.0, 0.8, 1.0], np.float32)


def decided(row0, counts, x, tokens, q, u, temps, most):
    """The oracle over the first 256 rows of each sequence."""
    kept, nxt, near = [], [], []
    for b, n in enumerate(counts):
        k, t, d = oracle.drafts.verify(x, tokens, [row0[b], row0[b] + min(n, 256)], u, most, None, q, temps[b:b + 1])
        kept, nxt, near = kept + k, nxt + t, near + d
    return kept, nxt, min(near)


@pytest.mark.parametrize('drawn', [False, True])
def test_chains_of_more_rows_than_are_verified(drawn):
    need_gpu()
    counts, row0, x, tokens, q, u, temps = long_chains(drawn)
    r = np.random.default_rng(2)
    layers = [PagedLayer(3, 4, n_pages=120, max_len=700, max_rows=300, page_size=16) for _ in range(2)]
    news = [some(r, sum(counts), 576) for _ in layers]
    ds = DraftStep(layers, 300)
    for layer, new in zip(layers, news):
        layer.draft(dev(some(r, sum(counts), 4, 576)).view(torch.bfloat16), dev(new).view(torch.bfloat16), None, counts)
    got = ds.finish(dev(x), dev(tokens), dev(u), draft=None if q is None else dev(q), temperature=dev(temps))
    kept, nxt, near = decided(row0, counts, x, tokens, q, u, temps, 300)
    assert near > 1e-9 and [len(k) for k in kept] == [256, 256, 4]
    assert got.counts.tolist() == [256, 256, 4] and got.next_token.tolist() == nxt
    assert got.kept.tolist() == [k + [-1] * (300 - len(k)) for k in kept]
    for layer, new in zip(layers, news):
        assert layer.lens.tolist() == [256, 256, 4] and host(layer.seq_len).tolist() == [256, 256, 4]
        for b in range(3):
            np.testing.assert_array_equal(rows_of(layer, b), new[row0[b]:row0[b] + len(kept[b])])
        layer.place([1, 1, 1])                              # the step is over


@pytest.mark.parametrize('made_on_it', [False, True])
def test_a_foreign_stream_is_not_touched_after_its_step(made_on_it, monkeypatch):
    """A stream that torch does not own may be gone when the next step comes:
    nothing is recorded on it then, and the steps' results are those of one stream."""
    need_gpu()
    side = torch.cuda.Stream()
    foreign = torch.cuda.ExternalStream(side.cuda_stream)
    layer, r = PagedLayer(1, 16, n_pages=20, max_len=100, max_rows=40, page_size=16), np.random.default_rng(3)
    logits = torch.zeros((3, 50), device='cuda')
    logits[:, 7] = 100.
    tokens, u = torch.full((3,), 7, dtype=torch.int32, device='cuda'), torch.full((3,), 0.5, device='cuda')
    news = [some(r, 3, 576) for _ in range(3)]
    torch.cuda.synchronize()

    def step(ds, new):
        layer.draft(dev(some(r, 3, 16, 576)).view(torch.bfloat16), dev(new).view(torch.bfloat16), None, [3])
        if ds is not None:
            got = ds.finish(logits, tokens, u)
            assert got.counts.tolist() == [3] and got.kept.tolist() == [[0, 1, 2, -1]] and got.next_token.tolist() == [7]
    with torch.cuda.stream(foreign if made_on_it else torch.cuda.current_stream()):
        ds = DraftStep([layer], 4)
    if not made_on_it:
        with torch.cuda.stream(foreign):
            step(ds, news[0])
    named, record = [], torch.cuda.Stream.record_event

    def seen(self, event=None):
        named.append(self.cuda_stream)
        return record(self, event)
    monkeypatch.setattr(torch.cuda.Stream, 'record_event', seen)
    for new in news[1:]:
        step(ds, new)
    assert side.cuda_stream not in named
    monkeypatch.undo()
    want = np.concatenate(news[1:] if made_on_it else news)
    np.testing.assert_array_equal(rows_of(layer, 0), want)


@pytest.mark.parametrize('window,sink', [(0, 0), (20, 3)])
def test_replayed_draft_launches_against_the_oracle(window, sink):
    """A captured launch of trees, replayed for steps of other sizes, within the
    bounds that test_gpu_paged.py derives; the steps' rows stay or leave between."""
    need_gpu()
    r, H, most = np.random.default_rng(11), 32, 24
    layer, m = PagedLayer(2, H, n_pages=80, max_len=500, max_rows=most, page_size=16, window=window, n_sink=sink), Model(2)
    first = some(r, 20, 576)
    layer.step(dev(some(r, 20, H, 576)).view(torch.bfloat16), dev(first).view(torch.bfloat16), [13, 7])
    m.rows = [first[:13], first[13:]]
    q = torch.zeros((most, H, 576), dtype=torch.bfloat16, device='cuda')
    x, parent = torch.zeros((most, 576), dtype=torch.bfloat16, device='cuda'), torch.full((most,), -1, dtype=torch.int32, device='cuda')
    g = torch.cuda.CUDAGraph()
    layer.place([0, 0], max_rows=most, drafts=True)
    with torch.cuda.graph(g):
        out, lse = layer.launch(q, x, parent=parent)
    none = torch.zeros((2, 1), dtype=torch.int32, device='cuda')
    layer.accept(none, none[:, 0].contiguous(), [0, 0])
    for step, (counts, kind) in enumerate([([10, 10], 'random'), ([24, 0], 'chain'), ([1, 9], 'star'), ([0, 24], 'forest'), ([11, 13], 'binary')]):
        T, row0 = sum(counts), np.concatenate([[0], np.cumsum(counts)])
        qb, xb, par = some(r, T, H, 576), some(r, T, 576), trees(kind, counts, step)
        for to, new in ((q, dev(qb).view(torch.bfloat16)), (x, dev(xb).view(torch.bfloat16)), (parent, dev(par))):
            to[:T].copy_(new)
        layer.place(counts, max_rows=most, drafts=True)
        g.replay()
        before = m.rows
        m.rows = [np.concatenate([m.rows[b], xb[row0[b]:row0[b + 1]]]) for b in range(2)]
        pool, table, page, lens = m.dense()
        ref = oracle.drafts.attention(qb, pool, table, page, row0, lens, par, SCALE, window, sink)
        check_attn((out[:T].float().cpu().numpy(), host(lse[:T])), ref, int(lens.max()), f'step {step}')
        keep = [[i for i in range(n) if r.random() < 0.5] for n in counts]
        kept = np.full((2, max(1, *map(len, keep))), -1, np.int32)
        for b, k in enumerate(keep):
            kept[b, :len(k)] = k
        layer.accept(dev(kept), dev(np.array([len(k) for k in keep], np.int32)), [len(k) for k in keep])
        m.rows = [np.concatenate([before[b], xb[row0[b]:row0[b + 1]][keep[b]]]) for b in range(2)]
        for b in range(2):
            np.testing.assert_array_equal(rows_of(layer, b), m.rows[b])
