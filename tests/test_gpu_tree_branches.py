"""Verification of drafted tokens row by row (a launch for each row that a branch
may have, where a batch has many rows beside its branches): deep branches that
end at odd and even levels, more rows allowed than a sequence has, graphs, other
streams, and a workspace shared with a batch that is summed whole. Every number has
to be the oracle's; no decision lies near its border (see
test_gpu_tree_verify.py)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, need_gpu
import indexer_top_kv_amd as ech
from test_gpu_tree_verify import Drafts

pytestmark = pytest.mark.gpu


class Deep(Drafts):
    """Most drafts are their row's likeliest token, which is all but certain."""

    def __init__(self, *args, right=0.9, **kw):
        super().__init__(*args, **kw)
        if self.draft is None:
            for b in range(self.B):
                for i in range(1, self.rows[b]):
                    if self.r.random() < right:
                        r0 = int(self.row0[b])
                        before = r0 + (i - 1 if self.parent is None else max(int(self.parent[r0 + i]), 0))
                        self.tokens[r0 + i] = self.x[before].argmax()

    def row_by_row(self):
        """By the workspace, which then holds two rows' sums a sequence instead of every row's."""
        chunks = -(-(self.V + 7) // 1024)
        n = ech.ech_draft_verify_ws_bytes(self.B, self.T, self.V, max(self.rows), self.most)
        return n < self.T * chunks * 16


CASES = [
    # rows, V, kind, drawn, temperatures, most, peak
    ([30] * 8, 140001, None, True, [0.8, 1.0, 0.0, 0.9], 7, 16.0),
    ([30] * 8, 140001, None, False, [0.8, 1.0, 0.0, 0.9], 7, 18.0),
    ([60, 0, 50, 61, 60, 64, 2, 60], 90001, 'random', False, [0.8, 1.0, 0.0], 6, 18.0),
    ([60, 64, 50, 61, 60, 64, 2, 60], 90001, 'binary', False, [0.7, 0.9], 6, 18.0),
    # `most` beyond the rows: the last kernel looks for a child of the last level's row
    ([8] * 16, 440001, None, True, [0.8, 1.0, 0.0, 0.9], 11, 18.0),
    ([8] * 16, 440001, None, False, [0.8, 0.0, 0.9], 9, 20.0),
    ([8] * 16, 440001, 'chain', False, [0.8, 0.0, 0.9], 8, 20.0),
    ([8] * 16, 440001, 'random', False, [0.8, 0.0], 9, 20.0),
]


@pytest.mark.parametrize('bf16', [True, False])
@pytest.mark.parametrize('rows,V,kind,drawn,temps,most,peak', CASES)
def test_deep_branches(rows, V, kind, drawn, temps, most, peak, bf16):
    need_gpu()
    c = Deep(rows, V, kind, bf16, drawn, seed=V + most, temps=temps, most=most, peak=peak)
    assert c.row_by_row()
    kept, _ = c.check()
    lengths = {len(k) for k in kept}
    assert max(lengths) > 3
    if bf16:                                               # odd and even ends; the fp32 rows draw other drafts
        assert len({n % 2 for n in lengths}) == 2
    if most >= max(rows) and kind in (None, 'chain'):
        assert max(rows) in lengths                        # whole chains


def graph_batches():
    return [Deep([64] * 8, 40001, None, drawn=True, seed=31, temps=[0.8, 0.0, 1.0], most=4, peak=14.0),
            Deep([7] * 6, 9000, 'random', seed=32, temps=[0.8], peak=12.0),
            Deep([64] * 8, 40001, 'binary', seed=33, temps=[0.9, 0.0], most=4, peak=14.0)]


def numbers(c, rep):
    return np.random.default_rng(500 + rep).random(c.T).astype(np.float32)


def test_row_by_row_in_a_graph_with_a_shared_workspace():
    """Both ways in turn on one workspace: on another stream, then captured and
    replayed on new numbers between eager calls; every result is the oracle's."""
    need_gpu()
    cs = graph_batches()
    assert [c.row_by_row() for c in cs] == [True, False, True]
    bufs = [c.buffers() for c in cs]
    ws = max((b[3] for b in bufs), key=lambda w: w.numel())
    s = torch.cuda.Stream()
    ins = [dict(logits=c.logits(), tokens=dev(c.tokens), row0=dev(c.row0), u=dev(c.u), temperature=dev(c.temps),
                parent=None if c.parent is None else dev(c.parent), draft=None if c.draft is None else dev(c.draft)) for c in cs]

    def calls(stream=None):
        for c, b, i in zip(cs, bufs, ins):
            ech.ech_draft_verify(max_rows=max(c.rows), kept=b[0], n_kept=b[1], next_token=b[2], ws=ws, stream=stream, **i)

    def check():
        torch.cuda.synchronize()
        for c, b in zip(cs, bufs):
            c.check([x.cpu().numpy() for x in b[:3]])
            for x in b[:3]:
                x.fill_(77)
        ws.fill_(0xff)
    torch.cuda.synchronize()
    calls(s)
    s.synchronize()
    check()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        calls()
    for rep in range(3):
        for c, i in zip(cs, ins):
            c.u = numbers(c, rep)
            i['u'].copy_(torch.from_numpy(c.u))
        torch.cuda.synchronize()
        g.replay()
        check()
        calls()
        check()


@pytest.mark.parametrize('drawn', [False, True])
def test_more_rows_than_the_bound(drawn):
    """Only the first max_rows rows of a sequence are looked at."""
    need_gpu()
    c = Deep([300, 5, 280], 60001, None, drawn=drawn, seed=41, temps=[0.9, 0.0], most=4, peak=14.0)
    for bound in (3, 256):
        got = [oracle.drafts.verify(c.x, c.tokens, [r, r + min(n, bound)], c.u, 4, None, c.draft, c.temps[b:b + 1])
               for b, (r, n) in enumerate(zip(c.row0, [300, 5, 280]))]
        assert min(d for x in got for d in x[2]) > 1e-9
        c.rows = [bound]                                   # of this, buffers and run take the largest
        assert c.row_by_row()
        kept, n_kept, nxt = c.run()
        assert n_kept.tolist() == [len(x[0][0]) for x in got] and nxt.tolist() == [x[1][0] for x in got]
        assert kept.tolist() == [x[0][0] + [-1] * (4 - len(x[0][0])) for x in got]
