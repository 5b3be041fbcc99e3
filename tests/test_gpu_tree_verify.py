"""Verification of drafted tokens (ech_draft_verify) against the oracle. Weights
are within 4e-11 of the formula's, relatively, and so are their sums (nothing is
subtracted), so both sides of a decision are within 1e-10: every number has to be
equal where no decision lies within 1e-9 of its border, which the oracle says and
the tests ask for."""
import numpy as np
import pytest
import torch

import oracle
from oracle.numerics import bf16_to_f64
from gpu_util import dev, need_gpu
import indexer_top_kv_amd as ech
from test_gpu_tree_attn import trees
import workloads as wk

pytestmark = pytest.mark.gpu


class Drafts:
    def __init__(self, rows, V, kind='random', bf16=True, drawn=False, seed=0, temps=None, most=None, lead=0, tail=0,
                 peak=6.0):
        r = self.r = np.random.default_rng(seed)
        self.rows, self.V, self.B = list(rows), V, len(rows)
        self.row0 = (lead + np.concatenate([[0], np.cumsum(rows)])).astype(np.int32)
        self.T = int(self.row0[-1]) + tail
        self.parent = None if kind is None else np.concatenate([np.full(lead, 3, np.int32), trees(kind, rows, seed + 1),
                                                                np.full(tail, -9, np.int32)])
        x = (1.5 * r.standard_normal((self.T, V))).astype(np.float32)
        x[np.arange(self.T), r.integers(0, V, self.T)] += peak
        self.bf16 = bf16
        self.bits = wk.to_bf16_bits(x)
        self.x = bf16_to_f64(self.bits).astype(np.float32) if bf16 else x
        before = np.array([int(self.row0[b]) + (i - 1 if kind is None else max(int(self.parent[self.row0[b] + i]), 0))
                           for b in range(self.B) for i in range(self.rows[b])], np.int64)
        before = np.concatenate([np.zeros(lead, np.int64), np.maximum(before, 0), np.zeros(tail, np.int64)])
        top = (np.argsort(-self.x, axis=1, kind='stable') if V < 20000 else np.argpartition(-self.x, 3, axis=1))[:, :3]
        self.tokens = np.where(r.random(self.T) < 0.8, top[before, r.integers(0, top.shape[1], self.T)],
                               r.integers(0, V, self.T)).astype(np.int32)
        self.draft = None
        if drawn:
            q = np.exp(self.x + 0.7 * r.standard_normal((self.T, V)))
            self.draft = (q / q.sum(1, keepdims=True)).astype(np.float32)
            self.tokens = np.array([r.choice(V, p=self.draft[p].astype(np.float64) / self.draft[p].astype(np.float64).sum())
                                    for p in before], np.int32)
        self.u = r.random(self.T).astype(np.float32)
        self.temps = None if temps is None else np.array([temps[b % len(temps)] for b in range(self.B)], np.float32)
        self.most = max(self.rows) if most is None else most

    def logits(self):
        return dev(self.bits).view(torch.bfloat16) if self.bf16 else dev(self.x)

    def buffers(self):
        i32 = dict(dtype=torch.int32, device='cuda')
        n = ech.ech_draft_verify_ws_bytes(self.B, self.T, self.V, max(self.rows), self.most)
        return (torch.full((self.B, self.most), 77, **i32), torch.full((self.B,), 77, **i32), torch.full((self.B,), 77, **i32),
                torch.full((n,), 0xff, dtype=torch.uint8, device='cuda'))

    def run(self, logits=None, draft=None, stream=None):
        kept, n_kept, nxt, ws = self.buffers()
        ech.ech_draft_verify(self.logits() if logits is None else logits, dev(self.tokens), dev(self.row0), max(self.rows),
                             dev(self.u), kept, n_kept, nxt, parent=None if self.parent is None else dev(self.parent),
                             draft=(None if self.draft is None else dev(self.draft)) if draft is None else draft,
                             temperature=None if self.temps is None else dev(self.temps), ws=ws, stream=stream)
        torch.cuda.synchronize()
        return kept.cpu().numpy(), n_kept.cpu().numpy(), nxt.cpu().numpy()

    def check(self, got=None, near=1e-9):
        kept, n_kept, nxt = self.run() if got is None else got
        k, t, d = oracle.drafts.verify(self.x, self.tokens, self.row0, self.u, self.most, self.parent, self.draft, self.temps)
        assert min(d) > near, 'a decision at its border: another seed is wanted'
        np.testing.assert_array_equal(n_kept, [len(x) for x in k])
        np.testing.assert_array_equal(kept, [x + [-1] * (self.most - len(x)) for x in k])
        np.testing.assert_array_equal(nxt, t)
        return k, t


SHAPES = [
    # rows, V, kind (None: chains), drawn, temperatures, most
    ([1], 1, 'random', False, None, None),
    ([1, 1], 2, None, False, None, None),
    ([4], 7, None, False, None, None),
    ([5, 0, 3, 1], 2047, None, False, [0.7, 1.0], None),
    ([8] * 9, 2048, 'random', False, [1.0, 0.0], None),
    ([12, 3, 30], 2049, 'random', False, [0.5], None),
    ([26, 1, 0, 7], 4091, 'forest', False, None, None),
    ([64] * 5, 5000, 'binary', False, [0.8, 0.0, 1.3], None),
    ([256, 9], 1000, 'random', False, [0.9], None),
    ([256], 300, 'star', False, [1.0], None),
    ([100, 200], 513, 'chain', False, [0.6], None),
    ([20] * 4, 6200, 'random', False, [0.8], 3),                  # branches are cut: nothing tried at their end
    ([20] * 4, 6200, 'random', False, [0.8], 1),
    ([6] * 7, 4099, None, True, [0.7, 1.0, 0.0], None),
    ([1, 2, 0, 9], 33, None, True, None, None),
    ([7] * 5, 6001, None, True, [0.9], 4),
    ([3] * 70, 129, None, False, [0.7, 0.0], None),               # more sequences than a wave has lanes
    ([2] * 300, 64, 'star', False, None, None),
    ([3, 2], 140001, 'star', False, [0.7], None),                 # more chunks than a wave has lanes
    ([3, 2, 1], 290000, None, True, [0.7, 1.0], None),
    ([3, 2], 140000, None, False, [0.0], None),
    # few rows of large batches: row by row
    ([20, 0, 20, 20, 20, 20, 20, 25, 20], 70001, 'random', False, [0.8, 0.0, 1.0], 2),
    ([20] * 8, 70000, None, True, [0.8, 0.0], 2),
    ([60] * 6, 70001, 'binary', False, [0.8], 4),
    ([64, 1, 64], 140001, 'forest', False, [1.0], 3),
    ([16] * 5, 140001, None, True, [1.2], 2),
    ([16] * 5, 140001, None, False, [1.2], 1),
]


@pytest.mark.parametrize('bf16', [True, False])
@pytest.mark.parametrize('rows,V,kind,drawn,temps,most', SHAPES)
def test_against_oracle(rows, V, kind, drawn, temps, most, bf16):
    need_gpu()
    Drafts(rows, V, kind, bf16, drawn, seed=V + sum(rows), temps=temps, most=most).check()


@pytest.mark.parametrize('drawn', [False, True])
@pytest.mark.parametrize('bf16', [True, False])
def test_every_alignment_of_rows(bf16, drawn):
    """Logits and drafts that are parts of wider tensors, from every offset."""
    need_gpu()
    for off in range(8):
        c = Drafts([3, 4], 4100, None if drawn else 'random', bf16, drawn, seed=off, temps=[0.8])
        wide = torch.full((c.T, c.V + 9), float('nan'), dtype=torch.bfloat16 if bf16 else torch.float32, device='cuda')
        wide[:, off:off + c.V] = c.logits()
        q = None
        if drawn:
            q = torch.full((c.T, c.V + 9), float('nan'), device='cuda')
            q[:, off:off + c.V] = dev(c.draft)
            q = q[:, off:off + c.V]
        c.check(c.run(logits=wide[:, off:off + c.V], draft=q))


def test_rows_of_no_sequence_and_more_rows_than_the_bound():
    need_gpu()
    c = Drafts([3, 4], 3000, 'random', seed=5, lead=2, tail=3, temps=[0.9, 0.8])
    c.check()
    c = Drafts([9, 12], 3000, None, seed=6)
    k, t, d = oracle.drafts.verify(c.x, c.tokens, c.row0, c.u, 12)
    kept, n_kept, nxt, ws = c.buffers()
    ech.ech_draft_verify(c.logits(), dev(c.tokens), dev(c.row0), 2, dev(c.u), kept, n_kept, nxt, ws=ws)
    torch.cuda.synchronize()
    cut = [oracle.drafts.verify(c.x, c.tokens, [r, r + 2], c.u, 12) for r in c.row0[:2]]
    assert kept[:, :2].tolist() == [(x[0][0] + [-1])[:2] for x in cut] and nxt.tolist() == [x[1][0] for x in cut]


@pytest.mark.parametrize('kind', ['random', 'star', None])
def test_numbers_at_their_ends(kind):
    """u = 0 and the last float below 1 (and what counts as them), in every
    combination a seed draws; peaked rows, so that masses far below 1 are left."""
    need_gpu()
    for seed in range(6):
        c = Drafts([9, 5, 17], 3000, kind, seed=seed, temps=[0.3, 1.0], peak=14.0)
        c.u = np.where(c.r.random(c.T) < 0.7, np.float32(1 - 2.0 ** -24), np.float32(0))
        want = c.check(near=0)
        c.u = np.where(c.u > 0, c.r.choice([1.0, 7.0, np.inf], c.T), c.r.choice([-0.0, -3.0, np.nan, -np.inf], c.T)).astype(np.float32)
        kept, n_kept, nxt = c.run()
        assert nxt.tolist() == want[1] and n_kept.tolist() == [len(k) for k in want[0]]


@pytest.mark.parametrize('drawn', [False, True])
def test_logits_that_are_not_finite(drawn):
    """Masked tokens (-inf, NaN, the type's lowest value), infinite ones, rows
    that are masked whole; temperatures that are extreme or none."""
    need_gpu()
    c = Drafts([4] * 12, 2500, None if drawn else 'star', bf16=False, drawn=drawn, seed=8,
               temps=[1.0, 0.0, np.nan, -2.0, np.inf, 1e-30, 0.5])
    r = c.r
    c.x[r.random(c.x.shape) < 0.5] = -np.inf
    c.x[r.random(c.x.shape) < 0.1] = np.nan
    c.x[r.random(c.x.shape) < 0.1] = np.finfo(np.float32).min
    c.x[4:8] = -np.inf
    c.x[8] = np.nan
    c.x[16] = np.where(np.arange(2500) % 700 == 5, np.inf, c.x[16])
    c.x[20, 13] = c.x[20, 2400] = np.inf
    c.x[24:28, :] = -np.inf
    c.x[24:28, 1234] = -3.0
    c.tokens[25:28] = [1234, 1234, 7]
    c.tokens[29:32] = [-1, 2500, 2 ** 31 - 1]
    if drawn:
        c.draft[3:6] = np.nan
        c.draft[32] = -1.0
        c.draft[36] = np.inf
        c.draft[40] = 0.0
    c.check()


def test_equal_logits_and_draft_equal_to_target():
    """Ties go to the lowest token; a draft that is the target itself leaves
    nothing behind a rejection (here forced by its number): the target is drawn
    from."""
    need_gpu()
    c = Drafts([3] * 4, 4200, None, bf16=False, drawn=True, seed=9, temps=[1.0, 0.0])
    c.x[:] = 0.0
    c.draft[:] = np.float32(2.0 ** -12)                   # above 1 / 4200: nowhere below the target
    c.u[:] = 0.9999
    c.tokens[:] = [0, 0, 5] * 4
    c.check()


def test_same_bits_on_another_stream_and_in_a_graph():
    """Two batches that share a workspace, captured, replayed with new numbers
    between eager work; every replay equals the eager call."""
    need_gpu()
    cs = [Drafts([7] * 6, 9000, 'random', seed=20, temps=[0.8]), Drafts([6] * 6, 9000, None, drawn=True, seed=21, temps=[0.8, 0.0])]
    s = torch.cuda.Stream()
    bufs = [c.buffers() for c in cs]
    ws = bufs[0][3] if bufs[0][3].numel() > bufs[1][3].numel() else bufs[1][3]
    ins = [dict(logits=c.logits(), tokens=dev(c.tokens), row0=dev(c.row0), u=dev(c.u), temperature=dev(c.temps),
                parent=None if c.parent is None else dev(c.parent), draft=None if c.draft is None else dev(c.draft)) for c in cs]

    def calls(stream=None):
        for c, b, i in zip(cs, bufs, ins):
            ech.ech_draft_verify(max_rows=max(c.rows), kept=b[0], n_kept=b[1], next_token=b[2], ws=ws, stream=stream, **i)
    torch.cuda.synchronize()
    calls(s)
    s.synchronize()
    for c, b in zip(cs, bufs):
        c.check([x.cpu().numpy() for x in b[:3]])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        calls(s)
    for rep in range(4):
        for c, i in zip(cs, ins):
            c.u = np.random.default_rng(100 + rep).random(c.T).astype(np.float32)
            i['u'].copy_(torch.from_numpy(c.u))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for c, b in zip(cs, bufs):
            c.check([x.cpu().numpy() for x in b[:3]])
            b[0].fill_(5)
