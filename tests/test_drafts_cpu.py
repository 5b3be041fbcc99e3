"""Drafted tokens without a GPU: refusals of the C ABI and of the binding, and
the oracle against closed forms and against the distribution that verification
has to keep."""
import itertools
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import draft_abi_checks
import indexer_top_kv_amd as ech
import oracle
from test_abi import ROOT, _clang_rt
import workloads as wk


@pytest.mark.parametrize('check', draft_abi_checks.CHECKS, ids=lambda f: f.__name__)
def test_argument_checks(check):
    check(ech.lib())


def test_argument_checks_under_asan_ubsan():
    from indexer_top_kv_amd import build as b
    rt = _clang_rt('asan')
    if rt is None or not os.path.exists(os.environ.get('HIPCC', '/opt/rocm/bin/hipcc')):
        pytest.skip('no hipcc or sanitizer runtime')
    lib = b.build_sanitized()
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS='detect_leaks=0:abort_on_error=1',
               UBSAN_OPTIONS='halt_on_error=1:print_stacktrace=1',
               LD_LIBRARY_PATH=os.path.dirname(rt) + ':' + os.environ.get('LD_LIBRARY_PATH', ''))
    r = subprocess.run([sys.executable, os.path.join(ROOT, 'tests', 'draft_abi_checks.py'), lib], env=env,
                       capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and 'draft abi checks ok' in r.stdout, out[-4000:]
    assert 'AddressSanitizer' not in out and 'runtime error' not in out, out[-4000:]


def test_binding_refuses_types_shapes_and_host_tensors():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    f = torch.float32
    good = dict(logits=z(4, 9, dt=f), tokens=z(4), row0=z(3), max_rows=2, u=z(4, dt=f), kept=z(2, 3), n_kept=z(2),
                next_token=z(2), parent=None, draft=None, temperature=None)
    for name, t in (('logits', z(4, 9, dt=torch.float16)), ('tokens', z(4, dt=torch.int64)), ('u', z(4, dt=torch.float64)),
                    ('draft', z(4, 9, dt=torch.bfloat16))):
        with pytest.raises((TypeError, ValueError)):
            ech.ech_draft_verify(**{**good, name: t})
    for bad in (dict(), dict(tokens=z(5)), dict(row0=z(2)), dict(kept=z(6)), dict(logits=z(9, 4, dt=f).t()),
                dict(max_rows=1 << 31), dict(parent=z(4), draft=z(4, 9, dt=f))):
        with pytest.raises(ValueError):                   # with nothing else wrong: host tensors
            ech.ech_draft_verify(**{**good, **bad})
    pool = z(64, 576, dt=torch.bfloat16)
    with pytest.raises(ValueError):
        ech.ech_paged_copy(pool, 16, z(2), z(2))
    with pytest.raises(ValueError):
        ech.ech_paged_accept(pool, z(1, 4), 16, z(2), z(1), z(1, 3), z(1), 3, 64, z(1))
    with pytest.raises(ValueError):
        ech.ech_paged_tree_attn(z(2, 4, 576, dt=torch.bfloat16), pool, z(1, 4), 16, z(2), z(1), z(2), 2, 64, 0.1,
                                z(2, 4, 512, dt=torch.bfloat16))
    with pytest.raises(ValueError):
        ech.ech_draft_verify_ws_bytes(1, 1 << 31, 10, 1, 1)


def test_oracle_tree_attention_closed_forms():
    """A chain is the causal call; a star sees the cached tokens, its root and
    itself; a window counts positions, not rows."""
    r = np.random.default_rng(1)
    pool = wk.to_bf16_bits(r.standard_normal((64, 576)).astype(np.float32))
    q = wk.to_bf16_bits(r.standard_normal((5, 2, 576)).astype(np.float32))
    table, row0, n = np.array([[3, 1, 0, 4]]), [0, 5], [20]
    for w, s in ((0, 0), (3, 2)):
        a = oracle.drafts.attention(q, pool, table, 8, row0, n, [-1, 0, 1, 2, 3], 0.1, w, s)
        b = oracle.paged.attention(q, pool, table, 8, row0, n, 0.1, w, s)
        for x, y in zip(a, b):
            np.testing.assert_array_equal(x, y)
    zero = np.zeros_like(q)
    _, lse, _, _ = oracle.drafts.attention(zero, pool, table, 8, row0, n, [-1, 0, 0, 0, 0], 1.0)
    np.testing.assert_allclose(lse[:, 0], np.log([16, 17, 17, 17, 17]))
    _, lse, _, _ = oracle.drafts.attention(zero, pool, table, 8, row0, n, [-1, 0, 0, 1, 9], 1.0, window=2)
    np.testing.assert_allclose(lse[:, 0], np.log([2, 2, 2, 2, 2]))
    _, lse, _, _ = oracle.drafts.attention(zero, pool, table, 8, row0, n, [-1, 0, 0, 1, -1], 1.0, window=1, n_sink=16)
    np.testing.assert_allclose(lse[:, 0], np.log([16, 17, 17, 17, 16]))


def _mean_next(p_logits, parent, tokens, draft, N, vary):
    """The distribution of the first emitted token, over a grid of N values of
    each of the first `vary` random numbers, the others being 0."""
    n, V = p_logits.shape
    out = np.zeros(V)
    grid = (np.arange(N) + 0.5) / N
    for us in itertools.product(grid, repeat=vary):
        kept, nxt, _ = oracle.drafts.verify(p_logits, tokens, [0, n], [*us] + [0.0] * (n - vary), n, parent=parent, draft=draft)
        first = int(tokens[kept[0][1]]) if len(kept[0]) > 1 else nxt[0]
        out[first] += 1.0 / N ** vary
    return out


def test_oracle_verification_keeps_the_distribution_of_a_tree():
    """Three proposals, one of them twice (whatever its number): the first token
    behind the root has the root's distribution. A grid of N values is off by at
    most 1/N a decision."""
    r = np.random.default_rng(2)
    x = r.standard_normal((4, 5)).astype(np.float32) * 1.5
    w = oracle.drafts.weights(x[0], 1.0)
    N = 20
    got = _mean_next(x, [-1, 0, 0, 0], np.array([0, 3, 1, 3]), None, N, 3)
    np.testing.assert_allclose(got, w / w.sum(), atol=3 / N)
    assert abs(got.sum() - 1) < 1e-9


def test_oracle_verification_keeps_the_distribution_of_a_drawn_chain():
    r = np.random.default_rng(3)
    x = r.standard_normal((2, 5)).astype(np.float32) * 1.5
    q = np.exp(r.standard_normal((2, 5)))
    q = (q / q.sum(1, keepdims=True)).astype(np.float32)
    N, out = 60, np.zeros(5)
    for t in range(5):
        out += q[0, t] * _mean_next(x, None, np.array([0, t]), q, N, 2)
    w = oracle.drafts.weights(x[0], 1.0)
    np.testing.assert_allclose(out, w / w.sum(), atol=2 / N)


def test_oracle_verification_by_hand():
    log = np.log
    x = np.array([[log(.5), log(.3), log(.2)], [log(.1), log(.2), log(.7)], [-np.inf, 0, -np.inf], [0, 0, 0.]])
    v = lambda u, **k: oracle.drafts.verify(x, k.pop('tokens', [9, 0, 2, 1]), [0, 4], u, k.pop('most', 4), **k)[:2]  # noqa: E731
    tree = dict(parent=[-1, 0, 1, 0])
    assert v([.5, .49, .69, .9], **tree) == ([[0, 1, 2]], [1])             # row 2's only token
    assert v([.5, .51, .0, .59], **tree) == ([[0, 3]], [1])                # .3 of the .5 left; row 3: thirds, .5 in the second
    assert v([.5, .51, .0, .61], **tree) == ([[0]], [2])                   # token 2 is all that is left
    assert v([.3, .49, .71, .0], **tree) == ([[0, 1]], [0])                # .1, .2 left: .09 lies in the first
    assert v([.34, .49, .71, .0], **tree) == ([[0, 1]], [1])
    assert v([.32, .49, .71, .0], **tree) == ([[0, 1]], [0])
    assert v([.9, .0, .0, .0], most=1, **tree) == ([[0]], [2])             # untried: all of row 0
    assert v([.5, .5, .5, .5], tokens=[9, 0, 2, 0], temperature=[0.], **tree) == ([[0, 1, 2]], [1])
    assert v([.5, .99, .5, .0], tokens=[9, 7, 2, -1], **tree) == ([[0]], [1])    # no token of the vocabulary: .5 lies at the border
    q = np.full((4, 3), 1 / 3, np.float32)
    assert v([.4, .9, .5, .5], tokens=[9, 2, 0, 0], draft=q) == ([[0]], [0])  # p(2) = .2 < .9 / 3; left: 1/6 of token 0
    assert v([.4, .59, .01, .5], tokens=[9, 2, 2, 0], draft=q) == ([[0, 1, 2]], [1])
    assert oracle.drafts.verify(x[:0], [], [0, 0], [], 3)[:2] == ([[]], [-1])


def test_oracle_accept():
    pool, table = np.arange(24).reshape(24, 1).copy(), np.array([[2, 0, 1], [5, 4, 3]])
    lens = oracle.drafts.accept(pool, table, 4, [0, 5, 7], [9, 7], [[0, 2, 3], [0]])
    assert lens == [7, 6]
    np.testing.assert_array_equal(pool[[0, 1, 2, 3, 4]][:, 0], [0, 2, 3, 3, 4])
    np.testing.assert_array_equal(pool[5:, 0], np.arange(5, 24))


def test_page_tables_of_forks():
    """Shared pages are free with their last holder; a request that does not fit
    changes nothing."""
    from indexer_top_kv_amd.pipeline import PageTables
    r = np.random.default_rng(6)
    t, lens = PageTables(5, 24, 8, 9), np.zeros(5, int)
    refused = forks = 0
    for _ in range(2000):
        before = (t.table.copy(), list(t.free), t.more.copy(), t.held.copy(), t.shared)
        try:
            if r.random() < 0.3 and (lens == 0).any() and lens.any():
                src = int(r.choice(np.flatnonzero(lens)))
                dst = [int(b) for b in np.flatnonzero(lens == 0)[:int(r.integers(1, 3))]]
                share = bool(r.random() < 0.8)
                copies = t.fork(src, dst, int(lens[src]), share)
                forks += 1
                for b in dst:
                    lens[b] = lens[src]
                    full = lens[src] // 8 if share else 0
                    mine = [c for c in copies if c[1] in t.table[b, :t.held[b]]]
                    assert np.array_equal(t.table[b, :full], t.table[src, :full]) and len(mine) == -(-lens[src] // 8) - full
                    assert sum(c[2] for c in mine) == lens[src] - 8 * full
            else:
                want = np.where(r.random(5) < 0.15, 0, np.clip(lens + r.integers(-6, 14, 5), 0, 80))
                want = np.where(want < lens, np.where(want == 0, 0, lens), want)   # sequences grow or end
                t.resize(want)
                lens = want
        except ValueError:
            refused += 1
            for x, y in zip(before, (t.table, t.free, t.more, t.held, t.shared)):
                assert np.array_equal(x, y)
        used = t.table[t.table >= 0]
        pages, times = np.unique(used, return_counts=True)
        assert np.array_equal(times - 1, t.more[pages]) and t.more.sum() == (times - 1).sum() == t.shared
        assert sorted(pages.tolist() + t.free) == list(range(24))
        assert np.array_equal(t.held, t.need(lens))
    assert refused > 50 and forks > 50


def test_layer_refuses_what_drafts_do_not_allow():
    """Out of turn, with a budget, of wrong shapes: nothing moves."""
    from indexer_top_kv_amd.pipeline import PagedLayer
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    layer = PagedLayer(2, 4, n_pages=20, max_len=600, max_rows=300, page_size=16, device='cpu')
    q, rows = z(6, 4, 576, dt=torch.bfloat16), z(6, 576, dt=torch.bfloat16)
    for call in (lambda: layer.accept(z(2, 2), z(2), [0, 0]),):
        with pytest.raises(RuntimeError, match='no drafts'):
            call()
    for bad in (dict(parent=z(5)), dict(parent=z(6, dt=torch.int64)), dict(parent=z(12)[::2]), dict(counts=[3, 2])):
        a = {**dict(parent=z(6), counts=[3, 3]), **bad}
        with pytest.raises(ValueError):
            layer.draft(q, rows, a['parent'], a['counts'])
        assert layer.lens.tolist() == [0, 0] and layer._drafts is None
    with pytest.raises(ValueError, match='256'):
        layer.draft(z(257, 4, 576, dt=torch.bfloat16), z(257, 576, dt=torch.bfloat16), z(257), [257, 0])
    with pytest.raises(ValueError, match='not placed as drafts'):
        layer.place([3, 3])
        layer.launch(q, rows, parent=z(6))
    layer.place([3, 3], drafts=True)
    for call in (lambda: layer.place([1, 1]), lambda: layer.release(0), lambda: layer.fork(0, 1)):
        with pytest.raises(RuntimeError, match='accept'):
            call()
    for counts in ([4, 0], [-1, 0], [1]):
        with pytest.raises(ValueError):
            layer.accept(z(2, 3), z(2), counts)
    assert layer.lens.tolist() == [6, 6]
    with pytest.raises(ValueError, match='budget'):
        PagedLayer(1, 4, n_pages=8, max_len=64, max_rows=8, page_size=16, budget=20, device='cpu').place([1], drafts=True)
    layer = PagedLayer(4, 4, n_pages=20, max_len=600, max_rows=300, page_size=16, device='cpu')
    layer.place([20, 0, 0, 5])
    for src, dst in ((0, 0), (0, [1, 1]), (0, 3), (0, 4), (0, -1), (0, [1, 3]), (-1, 1), (4, 1)):
        with pytest.raises(ValueError, match='empty'):
            layer.fork(src, dst)
    layer.fork(0, [1, 2])
    assert layer.lens.tolist() == [20, 20, 20, 5] and layer.pages.more.sum() == 2


def test_accept_refuses_counts_that_kept_does_not_hold():
    """The device cuts n_kept at kept's width: a host that counts more would
    have lengths with rows that never moved."""
    from indexer_top_kv_amd.pipeline import PagedLayer
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    layer = PagedLayer(2, 4, n_pages=20, max_len=200, max_rows=30, page_size=16, device='cpu')
    layer.place([20, 5])
    layer.place([6, 3], drafts=True)
    image = layer._image.copy()
    for kept, counts in ((z(2, 2), [3, 0]), (z(2, 2), [0, 3]), (z(2, 1), [2, 1]), (z(2), [1, 1]), (z(1, 6), [1, 1])):
        with pytest.raises(ValueError, match='kept|counts'):
            layer.accept(kept, z(2), counts)
        assert layer._drafts.tolist() == [6, 3] and layer.lens.tolist() == [26, 8]
        np.testing.assert_array_equal(layer._image, image)
    with pytest.raises(ValueError, match='GPU'):                # nothing wrong but that these are host tensors
        layer.accept(z(2, 2), z(2), [2, 2])


def test_finish_refuses_what_cannot_be_verified_before_anything_moves():
    from indexer_top_kv_amd.pipeline import DraftStep, PagedLayer
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    layers = [PagedLayer(2, 4, n_pages=60, max_len=400, max_rows=300, page_size=16, device='cpu') for _ in range(2)]
    for layer in layers:
        layer.place([6, 3], drafts=True)
    entered = []
    for layer in layers:
        layer._enter = lambda stream=None: entered.append(stream)
    step = DraftStep(layers, 4)
    for V in ((1 << 24) + 1, 0):
        with pytest.raises(ValueError, match='2\\^24'):
            step.finish(torch.zeros(1, 1).expand(9, V), z(9), torch.zeros(9))
    with pytest.raises(ValueError, match='placed'):
        step.finish(torch.zeros(8, 50), z(8), torch.zeros(8))
    assert not entered and all(x._drafts.tolist() == [6, 3] for x in layers)


def test_a_step_names_each_layer_once():
    """Twice in the list, a layer's rows would move twice."""
    from indexer_top_kv_amd.pipeline import DraftStep, PagedLayer
    mk = lambda B=2: PagedLayer(B, 4, n_pages=8, max_len=64, max_rows=16, page_size=16, device='cpu')  # noqa: E731
    a, b = mk(), mk()
    assert len(DraftStep([a, b], 3).layers) == 2
    for layers in ([a, a], [a, b, a], [], [a, mk(3)]):
        with pytest.raises(ValueError, match='layers'):
            DraftStep(layers, 3)
