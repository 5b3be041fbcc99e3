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
