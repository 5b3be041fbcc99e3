"""The resident paged cache without a GPU: refusals of the C ABI and of the
binding, and the oracle against closed forms."""
import os
import subprocess
import sys
import warnings

import numpy as np
import pytest
import torch

import indexer_top_kv_amd as ech
import oracle
import paged_abi_checks
from oracle.numerics import bf16_to_f64
from test_abi import ROOT, _clang_rt
import workloads as wk


@pytest.mark.parametrize('check', paged_abi_checks.CHECKS, ids=lambda f: f.__name__)
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
    r = subprocess.run([sys.executable, os.path.join(ROOT, 'tests', 'paged_abi_checks.py'), lib], env=env,
                       capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and 'paged abi checks ok' in r.stdout, out[-4000:]
    assert 'AddressSanitizer' not in out and 'runtime error' not in out, out[-4000:]


def test_binding_refuses_host_tensors_types_and_shapes():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    pool, q = z(64, 576, dt=torch.bfloat16), z(2, 4, 576, dt=torch.bfloat16)
    table, row0, n = z(1, 4), z(2), z(1)
    out = z(2, 4, 512, dt=torch.bfloat16)
    with pytest.raises(ValueError):                       # host tensors
        ech.ech_paged_attn(q, pool, table, 16, row0, n, 2, 64, 0.1, out)
    with pytest.raises(TypeError):
        ech.ech_paged_attn(q, pool.float(), table, 16, row0, n, 2, 64, 0.1, out)
    with pytest.raises(ValueError):
        ech.ech_paged_append(pool, table, 16, row0, n, z(2, 576, dt=torch.bfloat16))
    with pytest.raises(ValueError):
        ech.ech_paged_weight(q, z(2, 4, dt=torch.float32), pool, table, 16, row0, n, 2, 64, 0.1, None,
                             z(1, 64, dt=torch.float32))
    with pytest.raises(ValueError):
        ech.ech_paged_evict(z(1, 64, dt=torch.float32), n, 64, 8, 0, 0, z(1, 8), z(1))
    with pytest.raises(TypeError):
        ech.ech_paged_evict(z(1, 64, dt=torch.float32), z(1, dt=torch.int64), 64, 8, 0, 0, z(1, 8), z(1))


def test_oracle_attention_closed_forms():
    """One visible token: its value row; equal scores: the mean; the window and
    the first tokens by hand."""
    r = np.random.default_rng(1)
    pool = wk.to_bf16_bits(r.standard_normal((40, 576)).astype(np.float32))
    table = np.array([[3, 1, 0, 4]])
    v = bf16_to_f64(pool)[:, :512]
    sl = oracle.paged.slots(table[0], 8, 40, 20)
    np.testing.assert_array_equal(sl[:10], [24, 25, 26, 27, 28, 29, 30, 31, 8, 9])
    q = np.zeros((3, 2, 576), np.uint16)
    out, lse, _, _ = oracle.paged.attention(q, pool, table, 8, [0, 3], [20], 1.0)
    np.testing.assert_allclose(out[2, 1], v[sl].mean(0))
    np.testing.assert_allclose(lse[:, 0], np.log([18, 19, 20]))
    out, lse, _, _ = oracle.paged.attention(q, pool, table, 8, [0, 3], [20], 1.0, window=2, n_sink=1)
    np.testing.assert_allclose(out[1, 0], v[sl[[0, 17, 18]]].mean(0))
    out, lse, _, _ = oracle.paged.attention(q, pool, table, 8, [0, 3], [20], 1.0, window=1)
    np.testing.assert_allclose(out[:, 0], v[sl[17:20]])
    out, lse, _, _ = oracle.paged.attention(q, pool, np.full((1, 4), -1), 8, [0, 3], [20], 1.0)
    assert np.all(out == 0) and np.all(np.isneginf(lse))


def test_oracle_received_weight_hands_out_one():
    r = np.random.default_rng(2)
    pool = wk.to_bf16_bits(r.standard_normal((64, 576)).astype(np.float32))
    q = wk.to_bf16_bits(r.standard_normal((5, 3, 576)).astype(np.float32))
    table, row0, n = np.arange(8).reshape(2, 4), [0, 2, 5], [30, 17]
    _, lse, _, _ = oracle.paged.attention(q, pool, table, 8, row0, n, 0.07, 6, 2)
    acc = oracle.paged.received(q, lse, pool, table, 8, row0, n, 0.07, np.zeros((2, 32)), 1.0, 6, 2)
    np.testing.assert_allclose(acc.sum(1), [2 * 3, 3 * 3])
    assert acc[0, 2:23].sum() == 0 and np.all(acc[0, :2] > 0)


def test_oracle_evict_by_brute_force():
    r = np.random.default_rng(3)
    for _ in range(200):
        n, keep = int(r.integers(0, 12)), int(r.integers(1, 9))
        sink = int(r.integers(0, keep + 1))
        recent = int(r.integers(0, keep - sink + 1))
        acc = r.integers(0, 3, (1, 12)).astype(np.float32)
        got = oracle.paged.evict(acc, [n], keep, sink, recent)[0]
        assert len(got) == min(n, keep) and np.all(np.diff(got) > 0)
        if n > keep:
            assert set(range(sink)) <= set(got) and set(range(n - recent, n)) <= set(got)
            mid = [t for t in range(sink, n - recent)]
            inn = [t for t in mid if t in got]
            for t in set(mid) - set(got):
                assert all((acc[0, u], -u) > (acc[0, t], -t) for u in inn)


def test_page_tables():
    """Pages are given, returned and never held twice; a request that does not
    fit changes nothing."""
    from indexer_top_kv_amd.pipeline import PageTables
    r = np.random.default_rng(4)
    t = PageTables(4, 20, 8, 9)
    lens = np.zeros(4, int)
    for _ in range(300):
        want = np.clip(lens + r.integers(-30, 40, 4), 0, 80)
        before = (t.table.copy(), list(t.free))
        need = -(-want // 8)
        try:
            t.resize(want)
            lens = want
        except ValueError:
            assert need.max() > 9 or need.sum() > 20
            assert np.array_equal(before[0], t.table) and before[1] == t.free
        used = t.table[t.table >= 0]
        assert len(set(used.tolist())) == len(used) and sorted(used.tolist() + t.free) == list(range(20))
        for b in range(4):
            n = -(-int(lens[b]) // 8)
            assert np.all(t.table[b, :n] >= 0) and np.all(t.table[b, n:] == -1)


def test_workspace_of_long_batches():
    """A batch whose steps would not fit the plan's 31-bit sums is not split,
    and needs no workspace; a shorter one is and does."""
    assert ech.ech_paged_attn_ws_bytes(256, 256, 128, 1, 1 << 20) > 0
    assert ech.ech_paged_attn_ws_bytes(256, 256, 128, 1, 1 << 30) == 0
    assert ech.ech_paged_attn_ws_bytes(1, 1, 128, 1, 1 << 30) > 0


def test_binding_refuses_numbers_beyond_32_bits():
    """ctypes would cut them: 2^32 + 100 tokens would have been 100."""
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    q, out, lse = z(2, 4, 576, dt=torch.bfloat16), z(2, 4, 512, dt=torch.bfloat16), z(2, 4, dt=torch.float32)
    pool, table, row0, n, acc = z(64, 576, dt=torch.bfloat16), z(1, 4), z(2), z(1), z(1, 64, dt=torch.float32)
    far = (1 << 32) + 100
    ok = dict(page_size=16, max_rows=2, max_len=64, window=0, n_sink=0)
    beyond = 'more than 32 bits'    # found before the tensors' place, the host, is
    for name in ok:
        for v in (far, -far):
            a = {**ok, name: v}
            head = (table, a['page_size'], row0, n, a['max_rows'], a['max_len'], 0.1)
            tail = dict(window=a['window'], n_sink=a['n_sink'])
            with pytest.raises(ValueError, match=beyond):
                ech.ech_paged_attn(q, pool, *head, out, **tail)
            with pytest.raises(ValueError, match=beyond):
                ech.ech_paged_weight(q, lse, pool, *head, None, acc, **tail)
            if name != 'page_size':
                with pytest.raises(ValueError, match=beyond):
                    ech.ech_paged_attn_ws_bytes(1, 2, 4, a['max_rows'], a['max_len'], **tail)
    with pytest.raises(ValueError, match=beyond):
        ech.ech_paged_append(pool, table, far, row0, n, pool[:2])
    for call in (lambda: ech.ech_paged_weight_ws_bytes(1, 2, 4, 2, far), lambda: ech.ech_paged_evict_ws_bytes(1, far, 8),
                 lambda: ech.ech_paged_evict_ws_bytes(far, 64, 8),
                 lambda: ech.ech_paged_evict(acc, n, far, 8, 0, 0, z(1, 8), z(1)),
                 lambda: ech.ech_paged_evict(acc, n, 64, 8, far, 0, z(1, 8), z(1)),
                 lambda: ech.ech_paged_evict(acc, n, 64, 8, 0, far, z(1, 8), z(1))):
        with pytest.raises(ValueError, match=beyond):
            call()


def test_layer_refuses_a_step_before_anything_moves():
    """Wrong shapes, types, places or strides: no pages, lengths or offsets
    change."""
    from indexer_top_kv_amd.pipeline import PagedLayer
    layer = PagedLayer(2, 4, n_pages=20, max_len=100, max_rows=50, page_size=16, budget=60, device='cpu')
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    layer.place([20, 3])
    lens, table = layer.lens.copy(), layer.pages.table.copy()
    row0, n = layer.row0.clone(), layer.seq_len.clone()
    bad = [(z(33, 8, 576), z(33, 576)), (z(33, 4, 512), z(33, 576)), (z(33, 4, 576), z(33, 512)),
           (z(33, 4, 576, dt=torch.float16), z(33, 576)), (z(33, 4, 576), z(33, 576, dt=torch.float16)),
           (z(33, 4, 576), z(33, 576, dt=torch.int16)), (z(33, 4, 576), z(32, 576)), (z(32, 4, 576), z(33, 576)),
           (z(33, 4, 1152)[..., ::2], z(33, 576)), (z(33, 4, 580)[..., :576], z(33, 576)),
           (z(33 * 4 * 576 + 1)[1:].view(33, 4, 576), z(33, 576)), (z(33, 4, 576), z(33, 577)[:, :576]),
           (z(33, 4, 576), z(1, 576).expand(33, -1)), (z(33, 4, 576, dt=torch.int64), z(33, 576)),
           (z(33, 4, 576).to('meta'), z(33, 576))]
    for q, x in bad:
        with pytest.raises(ValueError):
            layer.step(q, x, [1, 32])
        with pytest.raises(ValueError):
            layer.launch(q, x)
        assert np.array_equal(layer.lens, lens) and np.array_equal(layer.pages.table, table)
        assert torch.equal(layer.row0, row0) and torch.equal(layer.seq_len, n)
    with pytest.raises(ValueError, match='23 rows were placed'):
        layer.launch(z(22, 4, 576), z(22, 576))


def test_layer_calls_take_the_steps_own_bounds():
    """The kernels' forms follow from host bounds: a step gives its own largest
    count and length, not the layer's; a captured launch what place was told."""
    from indexer_top_kv_amd.pipeline import PagedLayer
    B, H = 32, 16
    layer = PagedLayer(B, H, n_pages=4096, max_len=131072, max_rows=1024, page_size=64, budget=131072, device='cpu')
    sizes = (ech.ech_paged_attn_ws_bytes, ech.ech_paged_weight_ws_bytes)
    tight = lambda R, L, T: max(f(B, T, H, R, L) for f in sizes)  # noqa: E731
    layer.place([1000] + [7] * 31)
    assert layer._bounds(False) == (1000, 1024) and layer._bounds(True) == (1024, 131072)
    layer.place([1] * B)
    assert layer._bounds(False) == (1, 1024) and layer._bounds(True) == (1024, 131072)
    assert layer._ws_bytes(B, *layer._bounds(False)) == tight(1, 1024, B)
    assert tight(1, 1024, B) != tight(32, 131072, B)
    layer.place([24] + [0] * 31, max_rows=30)
    assert layer._bounds(False) == (30, 1280) and layer._bounds(True) == (30, 131072)
    layer.place([1] * B, max_rows=np.int64(1))
    assert layer._bounds(False) == (1, 1280) and layer._bounds(True) == (1, 131072)
    assert layer._ws_bytes(B, *layer._bounds(True)) == tight(1, 131072, B) and type(layer._fixed) is int
    lens = layer.lens.copy()
    for n in (0, 1, 256, 257, 5000, 10071, 65535, 65536, 131072):
        layer.lens = np.array([n // 2] * 31 + [n])
        assert n <= layer._len_bound() <= n + max(255, n // 8)
    layer.lens = lens.copy()
    for counts, most in (([2] + [0] * 31, 1), ([1] * B, 1025), ([1] * B, 0), ([1] * B, -1)):
        with pytest.raises(ValueError):
            layer.place(counts, max_rows=most)
    assert np.array_equal(layer.lens, lens) and layer._bounds(True) == (1, 131072)
    layer.place([0] * B)
    assert layer._bounds(False) == (0, 1280)
    # 129 decoded tokens of 128 heads are split over the CUs by their own bound, not by the layer's
    H = 128
    layer = PagedLayer(129, H, n_pages=600, max_len=16384, max_rows=1024, page_size=64, device='cpu')
    layer.place([200] * 129)
    layer.place([1] * 129)
    assert layer._ws_bytes(129, *layer._bounds(False)) > 0 == ech.ech_paged_attn_ws_bytes(129, 129, H, 129, 16384)


def test_layer_warns_of_a_window_over_kept_tokens():
    from indexer_top_kv_amd.pipeline import PagedLayer
    mk = lambda **kw: PagedLayer(1, 4, n_pages=8, max_len=64, max_rows=8, page_size=16, device='cpu', **kw)  # noqa: E731
    with pytest.warns(UserWarning, match='window'):
        mk(window=20, n_sink=2, budget=40, n_recent=18)
    with warnings.catch_warnings():
        warnings.simplefilter('error')
        mk(window=20, n_sink=2, budget=40, n_recent=19)
        mk(window=20, n_sink=2)
        mk(budget=40)
        mk(window=1, budget=40)
