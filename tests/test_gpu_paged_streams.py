"""PagedLayer over several streams: its calls run in their order whatever
streams they name, and its buffers take no memory that another stream still
uses. A step on one stream is the reference; results have to be the same bits."""
import numpy as np
import pytest
import torch

import workloads as wk
from gpu_util import dev, need_gpu
from indexer_top_kv_amd.pipeline import PagedLayer

pytestmark = pytest.mark.gpu
WAIT = 1_000_000    # cycles of a bounded spin: long beside a step, milliseconds at most


def bits(r, *shape):
    return dev(wk.to_bf16_bits(r.standard_normal(shape).astype(np.float32))).view(torch.bfloat16)


def test_calls_on_changing_streams_run_in_order():
    """place on the current stream, launch and trim on others, each stream kept
    busy before the call: lengths, tables, weights, rows and outputs as with
    one stream. The budget is a whole number of pages, so that some evictions
    change no table."""
    need_gpu()
    r = np.random.default_rng(21)
    mk = lambda: PagedLayer(2, 16, n_pages=60, max_len=400, max_rows=80, page_size=16, budget=64, n_sink=2,  # noqa: E731
                            n_recent=8, decay=0.5)
    a, b = mk(), mk()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    steps = [[70, 3], [1, 1], [1, 61], [2, 1], [1, 1], [0, 1], [5, 60], [1, 1], [1, 1]]
    for i, counts in enumerate(steps):
        T = sum(counts)
        q, x = bits(r, T, 16, 576), bits(r, T, 576)
        torch.cuda.synchronize()            # q and x are there for every stream
        for st in sides:
            with torch.cuda.stream(st):
                torch.cuda._sleep(WAIT)
        a.place(counts)
        out, lse = a.launch(q, x, stream=sides[i % 2])
        a.trim(stream=(None, sides[0], sides[1])[i % 3])
        want = b.step(q, x, counts)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i
        for name in ('acc', 'seq_len', 'table', 'pool', 'row0'):
            assert torch.equal(getattr(a, name), getattr(b, name)), (i, name)
        assert a.lens.tolist() == b.lens.tolist() == b.seq_len.tolist()
    a.release(0)
    a.place([1, 0])
    assert a.device.index == a.pool.device.index is not None


def test_a_launch_elsewhere_takes_no_memory_still_in_use():
    """A chunk's outputs may get memory that was freed while the current stream
    has yet to read it: the launch's stream waits for that."""
    need_gpu()
    r = np.random.default_rng(22)
    layer = PagedLayer(2, 16, n_pages=20, max_len=300, max_rows=64, page_size=16)
    side, T = torch.cuda.Stream(), 40
    q, x = bits(r, T, 16, 576), bits(r, T, 576)
    layer.place([T, 0])
    torch.cuda.synchronize()
    old = torch.full((T, 16, 512), 5.0, dtype=torch.bfloat16, device='cuda')
    seen = torch.empty_like(old)
    torch.cuda._sleep(WAIT)
    seen.copy_(old)
    del old
    out, _ = layer.launch(q, x, stream=side)
    torch.cuda.synchronize()
    assert torch.all(seen == 5.0) and not torch.any(torch.isnan(out))


def test_streams_by_handle():
    """Streams named by their handles, the default stream's 0 among them; one
    that torch does not own is waited for by an event of its own."""
    need_gpu()
    r = np.random.default_rng(23)
    a, b = (PagedLayer(2, 16, n_pages=60, max_len=400, max_rows=80, page_size=16, budget=64, n_recent=8)
            for _ in range(2))
    side = torch.cuda.Stream()
    foreign = torch.cuda.ExternalStream(side.cuda_stream)
    for i, counts in enumerate([[70, 3], [1, 62], [1, 1], [3, 3], [1, 1], [20, 1], [1, 1]]):
        T = sum(counts)
        q, x = bits(r, T, 16, 576), bits(r, T, 576)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(WAIT)
        torch.cuda._sleep(WAIT)
        a.place(counts)
        out, lse = a.launch(q, x, stream=(0, side.cuda_stream, foreign)[i % 3])
        a.trim(stream=(side.cuda_stream, 0)[i % 2])
        want = b.step(q, x, counts)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i
        for name in ('acc', 'seq_len', 'table', 'pool'):
            assert torch.equal(getattr(a, name), getattr(b, name)), (i, name)
    assert (a._done is None) == (a._last in (0, None))


def test_the_host_does_not_wait_for_the_device():
    """Steps with new pages and evictions are queued behind a busy device; its
    lengths, tables and results are those of steps that are waited for, after
    more uploads than can be under way as well."""
    need_gpu()
    r = np.random.default_rng(24)
    a, b = (PagedLayer(2, 16, n_pages=60, max_len=400, max_rows=80, page_size=16, budget=64, n_recent=8)
            for _ in range(2))
    steps = [[70, 3], [1, 62], [1, 20], [3, 30]]
    rows = [(bits(r, sum(c), 16, 576), bits(r, sum(c), 576)) for c in steps]
    for q, x in rows:                       # the blocks and buffers exist
        a.step(q, x, [len(x) - 1, 1])
        b.step(q, x, [len(x) - 1, 1])
    torch.cuda.synchronize()
    busy = torch.cuda.Event()
    torch.cuda._sleep(60 * WAIT)
    busy.record()
    got = []
    for counts, (q, x) in zip(steps[:3], rows):
        got.append(a.step(q, x, counts))
        assert a.lens.max() <= 64
    assert not busy.query()                 # three steps, three evictions: all queued, none begun
    for i in range(30):
        counts, (q, x) = steps[i % 4], rows[i % 4]
        got.append(a.step(q, x, counts))
    torch.cuda.synchronize()
    order = list(zip(steps[:3], rows)) + [(steps[i % 4], rows[i % 4]) for i in range(30)]
    for i, (counts, (q, x)) in enumerate(order):
        out, lse = b.step(q, x, counts)
        torch.cuda.synchronize()
        assert torch.equal(out, got[i][0]) and torch.equal(lse, got[i][1]), i
    for name in ('acc', 'seq_len', 'table', 'pool', 'row0'):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    assert a.seq_len.tolist() == a.lens.tolist() and np.array_equal(a.table.cpu().numpy(), a.pages.table)


def test_the_hosts_part_is_not_captured():
    need_gpu()
    r = np.random.default_rng(25)
    layer = PagedLayer(2, 16, n_pages=60, max_len=400, max_rows=80, page_size=16, budget=64)
    layer.place([80, 0])
    layer.launch(bits(r, 80, 16, 576), bits(r, 80, 576))
    q, x = bits(r, 1, 16, 576), bits(r, 1, 576)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in (lambda: layer.place([1, 0]), layer.trim, lambda: layer.release(0), lambda: layer.step(q, x, [0, 1])):
            with pytest.raises(RuntimeError, match='captured'):
                call()
        y = q * 2
    assert layer.lens.tolist() == [80, 0] and layer.seq_len.tolist() == [80, 0]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, q * 2) and layer.trim() and layer.lens.tolist() == [64, 0]


def test_a_chunks_workspace_lives_until_its_stream_is_done():
    """The layer drops a chunk's workspace when launch returns, while the side
    stream has not begun: allocations of its size, filled at once, must not get
    its memory. Against a second layer on the current stream."""
    need_gpu()
    r = np.random.default_rng(26)
    a, b = (PagedLayer(2, 16, n_pages=100, max_len=700, max_rows=64, page_size=16, budget=600) for _ in range(2))
    side = torch.cuda.Stream()
    for counts in ([64, 30], [64, 3], [64, 64], [64, 0], [40, 2], [33, 1], [17, 64], [64, 64]):
        T = sum(counts)
        q, x = bits(r, T, 16, 576), bits(r, T, 576)
        a.place(counts)
        size = a._ws_bytes(T, *a._bounds(False))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(10 * WAIT)
        out, lse = a.launch(q, x, stream=side)
        junk = [torch.full((max(size, 1),), 0xff, dtype=torch.uint8, device='cuda') for _ in range(3)]   # NaN patterns
        torch.cuda.current_stream().synchronize()
        want = b.step(q, x, counts)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(a.acc, b.acc)
        assert a.lens.max() < 128 or size > 0
        del junk
    assert torch.equal(a.pool, b.pool) and not a._ws
