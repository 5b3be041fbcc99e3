r"""One layer of the path, launched in order on up to three streams.

Decode step (ECHO explainer, "The top-k dependency" and "Decode: fetch above
a predicted threshold"): the recall of a step depends on its top-k; the early
fetch of tokens scoring above the predicted threshold starts before it:

    S0: ech_index_logits --> ech_topk(theta -> theta') --> FINAL maps --> FINAL recall
         \-> S1: EARLY(theta) maps -----/--> EARLY recall (PCIe) ----/

With fp8 keys the scores and the early fetch are one launch
(ech_index_logits_early): the early misses of a sequence get their slots, and
their rows start crossing PCIe, while later sequences are still being scored;
a copier on S1 takes them as they appear and, once S0 has the FINAL maps,
goes on to the FINAL rows with the link still busy:

    S0: scores + EARLY maps + band lists (one launch) --> ech_topk_early --> FINAL maps --> rest of both lists
    S1: live copier: early rows as allocated, then the FINAL rows ---------------------------/

theta is double-buffered (the early fetch reads the prediction while the
top-k writes its update). When the batch's
selections do not fit the cache at once (sum of min(k, len_b) > C),
sequences are processed in host-computed chunks, each an ECH_EARLY phase
then a FINAL phase; every selected token is resident at the end of its chunk.

Several layers (DecodeStack): one DecodeLayer per (layer, micro-batch), the
layers of a micro-batch in order, two micro-batches interleaved so that one
crosses PCIe while the other scores.

Prefill (ECHO explainer, "Prefill: one-round histogram"): query blocks are
scored one after another; the recall of block i runs on S1 while S0 scores
block i+1.

Resident layers (PagedLayer): a layer whose rows all stay on the device, in
pages of a pool (contexts below k tokens, where a selection would take every
token anyway; windowed layers; caches held to a budget of tokens). One step
takes any mix of prompt chunks and single tokens: append, attention over the
pages, and with a budget the received weights and the eviction by them. Steps
over drafted tokens bring trees of rows (draft), which DraftStep decides once
for all layers of a model and accept compacts; sequences fork with shared pages.

Nothing here computes: this module sizes buffers with torch, chooses the
order of the C-ABI calls and the stream events between them.
"""
from __future__ import annotations

import warnings
from typing import List, NamedTuple, Optional, Tuple

import numpy as np
import torch

from . import (ECH_EARLY, ECH_FINAL, ECH_PREFILL, LayerState, ech_cache_reset, ech_cache_step,
               ech_cache_step_ws_bytes, ech_index_logits, ech_index_logits_causal, ech_index_logits_early,
               ech_index_logits_early_ws_bytes, ech_kv_append, ech_recall, ech_recall_early_live, ech_recall_rest,
               ech_topk, ech_topk_early, ech_topk_ws_bytes, ech_paged_append, ech_paged_attn,
               ech_paged_attn_ws_bytes, ech_paged_evict, ech_paged_evict_ws_bytes, ech_paged_weight,
               ech_paged_weight_ws_bytes, ech_paged_tree_attn, ech_paged_tree_attn_ws_bytes, ech_paged_accept, ech_paged_copy, ech_draft_verify,
               ech_draft_verify_ws_bytes, _raw_stream, _stream)


def round_up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


def sequence_groups(B: int, groups: int) -> List[Tuple[int, int]]:
    """Split sequences 0..B-1 into at most `groups` consecutive ranges of
    nearly equal size."""
    g = max(1, min(int(groups), B))
    bounds = [round(i * B / g) for i in range(g + 1)]
    return [(bounds[i], bounds[i + 1]) for i in range(g) if bounds[i + 1] > bounds[i]]


def sequence_chunks(lens: np.ndarray, k: int, C: int) -> List[Tuple[int, int]]:
    """Split sequences into consecutive chunks, each the longest prefix of the
    remaining ones with sum(min(k, len_b)) <= C."""
    out, b0, acc = [], 0, 0
    for b, n in enumerate(np.asarray(lens).tolist()):
        d = min(k, int(n))
        if d > C:
            raise ValueError(f'one sequence needs {d} slots, the cache has {C}')
        if acc + d > C:
            out.append((b0, b))
            b0, acc = b, 0
        acc += d
    out.append((b0, len(lens)))
    return out


class DecodeLayer:
    """Buffers and launch order of one layer's decode step."""

    def __init__(self, kcache: torch.Tensor, kscale: Optional[torch.Tensor], w: torch.Tensor,
                 tok0: np.ndarray, lens: np.ndarray, C: int, k: int = 2048, cap: int = 512,
                 host_pool: Optional[torch.Tensor] = None, early: bool = True, topk_after_early: bool = False,
                 topk_first: Optional[bool] = None, fused: Optional[bool] = None,
                 capacity: Optional[np.ndarray] = None, device='cuda'):
        self.kcache, self.kscale, self.w = kcache, kscale, w
        self.topk_after_early = topk_after_early
        # Launch order of the two branches after the scores. A captured graph
        # keeps the branch launched first on the scores kernel's hardware
        # queue; the other starts after a cross-queue wait (~10 us). With a
        # few sequences the top-k chain is the longer branch, with many the
        # EARLY maps and their PCIe recall are.
        self.topk_first = (len(lens) <= 8) if topk_first is None else bool(topk_first)
        self.B = len(lens)
        self.lens_np = np.asarray(lens, np.int32)
        self.tok0_np = np.asarray(tok0, np.int64)
        # Growing contexts: sequence b may reach capacity[b] tokens (ech_kv_append
        # grows the device lengths); grids, buffers and chunks are sized for it.
        self.cap_np = self.lens_np.copy() if capacity is None else np.asarray(capacity, np.int32)
        if np.any(self.cap_np < self.lens_np):
            raise ValueError('capacity below the current length')
        self.max_len = int(self.cap_np.max())
        self.k, self.cap, self.C = k, cap, C
        self.early = early
        self.P = kcache.shape[0]
        dev = dict(device=device)
        self.tok0 = torch.from_numpy(self.tok0_np).to(**dev)
        self.lens = torch.from_numpy(self.lens_np).to(**dev)
        self.ld = round_up(max(self.max_len, 4), 64)
        self.logits = torch.zeros((self.B, self.ld), dtype=torch.float32, **dev)
        self.idx = torch.empty((self.B, k), dtype=torch.int32, **dev)
        self.kth = torch.empty(self.B, dtype=torch.float32, **dev)
        self.theta = [torch.full((self.B,), float('nan'), dtype=torch.float32, **dev) for _ in range(2)]
        self.parity = 0
        self.sel_slot = torch.empty((self.B, k), dtype=torch.int32, **dev)
        self.stats_early = torch.zeros((self.B, 4), dtype=torch.int32, **dev)
        self.stats_final = torch.zeros((self.B, 4), dtype=torch.int32, **dev)
        self.chunks = sequence_chunks(self.cap_np, k, C)
        self.seq_cap = torch.from_numpy(self.cap_np).to(**dev)
        cb = max(e - s for s, e in self.chunks)
        m_max = max(cb * min(k, self.max_len), cb * min(cap, self.max_len), 1)
        m_early = max(cb * min(cap, self.max_len), 1)   # the EARLY demand bound: no free slot beyond it is ranked
        self.state = LayerState.allocate(self.P, C, m_max, device, M_early=m_early)
        self.ws_topk = torch.empty(ech_topk_ws_bytes(self.B, self.max_len, k), dtype=torch.uint8, **dev)
        self.ws_early = torch.empty(ech_cache_step_ws_bytes(ECH_EARLY, cb, cb, k, self.max_len, C, m_max),
                                    dtype=torch.uint8, **dev)
        self.ws_final = torch.empty(ech_cache_step_ws_bytes(ECH_FINAL, cb, cb, k, self.max_len, C, m_max),
                                    dtype=torch.uint8, **dev)
        # Scores fused with the first chunk's early fetch: fp8 keys, a host
        # pool to copy from, and the early fetch on. By default only for
        # batches of more than 8 sequences: a sequence's early fetch starts
        # once its whole row is scored, so with a few long rows the fused
        # launch ends late (4 x 1M tokens: 261 us per step fused, 208 us
        # not), while with many rows their early rows cross PCIe under the
        # scoring (32 x 131072: 405 us vs 441 us; 64 x 110K: 2.06 vs 2.10 ms).
        can_fuse = early and host_pool is not None and kscale is not None and cap <= 4096
        self.fused = (can_fuse and self.B > 8) if fused is None else bool(fused)
        if self.fused and not can_fuse:
            raise ValueError('the fused scores + early fetch needs fp8 keys, a host pool, the early fetch and '
                             'cap <= 4096')
        if self.fused:
            # zero-filled once; every call leaves it ready for the next
            self.ws_fused = torch.zeros(ech_index_logits_early_ws_bytes(self.B, self.max_len, C, m_early),
                                        dtype=torch.uint8, **dev)
        self.host_pool = host_pool
        if host_pool is not None:
            self.dev_cache = torch.zeros((C, host_pool.shape[1]), dtype=host_pool.dtype, **dev)
        else:
            self.dev_cache = None
        self.s1 = torch.cuda.Stream(device=device)
        self.ev_fork = torch.cuda.Event()
        self.ev_logits = torch.cuda.Event()
        self.ev_early_maps = torch.cuda.Event()
        self.ev_early = torch.cuda.Event()
        ech_cache_reset(self.state)

    def reset(self) -> None:
        ech_cache_reset(self.state)
        for t in self.theta:
            t.fill_(float('nan'))
        self.parity = 0

    def _maps(self, phase: int, b0: int, b1: int, theta: torch.Tensor, stream) -> None:
        stats = self.stats_early if phase == ECH_EARLY else self.stats_final
        ech_cache_step(phase, self.state, self.tok0[b0:b1], self.lens[b0:b1], self.max_len,
                       idx=self.idx[b0:b1] if phase == ECH_FINAL else None, k=self.k,
                       logits=self.logits[b0:b1], theta=theta[b0:b1], cap=self.cap,
                       sel_slot=self.sel_slot[b0:b1] if phase == ECH_FINAL else None, stats=stats[b0:b1],
                       ws=self.ws_early if phase == ECH_EARLY else self.ws_final, stream=stream)

    def _recall(self, phase: int, stream) -> None:
        if self.host_pool is not None:
            ech_recall(self.host_pool, self.dev_cache, self.state, phase=phase, stream=stream)

    def append(self, new_rows: torch.Tensor, new_keys: torch.Tensor, new_scales: Optional[torch.Tensor] = None,
               stream=None) -> None:
        """Each sequence's decoded token joins the host pool and the key cache
        (ech_kv_append); the device lengths grow by one, up to the capacity."""
        ech_kv_append(self.host_pool, self.kcache, self.kscale, self.state, self.tok0, self.lens, self.seq_cap,
                      new_rows, new_keys, new_scales, stream=stream)

    def logits_only(self, q: torch.Tensor, stream=None) -> None:
        ech_index_logits(q, self.w, self.kcache, self.kscale, self.tok0, self.lens, self.max_len, self.logits,
                         stream=stream)

    def scores_launch(self, q: torch.Tensor, stream=None, mark=None) -> None:
        """The first launches of a step: the scores, and with the fused path
        also the first chunk's early fetch (its maps, written while the
        scoring runs) and, on S1, the live copy of its rows. `mark(name,
        stream)`, when given, records the copier's span as 'recall_live'."""
        if self.fused:
            s0 = torch.cuda.current_stream() if stream is None else stream
            self.ev_fork.record(s0)
            b0, b1 = self.chunks[0]
            ech_index_logits_early(q, self.w, self.kcache, self.kscale, self.tok0, self.lens, self.max_len,
                                   self.logits, b0, b1, self.theta[self.parity], self.cap, self.state,
                                   self.stats_early, self.ws_fused, stream=s0)
            # enqueued after the fused launch, waiting only for the step's start
            self.s1.wait_event(self.ev_fork)
            if mark is not None:
                mark('recall_live', self.s1)
            ech_recall_early_live(self.host_pool, self.dev_cache, self.state, self.ws_fused, stream=self.s1,
                                  final=True)
            if mark is not None:
                mark('recall_live', self.s1)
        else:
            self.logits_only(q, stream=stream)

    def step(self, q: Optional[torch.Tensor], marks: Optional[dict] = None,
             wait: Optional[torch.cuda.Event] = None, logits_done: Optional[torch.cuda.Event] = None,
             scores: bool = True, on_chunk=None) -> None:
        """Enqueue one decode step for query q [B, 64, 128] (bf16 bits) on the
        current stream (with S1 forked and joined inside). `marks`, when given,
        receives timing events recorded on the stream of each stage, as
        (start, end) pairs: logits, topk, final (S0: FINAL maps to the end of
        the step), early (S1: EARLY maps and recall of the first chunk), and
        early_maps, recall_early, final_maps, recall_final (one pair per
        chunk). `wait`, when given, is an event the scores wait for;
        `logits_done` is recorded once they are written (one group only).
        scores=False leaves the scores out: the caller has launched them
        (scores_launch) on the current stream already (q is then unused).

        on_chunk(b0, b1, stream), when given, is called once per sequence
        chunk, right after the chunk's FINAL recall is enqueued on `stream`:
        work the caller enqueues there (the attention over sel_slot[b0:b1])
        sees every selected token of sequences b0..b1-1 resident in the
        slot sel_slot names. When the batch's selections exceed the cache
        (several chunks), a later chunk's FINAL phase may evict an earlier
        chunk's tokens, so an earlier chunk's sel_slot rows are only valid
        until then: read them in on_chunk. With one chunk they stay valid
        until the next step."""
        s0 = torch.cuda.current_stream()
        if wait is not None:
            s0.wait_event(wait)

        def mark(name, stream):
            if marks is None:
                return None
            ev = torch.cuda.Event(enable_timing=True)
            ev.record(stream)
            marks.setdefault(name, []).append(ev)
            return ev

        th, th_next = self.theta[self.parity], self.theta[1 - self.parity]
        if scores:
            mark('logits', s0)
            self.scores_launch(q, stream=s0, mark=mark if marks is not None else None)
            mark('logits', s0)
        if logits_done is not None:
            logits_done.record(s0)
        first_b0, first_b1 = self.chunks[0]
        if self.early:
            self.ev_logits.record(s0)
        if self.fused:
            self._after_fused(th, th_next, s0, mark)   # the first chunk's FINAL recall included
        else:
            self._after_scores(th, th_next, s0, mark)
            mark('recall_final', s0)
            self._recall(ECH_FINAL, s0)
            mark('recall_final', s0)
        if on_chunk is not None:
            on_chunk(first_b0, first_b1, s0)
        for b0, b1 in self.chunks[1:]:
            for phase in ((ECH_EARLY, ECH_FINAL) if self.early else (ECH_FINAL,)):
                name = 'early' if phase == ECH_EARLY else 'final'
                mark(name + '_maps', s0)
                self._maps(phase, b0, b1, th, s0)
                mark(name + '_maps', s0)
                mark('recall_' + name, s0)
                self._recall(phase, s0)
                mark('recall_' + name, s0)
            if on_chunk is not None:
                on_chunk(b0, b1, s0)
        mark('final', s0)
        self.parity ^= 1

    def _after_fused(self, th, th_next, s0, mark) -> None:
        """First chunk after the fused launch: the top-k and the FINAL maps
        on S0, while on S1 the live copier goes on from the early rows to the
        FINAL ones as soon as S0 has completed the FINAL list. S0 then waits
        for the copier and copies what it left of both lists in one launch
        (ech_recall_rest)."""
        first_b0, first_b1 = self.chunks[0]
        mark('topk', s0)
        # from the band lists the scoring waves wrote (the scores are not read again)
        ech_topk_early(self.logits, self.lens, self.max_len, self.k, th, th_next, self.idx, self.kth, self.state,
                       self.ws_fused, stream=s0)
        mark('topk', s0)
        self.ev_early.record(self.s1)              # the copier is done
        mark('final', s0)
        mark('final_maps', s0)
        self._maps(ECH_FINAL, first_b0, first_b1, th, s0)
        mark('final_maps', s0)
        s0.wait_event(self.ev_early)
        mark('recall_final', s0)
        ech_recall_rest(self.host_pool, self.dev_cache, self.state, stream=s0)
        mark('recall_final', s0)

    def _after_scores(self, th, th_next, s0, mark) -> None:
        """First chunk after the plain scores: the EARLY maps and recall on
        S1 beside the top-k on S0, then the FINAL maps; ends with S0 waiting
        for the early rows."""
        first_b0, first_b1 = self.chunks[0]

        def early_branch():
            # S1: EARLY maps, then its rows cross PCIe while S0 carries on.
            self.s1.wait_event(self.ev_logits)
            mark('early', self.s1)
            mark('early_maps', self.s1)
            self._maps(ECH_EARLY, first_b0, first_b1, th, self.s1)
            mark('early_maps', self.s1)
            self.ev_early_maps.record(self.s1)
            mark('recall_early', self.s1)
            self._recall(ECH_EARLY, self.s1)
            mark('recall_early', self.s1)
            mark('early', self.s1)
            self.ev_early.record(self.s1)

        def topk_branch():
            # The top-k runs beside the EARLY maps (or after them, on request).
            if self.early and self.topk_after_early:
                s0.wait_event(self.ev_early_maps)
            mark('topk', s0)
            ech_topk(self.logits, self.lens, self.max_len, self.k, th, th_next, self.idx, self.kth, self.ws_topk,
                     stream=s0)
            mark('topk', s0)

        if self.early and not (self.topk_first and not self.topk_after_early):
            early_branch()
            topk_branch()
        else:
            topk_branch()
            if self.early:
                early_branch()
        mark('final', s0)
        if self.early and not self.topk_after_early:
            s0.wait_event(self.ev_early_maps)      # FINAL updates the maps EARLY left ...
        mark('final_maps', s0)
        self._maps(ECH_FINAL, first_b0, first_b1, th, s0)
        mark('final_maps', s0)
        if self.early:
            s0.wait_event(self.ev_early)           # ... but may reuse a slot EARLY is still filling

    @property
    def theta_current(self) -> torch.Tensor:
        return self.theta[self.parity]

    def capture(self, scores: bool = True) -> None:
        """Capture one decode step per threshold parity as a hipGraph that
        reads q from a static buffer (every tensor of the step has a fixed
        size and address, so the step replays unchanged). Nothing runs.
        scores=False captures the step after the scores (replay_after_scores);
        not with the fused path, whose live copier (launched with the scores)
        must precede the early rest and FINAL recalls of the same step: a
        graph of the rest alone would not wait for it."""
        if self.fused and not scores:
            raise ValueError('the fused path captures whole steps only (the scores launch starts the copier)')
        self.q_static = torch.zeros((self.B, 64, 128), dtype=torch.int16, device=self.logits.device)
        self.graphs = [None, None]
        self.graph_scores = scores
        for _ in range(2):
            p = self.parity
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self.step(self.q_static if scores else None, scores=scores)      # flips self.parity
            self.graphs[p] = g

    def replay(self, q: torch.Tensor) -> None:
        """One decode step through the captured graphs (on the current stream)."""
        if not self.graph_scores:
            raise ValueError('captured without the scores: use replay_after_scores')
        self.q_static.copy_(q, non_blocking=True)
        self.graphs[self.parity].replay()
        self.parity ^= 1

    def replay_after_scores(self) -> None:
        """The rest of a decode step through graphs captured with
        scores=False, after the caller's ech_index_logits on the current
        stream."""
        if self.graph_scores:
            raise ValueError('captured with the scores: use replay')
        self.graphs[self.parity].replay()
        self.parity ^= 1


class PrefillLayer:
    """Causal prefill of one sequence in query blocks: logits -> per-row top-k
    -> PREFILL cache step (union) -> recall of block i on S1 while S0 scores
    block i+1.

    With overlap=True the score buffer is doubled: S0 scores block i+1 into
    one buffer while S1 runs block i's top-k and cache step on the other
    (recalls on S2), so the selection work hides under the next block's
    matrix-core work."""

    def __init__(self, kcache: torch.Tensor, kscale: Optional[torch.Tensor], N: int, C: int, k: int = 2048,
                 block_rows: int = 4096, host_pool: Optional[torch.Tensor] = None, tok0: int = 0,
                 overlap: bool = False, device='cuda'):
        self.kcache, self.kscale = kcache, kscale
        self.N, self.C, self.k, self.block_rows, self.tok0 = N, C, k, block_rows, tok0
        self.overlap = overlap
        dev = dict(device=device)
        self.ld = round_up(N, 64)
        nbuf = 2 if overlap else 1
        self.logits_buf = [torch.empty((block_rows, self.ld), dtype=torch.float32, **dev) for _ in range(nbuf)]
        self.logits = self.logits_buf[0]
        self.idx = torch.empty((block_rows, k), dtype=torch.int32, **dev)
        self.kth = torch.empty(block_rows, dtype=torch.float32, **dev)
        self.theta = torch.full((block_rows,), float('nan'), dtype=torch.float32, **dev)
        self.sel_slot = torch.empty((block_rows, k), dtype=torch.int32, **dev)
        self.stats = torch.zeros((1, 4), dtype=torch.int32, **dev)
        self.m_max = min(N, block_rows * k)
        self.state = LayerState.allocate(N + tok0, C, self.m_max, device)
        self.ws_topk = torch.empty(ech_topk_ws_bytes(block_rows, N, k), dtype=torch.uint8, **dev)
        self.ws_cache = torch.empty(ech_cache_step_ws_bytes(ECH_PREFILL, 1, block_rows, k, N, C, self.m_max),
                                    dtype=torch.uint8, **dev)
        self.seq_tok0 = torch.tensor([tok0], dtype=torch.int64, **dev)
        self.seq_len = torch.tensor([N], dtype=torch.int32, **dev)
        self.row_len = torch.arange(1, block_rows + 1, dtype=torch.int32, **dev)
        self._row_lens = {}
        self.host_pool = host_pool
        self.dev_cache = (torch.zeros((C, host_pool.shape[1]), dtype=host_pool.dtype, **dev)
                          if host_pool is not None else None)
        self.s1 = torch.cuda.Stream(device=device)
        self.s2 = torch.cuda.Stream(device=device) if overlap else None
        self.ev_recall = torch.cuda.Event()
        self.ev_scored = [torch.cuda.Event() for _ in range(nbuf)]
        self.ev_used = [torch.cuda.Event() for _ in range(nbuf)]
        self.nblock = 0
        ech_cache_reset(self.state)

    def blocks(self):
        return [(r0, min(self.block_rows, self.N - r0)) for r0 in range(0, self.N, self.block_rows)]

    def reset_state(self) -> None:
        """Start the sequence again: empty cache, no threshold predictions."""
        ech_cache_reset(self.state)
        self.theta.fill_(float('nan'))
        self.nblock = 0

    def _row_len(self, row0: int, R: int) -> torch.Tensor:
        key = (row0, R)
        if key not in self._row_lens:
            self._row_lens[key] = self.row_len[:R] + row0
        return self._row_lens[key]

    def run_block(self, row0: int, q: torch.Tensor, w: torch.Tensor, first: bool, mark=None,
                  stage_marks: Optional[dict] = None) -> None:
        """q [R,64,128], w [R,64] for rows row0 .. row0+R-1, on the current
        stream. `mark`, when given, receives a (start, end) event pair around
        the scoring launch; `stage_marks`, when given, receives (start, end)
        pairs recorded on each stage's own stream under 'topk', 'cache' and
        'recall'."""

        def smark(name, stream):
            if stage_marks is not None:
                ev = torch.cuda.Event(enable_timing=True)
                ev.record(stream)
                stage_marks.setdefault(name, []).append(ev)

        s0 = torch.cuda.current_stream()
        R = q.shape[0]
        buf = self.nblock % len(self.logits_buf) if self.overlap else 0
        logits = self.logits_buf[buf][:R]
        self.logits = self.logits_buf[buf]
        row_len = self._row_len(row0, R)
        if self.overlap and self.nblock >= 2:
            s0.wait_event(self.ev_used[buf])      # the top-k two blocks back has read this buffer
        if mark is not None:
            ev = torch.cuda.Event(enable_timing=True)
            ev.record(s0)
            mark.append(ev)
        ech_index_logits_causal(q, w, self.kcache, self.kscale, self.tok0, row0, logits, stream=s0)
        if mark is not None:
            ev = torch.cuda.Event(enable_timing=True)
            ev.record(s0)
            mark.append(ev)
        self.nblock += 1
        if self.overlap:
            self.ev_scored[buf].record(s0)
            sel = self.s1
            sel.wait_event(self.ev_scored[buf])
        else:
            sel = s0
        # rows' thresholds: the EMA of the same row position in earlier blocks
        smark('topk', sel)
        ech_topk(logits, row_len, row0 + R, self.k, self.theta[:R], self.theta[:R], self.idx[:R], self.kth[:R],
                 self.ws_topk, stream=sel)
        smark('topk', sel)
        if self.overlap:
            self.ev_used[buf].record(sel)
        if not first:
            sel.wait_event(self.ev_recall)
        smark('cache', sel)
        ech_cache_step(ECH_PREFILL, self.state, self.seq_tok0, self.seq_len, self.N, idx=self.idx[:R], k=self.k,
                       sel_slot=self.sel_slot[:R], stats=self.stats, ws=self.ws_cache, stream=sel)
        smark('cache', sel)
        if self.host_pool is not None:
            rs = self.s2 if self.overlap else self.s1
            rs.wait_stream(sel)
            smark('recall', rs)
            ech_recall(self.host_pool, self.dev_cache, self.state, phase=ECH_PREFILL, stream=rs)
            smark('recall', rs)
            self.ev_recall.record(rs)
        else:
            self.ev_recall.record(sel)

    def finish(self) -> None:
        s0 = torch.cuda.current_stream()
        s0.wait_event(self.ev_recall)
        if self.overlap:
            s0.wait_stream(self.s1)


class DecodeStack:
    """One decode step over L layers for M micro-batches of the batch.

    Each (layer, micro-batch) pair is a DecodeLayer of its own: its slot map
    and device cache (the layer's cache split between the micro-batches),
    reading the layer's indexer keys and host pool at its sequences' token
    offsets. The cache is per layer because each layer's indexer selects its
    own tokens (ECHO explainer, "One layer, one step").

    Within a micro-batch the layers run in order: layer l+1 scores only after
    layer l's recall, because in the model the attention over the recalled
    rows stands between them and yields the next layer's query. The
    micro-batches are independent chains on streams of their own, started
    one score launch apart, so while one micro-batch's rows cross PCIe the
    other one scores:

        mb0: logits L0 | maps, recall L0 ............ | logits L1 | ...
        mb1:           | logits L0 | maps, recall L0 ............ | logits L1

    The queries of every layer are inputs of the step (no attention or MLP is
    computed between layers): qs[l][m] is DecodeLayer l, m's [B_m, 64, 128].
    """

    def __init__(self, layers: List[List[DecodeLayer]], device='cuda'):
        self.layers = [list(r) for r in layers]
        self.L, self.M = len(self.layers), (len(self.layers[0]) if self.layers else 0)
        if self.L == 0 or self.M == 0 or any(len(r) != self.M for r in self.layers):
            raise ValueError('layers must be a non-empty L x M list of DecodeLayer')
        # The stack launches each pair's scores itself and replays graphs of
        # the rest, which the fused path cannot split (see capture); it is
        # also slower here (4 layers x 2 micro-batches of 16 sequences: 471
        # us per layer fused, 408 us not).
        if any(d.fused for r in self.layers for d in r):
            raise ValueError('DecodeStack takes layers built with fused=False')
        # Two streams per micro-batch (scores and its chain; EARLY branch),
        # shared by its layers; micro-batch 0's chain is the caller's stream.
        # With two micro-batches these are four streams, one per hardware
        # queue at the runtime's default of four, so neither micro-batch
        # waits behind the other's work in a shared queue.
        self.streams = [None] + [torch.cuda.Stream(device=device) for _ in range(self.M - 1)]
        self.side = [torch.cuda.Stream(device=device) for _ in range(self.M)]
        for r in self.layers:
            for m, d in enumerate(r):
                d.s1 = self.side[m]
        self.ev_start = torch.cuda.Event()
        self.ev_end = [torch.cuda.Event() for _ in range(self.M)]
        self.ev_logits = [[torch.cuda.Event() for _ in range(self.M)]]

    def step(self, qs) -> None:
        """Enqueue one L-layer step on the current stream (micro-batch streams
        forked and joined inside)."""
        self._run(qs, graphs=False)

    def _run(self, qs, graphs: bool) -> None:
        # Per layer, every micro-batch's scores are enqueued before the rest
        # of any micro-batch's step, so each cross-stream wait is enqueued
        # right behind the event it waits for (the runtime can otherwise
        # resolve a wait only once later work on the recording stream has
        # been submitted and finished). Micro-batch m > 0 starts its first
        # scores after those of m - 1; from then on the chains run free, one
        # score launch apart.
        s = torch.cuda.current_stream()
        chain = [s] + self.streams[1:]          # micro-batch 0 runs on the caller's stream
        self.ev_start.record(s)
        for st in chain[1:]:
            st.wait_event(self.ev_start)
        for l in range(self.L):
            for m in range(self.M):
                st, d = chain[m], self.layers[l][m]
                if l == 0 and m > 0:
                    st.wait_event(self.ev_logits[0][m - 1])
                d.scores_launch(qs[l][m], stream=st)
                if l == 0:
                    self.ev_logits[0][m].record(st)
            for m in range(self.M):
                with torch.cuda.stream(chain[m]):
                    if graphs:
                        self.layers[l][m].replay_after_scores()
                    else:
                        self.layers[l][m].step(None, scores=False)
        for m in range(1, self.M):
            self.ev_end[m].record(chain[m])
            s.wait_event(self.ev_end[m])

    def capture(self) -> None:
        """Capture, for every (layer, micro-batch), its step after the scores
        as hipGraphs (one per threshold parity). Nothing runs. A replay then
        launches each pair's scores kernel and its graph on the micro-batch's
        stream, in the order and with the events of step()."""
        if len({d.parity for r in self.layers for d in r}) != 1:
            raise ValueError('every layer must be at the same threshold parity')
        for r in self.layers:
            for d in r:
                d.capture(scores=False)

    def replay(self, qs) -> None:
        """One L-layer step through the captured graphs (current stream)."""
        self._run(qs, graphs=True)


class PageTables:
    """Host side of a paged pool: which pages each sequence holds, in token
    order, and which are free. `table` [B, per_seq] int32 is what the kernels
    read (a copy of it goes to the device); entries past a sequence's pages are
    -1. Forked sequences hold the same full pages, each until the last of them
    returns it."""

    def __init__(self, B: int, n_pages: int, page_size: int, per_seq: int):
        self.page_size, self.n_pages, self.per_seq = page_size, n_pages, per_seq
        self.table = np.full((B, per_seq), -1, np.int32)
        self.held = np.zeros(B, np.int64)
        self.free = list(range(n_pages - 1, -1, -1))
        self.more = np.zeros(n_pages, np.int64)     # how many sequences hold a page beside the first
        self.shared = 0                             # their sum

    def need(self, lens) -> np.ndarray:
        """Pages that sequences of these lengths hold."""
        return -(-np.asarray(lens, np.int64) // self.page_size)

    def resize(self, lens) -> bool:
        """Give every sequence the pages of its length, taking free ones and
        returning those it no longer needs; True if the table changed. Raises,
        with nothing changed, if a sequence or the pool cannot hold them."""
        need = self.need(lens)
        if np.any(need > self.per_seq):
            raise ValueError(f'a sequence needs {int(need.max())} pages, its table has {self.per_seq}')
        extra = int((need - self.held).sum())
        if self.shared:                             # a shared page that is returned is free with its last holder
            back = [p for b in np.flatnonzero(need < self.held) for p in self.table[b, need[b]:self.held[b]]]
            pages, times = np.unique(np.array(back, np.int64), return_counts=True)
            extra += len(back) - int(np.sum(times > self.more[pages]))
        if extra > len(self.free):
            raise ValueError(f'{extra} more pages needed, {len(self.free)} are free')
        changed = np.flatnonzero(need != self.held)
        for b in changed[np.argsort((need - self.held)[changed])]:     # those that shrink first
            have, n = int(self.held[b]), int(need[b])
            if n < have:
                back = self.table[b, n:have][::-1]
                if self.shared:
                    others = self.more[back] > 0
                    self.more[back[others]] -= 1    # a sequence holds a page once
                    self.shared -= int(others.sum())
                    back = back[~others]
                self.free.extend(int(p) for p in back)
                self.table[b, n:have] = -1
            else:
                for i in range(have, n):
                    self.table[b, i] = self.free.pop()
            self.held[b] = n
        return len(changed) > 0

    def fork(self, src: int, dst, length: int, share: bool = True):
        """The sequences dst, which hold nothing, get src's pages: its full ones
        shared (share=False: none), the others as pages of their own. Returns
        the copies that makes: (pages of src, pages, their rows that are
        used). Raises, with nothing changed, if the pool cannot hold them."""
        held = int(self.held[src])
        full = length // self.page_size if share else 0
        if len(dst) * (held - full) > len(self.free):
            raise ValueError(f'{len(dst) * (held - full)} more pages needed, {len(self.free)} are free')
        copies = []
        for b in dst:
            self.table[b, :full] = self.table[src, :full]
            self.more[self.table[src, :full]] += 1
            self.shared += full
            for i in range(full, held):
                self.table[b, i] = self.free.pop()
                copies.append((int(self.table[src, i]), int(self.table[b, i]),
                               min(self.page_size, length - i * self.page_size)))
            self.held[b] = held
        return copies


UPLOADS = 8     # uploads of a PagedLayer under way together: a step has one, with an eviction two


class PagedLayer:
    """One resident layer: its pool of pages, page tables and buffers.

    step(q, rows, counts) takes the step's new rows of all sequences, counts[b]
    of them for sequence b (zero, one or a chunk) one after another: they join
    the pages, attend (causal; window and n_sink as in ech_paged_attn), and
    the step returns out [T, H, 512] bf16 and lse [T, H]. With a budget the
    rows' received weights join a running sum (times decay each step), and
    sequences longer than budget + slack are cut down to budget tokens: the
    first n_sink, the last n_recent, and the heaviest between.

    Window, n_sink and causality count the tokens that the cache holds: an
    eviction closes the gaps between those it keeps. With n_recent >= window - 1
    that is the model's own window, since what an eviction drops is out of every
    later row's sight. With fewer, tokens from behind the window come into sight
    again and some inside it are dropped: a window over kept tokens, which is
    another model than the one without evictions, so the layer warns of it.

    The host knows every length (an eviction leaves budget tokens) and uploads
    from pinned memory, so it queues steps without waiting for the device, up to
    UPLOADS uploads ahead of it. place(counts) does the host's part (its copies
    are on the current stream, before the kernels of launch), launch(q, rows)
    the step's kernels, trim() the eviction; a launch of the same T may be
    captured and replayed, the tables and lengths being read in place (the
    kernels' forms are chosen by the step's largest count and length; for a
    captured launch by the max_rows that place was given, else by the layer's).
    Buffers and workspace of a step of at most B rows (decoding) are the
    layer's, and the next step of the same T writes them again; those of more
    rows are new each time.

    Drafted tokens: draft(q, rows, parent, counts) is a step whose rows are
    trees (parent [T] int32, as in ech_paged_tree_attn; None: chains), or place
    with drafts=True and launch with parent. The rows are in the cache until
    accept(kept, n_kept, counts) leaves the accepted ones of each sequence
    (those of ech_draft_verify); nothing else may be placed, forked or released
    before it. DraftStep does both for a model's layers. A layer with a budget takes no
    drafts: the weights that rejected rows hand out would stay.

    fork(src, dst) lets the empty sequences dst go on from src's tokens: they
    share its full pages (with a budget, whose evictions move rows, they get
    copies), and own a copy of the last one.

    Steps of one layer run in the order of their calls, whatever streams these
    name: each call's stream waits for the layer's last one, and a stream other
    than the current one also for what is queued there (the copies of place, the
    last users of the memory that the buffers get). Only a replay is outside of
    this: it has to be on the stream of the place() before it, or to wait for
    that stream, and the next call on the replay's stream, or after it."""

    def __init__(self, B: int, H: int, n_pages: int, max_len: int, max_rows: int, page_size: int = 64,
                 sm_scale: float = 1.0 / 192.0 ** 0.5, window: int = 0, n_sink: int = 0,
                 budget: Optional[int] = None, n_recent: int = 0, slack: int = 0, decay: float = 1.0, device='cuda'):
        if budget is not None and (budget < 1 or n_sink + n_recent > budget or slack < 0):
            raise ValueError('budget must hold n_sink + n_recent tokens, slack must not be negative')
        if budget is not None and n_recent < window - 1:
            warnings.warn(f'n_recent {n_recent} is less than window - 1 = {window - 1}: after an eviction the window '
                          f'reaches over kept tokens that it had left behind', stacklevel=2)
        self.B, self.H, self.max_len, self.max_rows = B, H, max_len, max_rows
        self.sm_scale, self.window, self.n_sink = sm_scale, window, n_sink
        self.budget, self.n_recent, self.slack, self.decay = budget, n_recent, slack, decay
        self.pages = PageTables(B, n_pages, page_size, -(-max_len // page_size))
        dev = dict(device=device)
        self.pool = torch.zeros((n_pages * page_size, 576), dtype=torch.bfloat16, **dev)
        self.device = self.pool.device      # with its index: the current device may change
        self.lens = np.zeros(B, np.int64)
        # [row0 | seq_len | table]: the host's copy, the device's, and what is on its way between them
        n, per = 2 * B + 1, self.pages.per_seq
        self._image = np.zeros(n + B * per, np.int32)
        self._image[n:] = -1
        self.pages.table = self._image[n:].reshape(B, per)
        self._meta = torch.tensor(self._image, **dev)
        self.row0, self.seq_len, self.table = self._meta[:B + 1], self._meta[B + 1:n], self._meta[n:].view(B, per)
        self._ring, self._turn = [], 0
        self.status = torch.zeros(1, dtype=torch.int32, **dev)
        self.acc = torch.zeros((B, max_len), dtype=torch.float32, **dev) if budget is not None else None
        self.kept = torch.empty((B, budget), dtype=torch.int32, **dev) if budget is not None else None
        self.evict_ws = (torch.empty(ech_paged_evict_ws_bytes(B, max_len, budget), dtype=torch.uint8, **dev)
                         if budget is not None else None)
        # of decoding steps: outputs by T, the largest workspace so far, those that graphs hold
        self._bufs, self._ws, self._held = {}, None, []
        self._placed, self._most, self._fixed, self._long, self._sizes = 0, 0, None, 0, {}
        self._drafts = None                 # rows a sequence of the drafts that are placed and not accepted
        self._last = self._stream = self._done = None
        self._leave(self._enter()[1])       # the zeros above come before the first call

    def _enter(self, stream=None):
        """A call's begin: its stream is made to wait for the layer's last call
        and for the current stream. Returns that stream (None: the current one)
        and whether it records a graph; a capture orders nothing, it runs
        nothing. Steps on one stream cost a comparison here: an event a call
        would take 4 us of the device."""
        if self.device.type != 'cuda':      # host logic alone
            return None, False
        now = _raw_stream(self.device.index)
        raw = now if stream is None else _stream(stream)
        if raw == now == self._last:
            self._done = None               # if this call fails half-way, the next one waits for all of it
            return None, torch.cuda.is_current_stream_capturing()
        s = torch.cuda.current_stream(self.device) if raw == now else _as_stream(stream, self.device)
        if _capturing(s):
            return (None if raw == now else s), True
        if raw != now:
            s.wait_stream(torch.cuda.current_stream(self.device))
        if self._last is not None and self._last != raw:
            if self._done is not None:
                s.wait_event(self._done)
            else:
                s.wait_stream(self._stream)
        self._last, self._stream, self._done = raw, s, None
        # the layer's memory is not another's before s is done with it
        for t in (self.pool, self._meta, self.status, self.acc, self.kept, self.evict_ws,
                  self._ws, *(t for pair in self._bufs.values() for t in pair)):
            if t is not None:
                t.record_stream(s)
        return (None if raw == now else s), False

    def _leave(self, capturing: bool) -> None:
        """A call's end. A stream that is not torch's own may be destroyed
        before the next call: it is marked now."""
        if self._last and not capturing and self._stream.stream_id == self._last:
            self._done = self._stream.record_event()

    def _upload(self, first: int, last: int) -> None:
        """Numbers first .. last - 1 of [row0 | seq_len | table] go to the device,
        on the current stream. They leave from pinned memory, UPLOADS blocks in
        turn, so that the host waits only if the device is that many behind."""
        if self.device.type != 'cuda':
            self._meta[first:last].copy_(torch.from_numpy(self._image[first:last]))
            return
        if len(self._ring) < UPLOADS:
            pinned = torch.empty(len(self._image), dtype=torch.int32, pin_memory=True)
            self._ring.append((pinned, pinned.numpy(), torch.cuda.Event()))
            self._turn = len(self._ring) - 1
        pinned, block, done = self._ring[self._turn]
        self._turn = (self._turn + 1) % UPLOADS
        done.synchronize()                  # the copy that this block was last used for
        block[first:last] = self._image[first:last]
        self._meta[first:last].copy_(pinned[first:last], non_blocking=True)
        done.record(torch.cuda.current_stream(self.device))

    def _place_lens(self) -> None:
        self._image[self.B + 1:2 * self.B + 1] = self.lens

    def _not_captured(self, stream=None) -> None:
        """The host's part of a step is not a graph's: a replay would upload
        what the blocks hold by then."""
        if self.device.type == 'cuda' and (torch.cuda.is_current_stream_capturing() if stream is None else
                                           _capturing(_as_stream(stream, self.device))):
            raise RuntimeError('place, trim, accept, fork and release cannot be captured')

    def _no_drafts(self) -> None:
        if self._drafts is not None:
            raise RuntimeError('drafts are placed: accept has to come first')

    def _bounds(self, capturing: bool) -> Tuple[int, int]:
        """Host bounds of the placed step's rows a sequence and lengths, by which
        the calls choose their forms: its own ones (a few lengths share one, so
        that they share buffers). A captured launch holds for other steps too."""
        if capturing:
            return self.max_rows if self._fixed is None else self._fixed, self.max_len
        return self._most if self._fixed is None else self._fixed, self._long

    def _len_bound(self) -> int:
        """The longest length, up by less than 256 or an eighth."""
        n = int(self.lens.max())
        unit = max(256, (1 << n.bit_length()) // 16)
        return min(self.max_len, round_up(n, unit))

    def _ws_bytes(self, T: int, R: int, L: int, tree: bool = False) -> int:
        n = self._sizes.get((T, R, L, tree))
        if n is None:
            size = ech_paged_tree_attn_ws_bytes if tree else ech_paged_attn_ws_bytes
            n = size(self.B, T, self.H, min(R, T), L, self.window, self.n_sink)
            if self.budget is not None:     # the two calls run one after the other: one workspace
                n = max(n, ech_paged_weight_ws_bytes(self.B, T, self.H, min(R, T), L))
            if T <= self.B:
                self._sizes[T, R, L, tree] = n
        return n

    def _buffers(self, T: int, ws_bytes: int, s, capturing: bool):
        dev, keep = dict(device=self.device), T <= self.B
        got, ws = (self._bufs.get(T), self._ws) if keep else (None, None)
        new = []
        if got is None:
            got = new = [torch.empty((T, self.H, 512), dtype=torch.bfloat16, **dev),
                         torch.empty((T, self.H), dtype=torch.float32, **dev)]
            if keep:
                self._bufs[T] = got
        if ws is None or ws.numel() < ws_bytes:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, **dev)
            new = [*new, ws]
            if keep:
                self._ws = ws
        if keep and capturing and not any(ws is w for w in self._held):
            self._held.append(ws)
        if s is not None:                   # freed when dropped: not before that stream is done with them
            for t in new:
                t.record_stream(s)
        return (*got, ws)

    def _check_rows(self, q: torch.Tensor, rows: torch.Tensor, parent: Optional[torch.Tensor] = None) -> None:
        """Refuse a step's tensors before anything of it is done."""
        if parent is not None and (parent.shape != q.shape[:1] or parent.dtype != torch.int32 or
                                   parent.device != self.device or not parent.is_contiguous()):
            raise ValueError(f'parent: {tuple(parent.shape)} {parent.dtype} on {parent.device}, expected '
                             f'{tuple(q.shape[:1])} int32 on {self.device}, dense')
        T, bits = q.shape[0], (torch.bfloat16, torch.int16, torch.uint16)
        for name, t, shape, types in (('q', q, (T, self.H, 576), bits), ('rows', rows, (T, 576), bits[:1])):
            if t.shape != shape or t.dtype not in types or t.device != self.device:
                raise ValueError(f'{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected {shape} {types[0]} on '
                                 f'{self.device}')
            if t.is_contiguous() and t.data_ptr() % 16 == 0:
                continue
            steps = [st for n, st in zip(t.shape[:-1], t.stride()) if n > 1]
            if t.stride(-1) != 1 or any(st % 8 for st in steps) or t.data_ptr() % 16:
                raise ValueError(f'{name}: strides {t.stride()} at {t.data_ptr():#x}, expected a dense last dimension '
                                 f'and multiples of 16 bytes')
        if T > 1 and rows.stride(0) < 576:
            raise ValueError(f'rows: strides {rows.stride()}, the rows overlap')

    def place(self, counts, max_rows: Optional[int] = None, drafts: bool = False) -> int:
        """Pages and lengths of a step that brings counts[b] rows to sequence
        b; returns T. Raises, with nothing changed, if they do not fit.
        max_rows: the number of rows a sequence that the step's launch is made
        for, where that is to be more than the largest count. A launch captured
        after it is valid for steps that are placed with the same max_rows (1:
        decoding); one captured after a place without it for any step.
        drafts: the rows are drafts, which accept has to follow."""
        self._not_captured()
        self._no_drafts()
        if drafts and self.budget is not None:
            raise ValueError('a layer with a budget takes no drafts')
        counts = np.asarray(counts, np.int64)
        most = self.max_rows if max_rows is None else int(max_rows)
        if most > self.max_rows:
            raise ValueError(f'max_rows {max_rows}, the layer has {self.max_rows}')
        if counts.shape != (self.B,) or np.any(counts < 0) or np.any(counts > most):
            raise ValueError(f'counts must be {self.B} numbers from 0 to max_rows = {most}')
        lens = self.lens + counts
        if np.any(lens > self.max_len):
            raise ValueError(f'a sequence would have {int(lens.max())} tokens, max_len is {self.max_len}')
        moved = self.pages.resize(lens)
        self.lens, self._placed = lens, int(counts.sum())
        self._drafts = counts.copy() if drafts else None
        self._most, self._fixed, self._long = int(counts.max()), None if max_rows is None else most, self._len_bound()
        np.cumsum(counts, out=self._image[1:self.B + 1])
        self._place_lens()
        _, capturing = self._enter()
        self._upload(0, len(self._image) if moved else 2 * self.B + 1)
        self._leave(capturing)
        return self._placed

    def launch(self, q: torch.Tensor, rows: torch.Tensor, stream=None, parent: Optional[torch.Tensor] = None):
        """The kernels of the step that place() prepared: q [T, H, 576], rows
        [T, 576] bf16 -> (out, lse). T is at least the number of rows placed;
        those behind are no sequence's, and their outputs mean nothing. parent
        [T] int32: the rows are trees (at most 256 rows a sequence; a captured
        launch needs a place with such a max_rows before it)."""
        self._check_rows(q, rows, parent)
        return self._launch(q, rows, stream, parent)

    def _launch(self, q: torch.Tensor, rows: torch.Tensor, stream=None, parent: Optional[torch.Tensor] = None):
        T, ps = q.shape[0], self.pages.page_size
        if T < self._placed:
            raise ValueError(f'{self._placed} rows were placed, q has {T}')
        if parent is not None and self._drafts is None:
            raise ValueError('parent: the rows were not placed as drafts')
        s, capturing = self._enter(stream)
        R, L = self._bounds(capturing)
        if parent is not None and R > 256:
            self._leave(capturing)
            raise ValueError(f'trees of up to {R} rows a sequence, 256 are possible')
        out, lse, ws = self._buffers(T, self._ws_bytes(T, R, L, parent is not None), s, capturing)
        ech_paged_append(self.pool, self.table, ps, self.row0, self.seq_len, rows, self.status, stream=stream)
        if parent is None:
            ech_paged_attn(q, self.pool, self.table, ps, self.row0, self.seq_len, R, L, self.sm_scale, out, lse,
                           window=self.window, n_sink=self.n_sink, ws=ws, stream=stream)
        else:
            ech_paged_tree_attn(q, self.pool, self.table, ps, self.row0, self.seq_len, parent, R, L, self.sm_scale, out,
                                lse, window=self.window, n_sink=self.n_sink, ws=ws, stream=stream)
        if self.budget is not None:
            ech_paged_weight(q, lse, self.pool, self.table, ps, self.row0, self.seq_len, R, L, self.sm_scale, self.acc,
                             self.acc, decay=self.decay, window=self.window, n_sink=self.n_sink, ws=ws, stream=stream)
        self._leave(capturing)
        return out, lse

    def trim(self, stream=None) -> bool:
        """Cut sequences longer than budget + slack down to budget tokens (all
        that are longer than budget go with them); True if any was."""
        if self.budget is None or not np.any(self.lens > self.budget + self.slack):
            return False
        self._not_captured(stream)
        s, capturing = self._enter(stream)
        # weights at and past every length are 0 as they are: none is behind the bound
        ech_paged_evict(self.acc, self.seq_len, self._len_bound(), self.budget, self.n_sink, self.n_recent, self.kept,
                        self.seq_len, acc_out=self.acc, pool=self.pool, src_table=self.table, dst_table=self.table,
                        page_size=self.pages.page_size, ws=self.evict_ws, stream=stream)
        self.lens = np.minimum(self.lens, self.budget)
        self._place_lens()                  # as the eviction leaves them on the device
        if self.pages.resize(self.lens):
            with torch.cuda.stream(s):
                self._upload(2 * self.B + 1, len(self._image))
        self._leave(capturing)
        return True

    def step(self, q: torch.Tensor, rows: torch.Tensor, counts):
        """place, launch and trim on the current stream; returns (out, lse)."""
        T = int(np.sum(counts))
        if q.shape[0] != T or rows.shape[0] != T:
            raise ValueError(f'counts name {T} rows, q has {q.shape[0]} and rows {rows.shape[0]}')
        self._check_rows(q, rows)
        self.place(counts)
        got = self._launch(q, rows)
        self.trim()
        return got

    def draft(self, q: torch.Tensor, rows: torch.Tensor, parent: Optional[torch.Tensor], counts):
        """place and launch of a step of drafts on the current stream; returns
        (out, lse). accept follows."""
        T = int(np.sum(counts))
        if q.shape[0] != T or rows.shape[0] != T:
            raise ValueError(f'counts name {T} rows, q has {q.shape[0]} and rows {rows.shape[0]}')
        self._check_rows(q, rows, parent)
        if parent is not None and np.max(counts, initial=0) > 256:
            raise ValueError(f'a tree of {int(np.max(counts))} rows, 256 are possible')
        self.place(counts, drafts=True)
        return self._launch(q, rows, None, parent)

    def _accept_launch(self, kept: torch.Tensor, n_kept: torch.Tensor, stream=None):
        s, capturing = self._enter(stream)
        ech_paged_accept(self.pool, self.table, self.pages.page_size, self.row0, self.seq_len, kept, n_kept, self._most,
                         self.max_len, self.seq_len, stream=stream)
        return s, capturing

    def _accept_host(self, counts: np.ndarray, s, capturing: bool) -> None:
        self.lens = self.lens - self._drafts + counts
        self._drafts = None
        self._place_lens()                  # as the call leaves them on the device
        if self.pages.resize(self.lens):
            with torch.cuda.stream(s):
                self._upload(2 * self.B + 1, len(self._image))
        self._leave(capturing)

    def accept(self, kept: torch.Tensor, n_kept: torch.Tensor, counts, stream=None) -> None:
        """The placed drafts' accepted rows stay, the others leave the cache: kept
        [B, most], n_kept [B] int32 on the device, as ech_draft_verify writes
        them; counts [B]: n_kept's numbers, on the host, at most `most` each."""
        if self._drafts is None:
            raise RuntimeError('no drafts are placed')
        self._not_captured(stream)
        if kept.dim() != 2 or kept.shape[0] != self.B:
            raise ValueError(f'kept: shape {tuple(kept.shape)}, expected ({self.B}, most)')
        counts = np.asarray(counts, np.int64)
        # the device cuts n_kept at both bounds: beyond them its lengths are not the host's
        if counts.shape != (self.B,) or np.any(counts < 0) or np.any(counts > np.minimum(self._drafts, kept.shape[1])):
            raise ValueError(f'counts must be {self.B} numbers from 0 to the rows placed, and to the {kept.shape[1]} that '
                             f'kept holds')
        self._accept_host(counts, *self._accept_launch(kept, n_kept, stream))

    def fork(self, src: int, dst) -> None:
        """The empty sequences dst (a number or several) go on from src's tokens:
        those that launches before it wrote (not between a place and its launch)."""
        self._not_captured()
        self._no_drafts()
        dst = [int(b) for b in np.atleast_1d(dst)]
        if not 0 <= src < self.B or len(set(dst)) < len(dst) or any(
                not 0 <= b < self.B or b == src or self.lens[b] for b in dst):
            raise ValueError(f'fork {src} to {dst}: these have to be different empty sequences')
        copies = self.pages.fork(src, dst, int(self.lens[src]), share=self.budget is None)
        self.lens = self.lens.copy()
        self.lens[dst] = self.lens[src]
        self._place_lens()
        _, capturing = self._enter()
        self._upload(self.B + 1, len(self._image))
        if copies and self.device.type == 'cuda':
            host = torch.tensor(copies, dtype=torch.int32).t().contiguous().pin_memory()
            which = host.to(self.device, non_blocking=True)
            ech_paged_copy(self.pool, self.pages.page_size, which[0], which[1], which[2])
        if self.acc is not None:
            for b in dst:
                self.acc[b].copy_(self.acc[src])
        self._leave(capturing)

    def release(self, b: int) -> None:
        """Sequence b ends: its pages are free and its place starts empty."""
        self._not_captured()
        self._no_drafts()
        lens = self.lens.copy()
        lens[b] = 0
        self.pages.resize(lens)
        self.lens = lens
        self._place_lens()
        _, capturing = self._enter()
        self._upload(self.B + 1, len(self._image))
        if self.acc is not None:
            self.acc[b].zero_()
        self._leave(capturing)


class Accepted(NamedTuple):
    """What a step of drafts came to, on the host: rows kept a sequence, which
    (ascending within the sequence's rows, -1 padded), and the tokens that follow."""
    counts: np.ndarray
    kept: np.ndarray
    next_token: np.ndarray


class DraftStep:
    """The end of a step of drafts, for all resident layers of a model: which
    drafts the target accepts is decided once, and every layer keeps those rows.

    The layers hold the same sequences, and each had its draft() or launch() of
    the step. finish(logits, tokens, u) takes the target's logits [T, V] for
    what follows each row, the rows' tokens and random numbers (as in
    ech_draft_verify), and waits for the decision: the next step's tokens are
    the host's. The layers' rows move while it waits. `most`: rows that a branch
    may keep (its depth + 1). Of a chain of more than 256 rows the first 256 are
    looked at: a branch that has them all ends there, and the token that follows
    is the target's."""

    MOST = 256      # rows of a sequence that ech_draft_verify looks at

    def __init__(self, layers, most: int):
        self.layers = list(layers)
        if not self.layers or len({id(x) for x in self.layers}) < len(self.layers):
            raise ValueError('layers: at least one, each once')
        self.B, self.most, self.device = self.layers[0].B, int(most), self.layers[0].device
        if any(x.B != self.B or x.device != self.device for x in self.layers) or self.most < 1:
            raise ValueError('the layers hold the same sequences on one device; most is at least 1')
        B, n = self.B, self.B * (self.most + 2)
        self._out = torch.empty(n, dtype=torch.int32, device=self.device)
        self._host = torch.empty(n, dtype=torch.int32, pin_memory=self.device.type == 'cuda')
        self.kept, self.n_kept, self.next_token = self._split(self._out)
        # the buffers may be memory that this stream still uses
        self._ws, self._last = None, torch.cuda.current_stream(self.device) if self.device.type == 'cuda' else None
        self._mark()

    def _mark(self) -> None:
        """The buffers' last use so far. A stream that is not torch's own may be
        destroyed before the next step: it is marked now."""
        s = self._last
        self._done = s.record_event() if s is not None and s.cuda_stream and s.stream_id == s.cuda_stream else None

    def _split(self, x: torch.Tensor):
        B = self.B
        return x[:B * self.most].view(B, self.most), x[B * self.most:B * self.most + B], x[B * self.most + B:]

    def finish(self, logits: torch.Tensor, tokens: torch.Tensor, u: torch.Tensor, parent: Optional[torch.Tensor] = None,
               draft: Optional[torch.Tensor] = None, temperature: Optional[torch.Tensor] = None) -> Accepted:
        placed = [x._drafts for x in self.layers]
        if any(p is None or not np.array_equal(p, placed[0]) for p in placed):
            raise RuntimeError('every layer has to have the same drafts placed')
        first = self.layers[0]
        first._not_captured()
        if logits.dim() != 2 or logits.shape[0] < first._placed:
            raise ValueError(f'{first._placed} rows were placed, logits has shape {tuple(logits.shape)}')
        T, V = logits.shape
        rows = min(first._most, self.MOST)
        need = ech_draft_verify_ws_bytes(self.B, T, V, rows, self.most)
        if need == 0:                       # before a layer or a buffer is touched
            raise ValueError(f'{T} rows of {V} tokens cannot be verified: 1 to 2^24 tokens, and rows times ceil((tokens + 7) '
                             f'/ 1024) below 2^31 - 4')
        s = torch.cuda.current_stream(self.device)
        if self._last != s:                 # behind the buffers' last use
            if self._done is not None:
                s.wait_event(self._done)
            else:
                s.wait_stream(self._last)
            self._out.record_stream(s)
            if self._ws is not None:
                self._ws.record_stream(s)
            self._last = s
        self._done = None
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        for x in self.layers:               # the first one's offsets are read: behind its own last call
            x._enter()
        ech_draft_verify(logits, tokens, first.row0, rows, u, self.kept, self.n_kept, self.next_token, parent=parent,
                         draft=draft, temperature=temperature, ws=self._ws)
        self._host.copy_(self._out, non_blocking=True)
        done = torch.cuda.Event()
        done.record(s)
        under_way = [x._accept_launch(self.kept, self.n_kept) for x in self.layers]
        done.synchronize()
        kept, counts, nxt = (x.numpy().copy() for x in self._split(self._host))
        for x, w in zip(self.layers, under_way):
            x._accept_host(counts.astype(np.int64), *w)
        self._mark()
        return Accepted(counts, kept, nxt)


def _as_stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, int) and stream == 0:     # torch takes a 0 for no handle
        return torch.cuda.default_stream(device)
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)


def _capturing(s) -> bool:
    """Whether the current stream or s records a graph."""
    if torch.cuda.is_current_stream_capturing():
        return True
    with torch.cuda.stream(s):
        return torch.cuda.is_current_stream_capturing()
